// C entry points of the operators around the layer: argument checks, workspace
// layout and launches on the caller's stream.  See include/gsa.h.
//
// Lengths and block tables live on the device, so what is wrong in them is found
// there: a kernel leaves the bad part out and records a code in the device's
// status words, which start at zero and keep the first code until
// gsa_operator_status reads and clears them.  Bounded waits have a word of their
// own: a wait looks at its word to stop early, and a bad page of one sequence
// must not stop the others.
#include <math.h>
#include <mutex>
#include <string.h>

#include "../../include/gsa.h"
#include "operators.h"

using namespace gsa;

namespace {

static __device__ int g_status[2];     // bounds, timeout

constexpr int MAX_DEVICES = 64;
std::mutex g_mu;
int* g_addr[MAX_DEVICES] = {};

// device address of the status words on the current device (looked up once)
int status_words(int** out) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= MAX_DEVICES) return GSA_ERR_CUDA;
  std::lock_guard<std::mutex> lock(g_mu);
  if (!g_addr[dev]) {
    void* p = nullptr;
    if (cudaGetSymbolAddress(&p, g_status) != cudaSuccess || !p) return GSA_ERR_CUDA;
    g_addr[dev] = static_cast<int*>(p);
  }
  *out = g_addr[dev];
  return GSA_OK;
}

size_t esize(int dtype) { return dtype == GSA_BF16 ? 2 : 4; }
bool is_dtype(int dtype) { return dtype == GSA_BF16 || dtype == GSA_FP32; }
bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

// Rows of n_outer x n_tokens tokens.  Written rows may not lie on one another: a
// stride of zero is refused where there is more than one.
int check_rows(const gsa_rows* r, int dtype, int64_t n_outer, int64_t n_tokens, bool written) {
  if (r->heads < 1 || r->heads > 65535) return GSA_ERR_INVALID_ARG;
  const int64_t s[3] = {r->stride_outer, r->stride_token, r->stride_head};
  const int64_t n[3] = {n_outer, n_tokens, r->heads};
  const int64_t unit = 16 / static_cast<int64_t>(esize(dtype));
  for (int i = 0; i < 3; ++i) {
    if (n[i] <= 1) continue;               // not used
    if (s[i] < 0 || s[i] % unit) return GSA_ERR_INVALID_ARG;
    if (written && s[i] < D) return GSA_ERR_INVALID_ARG;
  }
  if (n_outer > 0 && n_tokens > 0 && (!r->data || !aligned16(r->data))) return GSA_ERR_INVALID_ARG;
  return GSA_OK;
}

Rows make_rows(const gsa_rows* r) {
  Rows o;
  memset(&o, 0, sizeof(o));
  if (!r) return o;
  o.p = r->data;
  o.so = r->stride_outer;
  o.st = r->stride_token;
  o.sh = r->stride_head;
  o.heads = r->heads;
  return o;
}

int check_op(const gsa_norm_rope* op) {
  if (!op || !is_dtype(op->dtype)) return GSA_ERR_INVALID_ARG;
  if (op->norm < GSA_NORM_NONE || op->norm > GSA_NORM_RMS) return GSA_ERR_INVALID_ARG;
  if (op->norm != GSA_NORM_NONE && !(op->eps >= 0.f && !isinf(op->eps))) return GSA_ERR_INVALID_ARG;
  if (op->rope_axes < 0 || op->rope_axes > 2) return GSA_ERR_INVALID_ARG;
  if (op->rope_axes > 0 && !(op->rope_base > 0.0 && !isinf(op->rope_base))) return GSA_ERR_INVALID_ARG;
  return GSA_OK;
}

// Turns per unit of position, base^(-i / half) / (2 pi), modulo a turn in 64-bit fixed point.
// One power and a product for each next pair (32 powers were 3 us of a call).  In units of 2^-64
// relative: the constant and the quotient 1 each, the power 2 (one place of the last), a product
// 2 + 1, so at most 2 + 31 * 3 = 95.  With a base of 1 or more no frequency is above 1 / (2 pi), so
// it is off by less than 0.16 * 95 + 1 (the cut to fixed point) < 2^5 units of 2^-64 of a turn, and a
// position of up to 2^31 by less than 2^-28 of a turn.  With a base below 1 frequencies grow, up to
// base^-1 / (2 pi) turns, and the error in proportion (still 95 roundings of 2^-64 of the angle).
void make_table(const gsa_norm_rope* op, RopeTable* t) {
  memset(t, 0, sizeof(*t));
  if (op->rope_axes == 0) return;
  const int half = 32 / op->rope_axes;
  const long double ratio = powl(op->rope_base, -1.0L / half);
  long double f = 1.0L / 6.283185307179586476925286766559L;
  for (int i = 0; i < half; ++i, f *= ratio)
    t->f[i] = static_cast<unsigned long long>((f < 1.0L ? f : f - floorl(f)) * 0x1p64L);
}

// weight and bias of one normed tensor
int check_affine(const gsa_norm_rope* op, const void* w, const void* b) {
  if (op->norm != GSA_NORM_NONE && (!w || !aligned16(w))) return GSA_ERR_INVALID_ARG;
  if (b && (op->norm != GSA_NORM_LAYER || !aligned16(b))) return GSA_ERR_INVALID_ARG;
  return GSA_OK;
}

int check_positions(const gsa_norm_rope* op, const int32_t* pos, int64_t n_outer, int64_t so, bool may_lack) {
  if (op->rope_axes == 0) return pos ? GSA_ERR_INVALID_ARG : GSA_OK;
  if (!pos) return may_lack && op->rope_axes == 1 ? GSA_OK : GSA_ERR_INVALID_ARG;
  if (!aligned4(pos) || (n_outer > 1 && so < 0)) return GSA_ERR_INVALID_ARG;
  return GSA_OK;
}

bool count_ok(int64_t n_outer, int64_t n_tokens) {
  return n_outer >= 0 && n_tokens >= 0 && n_outer < (1LL << 31) && n_tokens < (1LL << 31);
}

int check_cache(const gsa_kv_cache* c) {
  if (!c || !is_dtype(c->dtype)) return GSA_ERR_INVALID_ARG;
  if (c->num_pages < 1 || c->kv_heads < 1 || c->batch < 0 || c->max_pages < 0) return GSA_ERR_INVALID_ARG;
  if (c->page_size != 16 && c->page_size != 32 && c->page_size != 64 && c->page_size != 128 && c->page_size != 256)
    return GSA_ERR_UNSUPPORTED;
  // rows of the pool are counted in 32 bits by the copy engine's coordinates
  if (static_cast<int64_t>(c->num_pages) * c->kv_heads * c->page_size >= (1LL << 31)) return GSA_ERR_UNSUPPORTED;
  if (!c->k_pages || !c->v_pages || !aligned16(c->k_pages) || !aligned16(c->v_pages)) return GSA_ERR_INVALID_ARG;
  if (c->batch > 0 && c->max_pages > 0 &&
      (!c->block_table || !aligned4(c->block_table) || (c->batch > 1 && c->table_stride < c->max_pages)))
    return GSA_ERR_INVALID_ARG;
  // places in a sequence, rounded up to a tile of keys, are counted in 32 bits
  if (static_cast<int64_t>(c->max_pages) * c->page_size > 0x7fffffff - 256) return GSA_ERR_UNSUPPORTED;
  return GSA_OK;
}

PagedCache make_cache(const gsa_kv_cache* c) {
  PagedCache p;
  p.k = c->k_pages;
  p.v = c->v_pages;
  p.table = c->block_table;
  p.table_stride = c->table_stride;
  p.num_pages = c->num_pages;
  p.page_shift = 4;
  while ((1 << p.page_shift) < c->page_size) ++p.page_shift;
  p.heads = c->kv_heads;
  p.batch = c->batch;
  p.max_pages = c->max_pages;
  return p;
}

cudaStream_t stream_of(void* s) { return reinterpret_cast<cudaStream_t>(s); }

}  // namespace

#define GSA_TRY(call)                    \
  do {                                   \
    const int rc_ = (call);              \
    if (rc_ != GSA_OK) return rc_;       \
  } while (0)

extern "C" int gsa_qk_norm_rope(const gsa_norm_rope* op, int64_t n_outer, int64_t n_tokens, const gsa_rows* q,
                                const gsa_rows* k, const gsa_rows* v, const gsa_rows* q_out, const gsa_rows* k_out,
                                const gsa_rows* v_out, const void* q_weight, const void* q_bias,
                                const void* k_weight, const void* k_bias, const int32_t* positions,
                                int64_t pos_stride_outer, void* stream) {
  GSA_TRY(check_op(op));
  if (!count_ok(n_outer, n_tokens)) return GSA_ERR_INVALID_ARG;
  const gsa_rows* in[3] = {q, k, v};
  const gsa_rows* out[3] = {q_out, k_out, v_out};
  if (!q && !k && !v) return GSA_ERR_INVALID_ARG;
  NormRopeArgs a;
  memset(&a, 0, sizeof(a));
  for (int i = 0; i < 3; ++i) {
    if (!in[i] != !out[i]) return GSA_ERR_INVALID_ARG;
    if (!in[i]) continue;
    GSA_TRY(check_rows(in[i], op->dtype, n_outer, n_tokens, false));
    GSA_TRY(check_rows(out[i], op->dtype, n_outer, n_tokens, true));
    if (in[i]->heads != out[i]->heads) return GSA_ERR_SHAPE;
    a.in[i] = make_rows(in[i]);
    a.out[i] = make_rows(out[i]);
  }
  if (q) GSA_TRY(check_affine(op, q_weight, q_bias));
  if (k) GSA_TRY(check_affine(op, k_weight, k_bias));
  if (n_outer == 0 || n_tokens == 0) return GSA_OK;
  GSA_TRY(check_positions(op, positions, n_outer, pos_stride_outer, false));
  a.w[0] = q_weight; a.w[1] = k_weight;
  a.b[0] = q_bias; a.b[1] = k_bias;
  a.pos = positions;
  a.pos_so = pos_stride_outer;
  a.n_outer = n_outer;
  a.n_tokens = n_tokens;
  a.eps = op->eps;
  make_table(op, &a.rope);
  return launch_norm_rope(a, op->dtype == GSA_FP32, op->norm, op->rope_axes, stream_of(stream)) == cudaSuccess
             ? GSA_OK : GSA_ERR_CUDA;
}

extern "C" size_t gsa_qk_norm_rope_workspace_bytes(void) { return sizeof(float) * 2 * 128 * NORM_BWD_BLOCKS; }

extern "C" int gsa_qk_norm_rope_backward(const gsa_norm_rope* op, int grad_dtype, int64_t n_outer, int64_t n_tokens,
                                         const gsa_rows* q, const gsa_rows* k, const gsa_rows* dq_out,
                                         const gsa_rows* dk_out, const gsa_rows* dv_out, const gsa_rows* dq,
                                         const gsa_rows* dk, const gsa_rows* dv, const void* q_weight,
                                         const void* k_weight, const int32_t* positions, int64_t pos_stride_outer,
                                         float* dq_weight, float* dq_bias, float* dk_weight, float* dk_bias,
                                         void* workspace, size_t workspace_bytes, void* stream) {
  GSA_TRY(check_op(op));
  if (!is_dtype(grad_dtype) || (grad_dtype == GSA_BF16 && op->dtype != GSA_BF16)) return GSA_ERR_INVALID_ARG;
  if (!count_ok(n_outer, n_tokens)) return GSA_ERR_INVALID_ARG;
  const gsa_rows* x[3] = {q, k, nullptr};
  const gsa_rows* go[3] = {dq_out, dk_out, dv_out};
  const gsa_rows* gi[3] = {dq, dk, dv};
  float* dw[2] = {dq_weight, dk_weight};
  float* db[2] = {dq_bias, dk_bias};
  const void* w[2] = {q_weight, k_weight};
  if (!dq_out && !dk_out && !dv_out) return GSA_ERR_INVALID_ARG;
  NormRopeBwdArgs a;
  memset(&a, 0, sizeof(a));
  bool sums = false;
  for (int i = 0; i < 3; ++i) {
    if (!go[i] != !gi[i]) return GSA_ERR_INVALID_ARG;
    if (i < 2 && (dw[i] || db[i])) {
      // sums of a tensor that is not there, of no norm, or a bias that the norm has not
      if (!go[i] || op->norm == GSA_NORM_NONE || (db[i] && op->norm != GSA_NORM_LAYER)) return GSA_ERR_INVALID_ARG;
      if (!aligned4(dw[i]) || !aligned4(db[i])) return GSA_ERR_INVALID_ARG;
      sums = true;
    }
    if (!go[i]) continue;
    GSA_TRY(check_rows(go[i], grad_dtype, n_outer, n_tokens, false));
    GSA_TRY(check_rows(gi[i], grad_dtype, n_outer, n_tokens, true));
    if (go[i]->heads != gi[i]->heads) return GSA_ERR_SHAPE;
    a.dout[i] = make_rows(go[i]);
    a.din[i] = make_rows(gi[i]);
    if (i == 2 || op->norm == GSA_NORM_NONE) continue;
    if (!x[i]) return GSA_ERR_INVALID_ARG;
    GSA_TRY(check_rows(x[i], op->dtype, n_outer, n_tokens, false));
    if (x[i]->heads != go[i]->heads) return GSA_ERR_SHAPE;
    GSA_TRY(check_affine(op, w[i], nullptr));
    a.in[i] = make_rows(x[i]);
  }
  if (sums && (!workspace || !aligned16(workspace) || workspace_bytes < gsa_qk_norm_rope_workspace_bytes()))
    return GSA_ERR_INVALID_ARG;
  const bool empty = n_outer == 0 || n_tokens == 0;
  if (empty && !sums) return GSA_OK;
  if (!empty) GSA_TRY(check_positions(op, positions, n_outer, pos_stride_outer, false));
  a.pos = positions;
  a.pos_so = pos_stride_outer;
  a.n_outer = n_outer;
  a.n_tokens = n_tokens;
  a.eps = op->eps;
  make_table(op, &a.rope);
  a.part = sums ? static_cast<float*>(workspace) : nullptr;
  for (int i = 0; i < 2; ++i) {
    a.w[i] = w[i];
    a.dw[i] = dw[i];
    a.db[i] = db[i];
  }
  return launch_norm_rope_bwd(a, op->dtype == GSA_FP32, grad_dtype == GSA_FP32, op->norm, op->rope_axes,
                              stream_of(stream)) == cudaSuccess
             ? GSA_OK : GSA_ERR_CUDA;
}

extern "C" int gsa_cache_append(const gsa_kv_cache* cache, const gsa_norm_rope* op, int64_t n_tokens,
                                const gsa_rows* k, const gsa_rows* v, const int32_t* cu_tokens,
                                const int32_t* start, const void* k_weight, const void* k_bias,
                                const int32_t* positions, void* stream) {
  GSA_TRY(check_cache(cache));
  GSA_TRY(check_op(op));
  if (!k || !v || !count_ok(1, n_tokens)) return GSA_ERR_INVALID_ARG;
  if (op->dtype != cache->dtype) return GSA_ERR_INVALID_ARG;
  GSA_TRY(check_rows(k, op->dtype, 1, n_tokens, false));
  GSA_TRY(check_rows(v, op->dtype, 1, n_tokens, false));
  if (k->heads != cache->kv_heads || v->heads != cache->kv_heads) return GSA_ERR_SHAPE;
  GSA_TRY(check_affine(op, k_weight, k_bias));
  if (n_tokens == 0 || cache->batch == 0) return GSA_OK;
  if (!cu_tokens || !start || !aligned4(cu_tokens) || !aligned4(start)) return GSA_ERR_INVALID_ARG;
  GSA_TRY(check_positions(op, positions, 1, 0, true));
  int* words = nullptr;
  GSA_TRY(status_words(&words));
  NormRopeArgs a;
  memset(&a, 0, sizeof(a));
  a.c = make_cache(cache);
  a.in[1] = make_rows(k);
  a.in[2] = make_rows(v);
  a.out[1].p = cache->k_pages;
  a.out[2].p = cache->v_pages;
  a.out[1].sh = a.out[2].sh = static_cast<long long>(cache->page_size) * D;
  a.out[1].heads = a.out[2].heads = cache->kv_heads;
  a.w[1] = k_weight;
  a.b[1] = k_bias;
  a.cu = cu_tokens;
  a.start = start;
  a.pos = positions;
  a.n_outer = 1;
  a.n_tokens = n_tokens;
  a.eps = op->eps;
  make_table(op, &a.rope);
  a.err = words;
  return launch_append(a, op->dtype == GSA_FP32, op->norm, op->rope_axes, stream_of(stream)) == cudaSuccess
             ? GSA_OK : GSA_ERR_CUDA;
}

static int check_attention_sizes(const gsa_kv_cache* c, int64_t n_tokens, int q_heads, int max_new, int64_t max_len) {
  GSA_TRY(check_cache(c));
  if (!count_ok(1, n_tokens) || max_new < 0 || max_len < 0 || q_heads < 1 || q_heads > 65535) return GSA_ERR_INVALID_ARG;
  if (q_heads % c->kv_heads) return GSA_ERR_SHAPE;
  // sequences and key heads, and the tiles of one (at least 64 rows), are dimensions of the grid
  const int64_t rows = static_cast<int64_t>(max_new) * (q_heads / c->kv_heads);
  if (rows > 65535ll * 64 || n_tokens * q_heads >= (1LL << 40) ||
      static_cast<int64_t>(c->batch) * c->kv_heads >= (1LL << 31))
    return GSA_ERR_UNSUPPORTED;
  return GSA_OK;
}

extern "C" size_t gsa_cache_attention_workspace_bytes(const gsa_kv_cache* cache, int64_t n_tokens, int q_heads,
                                                      int max_new, int64_t max_len) {
  if (check_attention_sizes(cache, n_tokens, q_heads, max_new, max_len) != GSA_OK) return 0;
  if (n_tokens == 0 || cache->batch == 0 || max_new == 0) return 0;
  return plan_cache_attn(cache->dtype == GSA_FP32, cache->batch, cache->kv_heads, q_heads, n_tokens, max_new, max_len)
      .bytes;
}

extern "C" int gsa_cache_attention(const gsa_kv_cache* cache, int64_t n_tokens, const gsa_rows* q, const gsa_rows* out,
                                   const int32_t* cu_tokens, const int32_t* lengths, int max_new, int64_t max_len,
                                   int causal, float softmax_scale, float* lse, void* workspace,
                                   size_t workspace_bytes, void* stream) {
  if (!q || !out) return GSA_ERR_INVALID_ARG;
  GSA_TRY(check_attention_sizes(cache, n_tokens, q->heads, max_new, max_len));
  GSA_TRY(check_rows(q, cache->dtype, 1, n_tokens, false));
  GSA_TRY(check_rows(out, cache->dtype, 1, n_tokens, true));
  if (out->heads != q->heads) return GSA_ERR_SHAPE;
  if (!(softmax_scale >= 0.f) || isinf(softmax_scale * LOG2E)) return GSA_ERR_INVALID_ARG;
  if (n_tokens == 0 || cache->batch == 0) return GSA_OK;
  if (!cu_tokens || !lengths || !aligned4(cu_tokens) || !aligned4(lengths) || !aligned4(lse)) return GSA_ERR_INVALID_ARG;
  const bool fp32 = cache->dtype == GSA_FP32;
  // (with max_new 0 the blocks only look for sequences that have tokens all the same)
  const CacheAttnPlan p =
      plan_cache_attn(fp32, cache->batch, cache->kv_heads, q->heads, n_tokens, max_new, max_new ? max_len : 0);
  if (p.bytes && (!workspace || !aligned16(workspace) || workspace_bytes < p.bytes)) return GSA_ERR_INVALID_ARG;
  int* words = nullptr;
  GSA_TRY(status_words(&words));
  CacheAttnArgs a;
  memset(&a, 0, sizeof(a));
  a.c = make_cache(cache);
  a.q = make_rows(q);
  a.out = make_rows(out);
  a.cu = cu_tokens;
  a.len = lengths;
  a.n_tokens = static_cast<int>(n_tokens);
  a.max_new = max_new;
  a.group = q->heads / cache->kv_heads;
  a.causal = causal != 0;
  a.scale_log2 = (softmax_scale > 0.f ? softmax_scale : 0.125f) * LOG2E;
  a.row_tiles = p.row_tiles;
  a.n_split = p.n_split;
  a.tiles_per_split = p.tiles_per_split;
  a.lse = lse;
  if (p.n_split > 1) {
    a.part_o = static_cast<float*>(workspace);
    a.part_ml = a.part_o + static_cast<size_t>(p.n_split) * n_tokens * q->heads * D;
  }
  a.err = words;
  return launch_cache_attn(a, fp32, p.kind, stream_of(stream)) == cudaSuccess ? GSA_OK : GSA_ERR_CUDA;
}

extern "C" int gsa_operator_status(void* stream) {
  int* words = nullptr;
  GSA_TRY(status_words(&words));
  int code[2] = {0, 0};
  if (cudaStreamSynchronize(stream_of(stream)) != cudaSuccess) return GSA_ERR_CUDA;
  if (cudaMemcpy(code, words, sizeof(code), cudaMemcpyDeviceToHost) != cudaSuccess) return GSA_ERR_CUDA;
  if ((code[0] || code[1]) && cudaMemset(words, 0, sizeof(code)) != cudaSuccess) return GSA_ERR_CUDA;
  return code[1] ? code[1] : code[0];
}
