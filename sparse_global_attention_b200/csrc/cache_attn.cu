// Attention of new tokens over a paged cache.
//
// A block takes a tile of rows of one sequence and key head: row r is the query
// of token r / group and head r % group of the group that shares the key head,
// so the group's heads read each key once.  Softmax is one pass with the running
// maximum and sum per row; rows see keys below their own limit (causal), and the
// key tiles past the tile's largest limit are never read.  With few rows the key
// range is split over blocks and a second kernel joins the parts.
//
// bf16 runs on the tensor cores (tcgen05, TMEM accumulators, K/V pages by TMA,
// one box per page and tile): S = Q K^T from shared memory, P in TMEM, O += P V.
// A stream is 128 rows with S, P and O in TMEM and its softmax warps (thread = row = TMEM
// lane; two warps share 32 rows, 64 keys of a tile each); a block keeps two streams, one
// TMA producer and one MMA issuer.  What bounds a chunk of tokens is the softmax: at 64
// channels a tile's exponentials (16 results per clock and SM) take twice as long as its
// products.  Two streams let one's exponentials run beside the other's waits; the issuer's
// fixed order (S and P V of one stream, then of the other) keeps them out of step, which an
// issuer for each stream did not (1183 against 977 us, 1301 queries of 16 heads over 83,264
// keys, one block per 256 rows), nor turns taken by barriers (1000), three streams
// of 64-key tiles (1404), or reading the next scores under the exponentials (1464).  (With two
// warps per 32 rows and the keys split over three blocks the call takes 670 to 700.)  3 of
// 16 exponentials run on the FMA pipe (913 against 924 us; 4 of 16: 961).
// Variants by the rows of a sequence and key head:
//   ROW_TILES (a chunk of tokens): the streams are two row tiles over the same keys;
//   ONE_TILE (up to 128 rows): the streams take every other tile of the keys for the same
//     rows, and their sums are joined at the end;
//   QUARTERS (up to 32 rows, single tokens): one stream of 128-key tiles, two blocks per
//     SM; the rows are repeated in the four 32-lane quarters of TMEM and each softmax
//     warp takes 32 of a tile's keys for all of them (its P is zero elsewhere), so no
//     warp does four times the exponentials.
// Rows of V that no key stands for (the cache's memory behind a sequence's last
// token, pages that do not exist) are zeroed in shared memory before the product,
// since 0 * NaN is NaN; scores of such keys are replaced, not added to.
//
// fp32 runs on the FMA pipe with the same splits: 64 rows by 64 keys per step through shared
// memory, or, with few rows, warps that stream keys and values through registers.
//
// All mbarrier waits are bounded; one that runs out records GSA_ERR_DEVICE_TIMEOUT.
#include <atomic>
#include <math.h>
#include <cuda.h>
#include <string.h>
#include <type_traits>

#include "operators.h"
#include "tc_ptx.cuh"
#include "tc_softmax.cuh"

namespace gsa {

namespace {

using namespace tc;

constexpr int TM = 128;                  // rows of a tile
constexpr int QTILE = TM * 128;          // bytes of 128 rows of 64 bf16
constexpr float RESCALE_LOG2 = 8.f;      // rescale O when the max grows by > 2^8
constexpr int FMA_PAIRS = 3;              // of 16 pairs of a tile's exponentials, on the FMA pipe
constexpr float LN2 = 0.6931471805599453f;
// kernel variants
enum Kind : int { ROW_TILES = 0, ONE_TILE = 1, QUARTERS = 2, F32_64 = 3, F32_8 = 4, F32_4 = 5 };

template <int KIND>
struct Lay {
  static constexpr bool QUAD = KIND == QUARTERS;
  static constexpr int NS = QUAD ? 1 : 2;                    // streams: TWARP softmax warps each
  static constexpr int R = KIND == ROW_TILES ? 2 : 1;        // row tiles; with one, stream s takes tiles s, s + NS, ..
  static constexpr int STEP = KIND == ONE_TILE ? NS : 1;
  static constexpr int ROWS = QUAD ? 32 : R * TM;
  static constexpr int TK = 128;                             // keys per tile
  static constexpr int NST = QUAD ? 3 : (R == 2 ? 5 : 6);    // K/V ring depth
  static constexpr int HALVES = QUAD ? 1 : 2;                // softmax warps that share 32 rows, 64 keys of a tile each
  static constexpr int TWARP = 4 * HALVES;                   // softmax warps of a stream
  static constexpr int NWARP = TWARP * NS;                   // then the producer and the issuer
  static constexpr int NTHREADS = 32 * (NWARP + 2);
  static constexpr int COLS = QUAD ? 256 : 512;              // TMEM columns: S, O and P of each stream
  static constexpr int TO = TK * NS, TP = TO + 64 * NS;
  static constexpr int TILE = TK * 128;                      // bytes of a tile of K or V
  static constexpr int KV = R * QTILE;
  static constexpr int STAGE = 2 * TILE;
  static constexpr int BAR = KV + NST * STAGE;
  // q_full, full[NST], empty[NST], then s_full, s_free, p_full, pv_done of each stream, fin
  static constexpr int NBAR = 2 + 2 * NST + 4 * NS;
  static constexpr int INFO = BAR + NBAR * 8;                // valid boxes of each stage, "some are not"
  static constexpr int SLOT = INFO + 4 * (NST + 1);
  static constexpr int XCH = (SLOT + 4 + 15) / 16 * 16;      // one float per row between two halves
  static constexpr int BYTES = XCH + (HALVES == 2 ? 4 * TM * NS : 0);
  static constexpr uint32_t IDESC_QK = idesc_bf16(128, TK, false);
  static constexpr uint32_t IDESC_PV = idesc_bf16(128, 64, true);
};
static_assert(2 * (Lay<QUARTERS>::BYTES + 1024) <= 228 * 1024, "two blocks per SM");
static_assert(Lay<ROW_TILES>::BYTES <= 227 * 1024 && Lay<ONE_TILE>::BYTES <= 227 * 1024, "one block per SM");
constexpr int PITCH = 66;                // floats of a row's part (64 sums, max, sum) in shared memory
static_assert(4 * 32 * PITCH * 4 <= Lay<QUARTERS>::NST * Lay<QUARTERS>::STAGE, "the quarters' parts fit the ring");
static_assert(TM * PITCH * 4 <= Lay<ONE_TILE>::NST * Lay<ONE_TILE>::STAGE, "a stream's part fits the ring");

template <int KIND>
struct Bars {
  using L = Lay<KIND>;
  uint32_t base;
  __device__ uint32_t q_full() const { return base; }
  __device__ uint32_t full(int s) const { return base + 8 * (1 + s); }
  __device__ uint32_t empty(int s) const { return base + 8 * (1 + L::NST + s); }
  __device__ uint32_t s_full(int i) const { return base + 8 * (1 + 2 * L::NST + 4 * i); }
  __device__ uint32_t s_free(int i) const { return base + 8 * (2 + 2 * L::NST + 4 * i); }
  __device__ uint32_t p_full(int i) const { return base + 8 * (3 + 2 * L::NST + 4 * i); }
  __device__ uint32_t pv_done(int i) const { return base + 8 * (4 + 2 * L::NST + 4 * i); }
  __device__ uint32_t fin() const { return base + 8 * (1 + 2 * L::NST + 4 * L::NS); }
};

// whether any of the 64 threads of two warps says so (and a barrier between them)
__device__ __forceinline__ bool pair_any(int id, bool p) {
  uint32_t r;
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.u32 p, %2, 0;\n barrier.cta.red.or.pred q, %1, 64, p;\n"
      " selp.u32 %0, 1, 0, q;\n}\n"
      : "=r"(r)
      : "r"(id), "r"(static_cast<uint32_t>(p))
      : "memory");
  return r != 0;
}

// a warp's bounded wait: true if the phase is complete for all its lanes
__device__ __forceinline__ bool wait_all(uint32_t bar, uint32_t parity, int* err) {
  uint32_t ok;
  asm volatile(
      "{\n .reg .pred p, q;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n"
      " vote.sync.all.pred q, p, 0xffffffff;\n selp.u32 %0, 1, 0, q;\n}\n"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  if (ok) return true;
  return __all_sync(0xffffffffu, mbar_wait(bar, parity, err));
}

// values that an asynchronous load has written by now: nothing reads them earlier
template <int N>
__device__ __forceinline__ void tie(uint32_t* v) {
#pragma unroll
  for (int e = 0; e < N; ++e) asm volatile("" : "+r"(v[e]));
}

// the largest of N values, three at a time, in four chains
__device__ __forceinline__ float max3(float a, uint32_t b, uint32_t c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;\n" : "=f"(d) : "f"(a), "f"(__uint_as_float(b)), "f"(__uint_as_float(c)));
  return d;
}
template <int N>
__device__ __forceinline__ float row_max(const uint32_t* v) {
  float m[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) m[k] = fmaxf(__uint_as_float(v[2 * k]), __uint_as_float(v[2 * k + 1]));
#pragma unroll
  for (int e = 8; e < N; e += 8)
#pragma unroll
    for (int k = 0; k < 4; ++k) m[k] = max3(m[k], v[e + 2 * k], v[e + 2 * k + 1]);
  return fmaxf(fmaxf(m[0], m[1]), fmaxf(m[2], m[3]));
}

// Two exponentials on the FMA and integer pipes instead of the exponential unit
// (16 results per clock and SM, what bounds a chunk of tokens): 2^x = 2^n 2^r with n
// the nearest integer, r in [-1/2, 1/2] (Cody and Waite's reduction, exact here), 2^r by
// the degree-4 polynomial of least relative error (2.6e-6 = 2^-18.6, fitted by Remez'
// exchange; bf16 weights keep 2^-8, their fp32 sum 2^-18).  Adding 1.5 * 2^23 + 127 leaves
// n + 127 in the low bits, so one shift gives the float 2^n.  x is held above -127, whose 2^n
// is 0: less than 2^-126.5, and -inf, give 0 as the exponential unit does; NaN stays NaN.
__device__ __forceinline__ void exp2_pair_fma(uint32_t s0, uint32_t s1, float sl2, float nmb, float& l0, float& l1,
                                              float& p0, float& p1) {
  float x0, x1;
  asm("{\n .reg .b64 a, b, c, d;\n"
      " mov.b64 a, {%2, %3};\n mov.b64 b, {%4, %4};\n mov.b64 c, {%5, %5};\n"
      " fma.rn.f32x2 d, a, b, c;\n mov.b64 {%0, %1}, d;\n}\n"
      : "=f"(x0), "=f"(x1)
      : "r"(s0), "r"(s1), "f"(sl2), "f"(nmb));
  asm("max.NaN.f32 %0, %0, 0fC2FE0000;\n" : "+f"(x0));      // -127
  asm("max.NaN.f32 %0, %0, 0fC2FE0000;\n" : "+f"(x1));
  constexpr float MAGIC = 12583039.f;                       // 1.5 * 2^23 + 127
  asm("{\n .reg .b64 x, t, r, p, c, m;\n .reg .b32 t0, t1;\n"
      " mov.b64 x, {%0, %1};\n mov.b64 m, {%4, %4};\n add.rn.f32x2 t, x, m;\n"
      " mov.b64 m, {%5, %5};\n add.rn.f32x2 r, t, m;\n"
      " mov.b64 m, {%6, %6};\n fma.rn.f32x2 r, r, m, x;\n"
      " mov.b64 p, {%7, %7};\n mov.b64 c, {%8, %8};\n fma.rn.f32x2 p, p, r, c;\n"
      " mov.b64 c, {%9, %9};\n fma.rn.f32x2 p, p, r, c;\n"
      " mov.b64 c, {%10, %10};\n fma.rn.f32x2 p, p, r, c;\n"
      " mov.b64 c, {%11, %11};\n fma.rn.f32x2 p, p, r, c;\n"
      " mov.b64 {t0, t1}, t;\n shl.b32 t0, t0, 23;\n shl.b32 t1, t1, 23;\n mov.b64 t, {t0, t1};\n"
      " mul.rn.f32x2 p, p, t;\n mov.b64 {%0, %1}, p;\n"
      " mov.b64 c, {%2, %3};\n add.rn.f32x2 c, c, p;\n mov.b64 {%2, %3}, c;\n}\n"
      : "+f"(x0), "+f"(x1), "+f"(l0), "+f"(l1)
      : "f"(MAGIC), "f"(-MAGIC), "f"(-1.f), "f"(0.009570102207362652f), "f"(0.05591785907745361f),
        "f"(0.240247443318367f), "f"(0.6931217908859253f), "f"(0.9999992847442627f));
  p0 = x0;
  p1 = x1;
}

// where a block's work lies: one tile of rows of one sequence and key head, and
// one split of its key tiles
struct Block {
  int b, h, split;
  Sequence seq;
  int len;                   // cached tokens that the block table can hold
  int row0, rows;            // first row of the tile, rows of the sequence and key head
  int t_begin, ntile;        // key tiles
  bool any;                  // there are rows
};

template <int TROWS, int TKEYS>
__device__ __forceinline__ Block block_of(const CacheAttnArgs& a) {
  Block k;
  // key heads fastest, then sequences, tiles and splits: later splits are those that shorter
  // sequences do not have
  k.b = blockIdx.x / a.c.heads;
  k.h = blockIdx.x - k.b * a.c.heads;
  k.split = blockIdx.z;
  int tile = blockIdx.y;
  k.seq = sequence_of(a, k.b);
  const long long room = static_cast<long long>(a.c.max_pages) << a.c.page_shift;
  k.len = static_cast<int>(min(static_cast<long long>(k.seq.len), room));
  if (threadIdx.x == 0 && (!k.seq.ok || (k.len != k.seq.len && k.seq.n > 0))) set_error(a.err, ERR_BOUNDS);
  k.rows = k.seq.ok ? k.seq.n * a.group : 0;
  // with a causal mask a sequence's last tile has the most keys: every sequence's last one starts first
  if (a.causal) tile = (k.rows + TROWS - 1) / TROWS - 1 - tile;
  k.row0 = tile * TROWS;
  k.any = tile >= 0 && k.row0 < k.rows;
  k.t_begin = k.ntile = 0;
  if (k.any) {
    const int last = min(k.row0 + TROWS, k.rows) - 1;
    int lim = k.len;
    if (a.causal) lim = min(k.len, max(0, k.seq.len - k.seq.n + last / a.group + 1));
    const int all = (lim + TKEYS - 1) / TKEYS;
    k.t_begin = min(k.split * a.tiles_per_split, all);
    const int end = k.split == a.n_split - 1 ? all : min(k.t_begin + a.tiles_per_split, all);
    k.ntile = end - k.t_begin;
  }
  return k;
}

// keys that row r of the sequence sees
__device__ __forceinline__ int row_limit(const CacheAttnArgs& a, const Block& k, int token) {
  return a.causal ? min(k.len, max(0, k.seq.len - k.seq.n + token + 1)) : k.len;
}

// an entry of the block table, -1 if the pool has no such page
__device__ __forceinline__ int page_of(const CacheAttnArgs& a, int raw) {
  return raw >= 0 && raw < a.c.num_pages ? raw : -1;
}

// The join kernel of a split call is launched while the blocks that write the parts still run
// (programmatic dependent launch): they allow it when they start, it waits for their end.
__device__ __forceinline__ void allow_join() { asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory"); }
__device__ __forceinline__ void wait_for_parts() { asm volatile("griddepcontrol.wait;\n" ::: "memory"); }

// a row's result: normalised output and log-sum-exp, or this split's part
template <int N>
__device__ __forceinline__ void write_row(const CacheAttnArgs& a, const Block& blk, int at, int head, int e0,
                                          const float (&o)[N], float m, float l) {
  if (a.n_split == 1) {
    const float inv = l > 0.f ? 1.f / l : (l == l ? 0.f : l);        // a NaN stays one
    __nv_bfloat16* d = static_cast<__nv_bfloat16*>(a.out.p) + at * a.out.st + head * a.out.sh + e0;
#pragma unroll
    for (int e = 0; e < N; e += 8)
      *reinterpret_cast<uint4*>(d + e) =
          make_uint4(pack_bf16(o[e] * inv, o[e + 1] * inv), pack_bf16(o[e + 2] * inv, o[e + 3] * inv),
                     pack_bf16(o[e + 4] * inv, o[e + 5] * inv), pack_bf16(o[e + 6] * inv, o[e + 7] * inv));
    if (a.lse && e0 == 0)
      a.lse[static_cast<long long>(head) * a.n_tokens + at] = l == 0.f ? -INFINITY : (m * a.scale_log2 + log2f(l)) * LN2;
  } else {
    const long long pr = (static_cast<long long>(blk.split) * a.n_tokens + at) * a.q.heads + head;
    if (blk.ntile > 0) {
#pragma unroll
      for (int e = 0; e < N; e += 4)
        *reinterpret_cast<float4*>(a.part_o + pr * D + e0 + e) = make_float4(o[e], o[e + 1], o[e + 2], o[e + 3]);
    }
    if (e0 == 0) *reinterpret_cast<float2*>(a.part_ml + pr * 2) = make_float2(m, l);
  }
}

template <int KIND>
__global__ void __launch_bounds__(Lay<KIND>::NTHREADS, KIND == QUARTERS ? 2 : 1)
    cache_attn_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                      const __grid_constant__ CacheAttnArgs a) {
  using L = Lay<KIND>;
  constexpr int TN = L::TK;
  extern __shared__ __align__(1024) uint8_t smem[];
  const uint32_t sbase = smem_u32(smem);          // 1024-byte aligned: no static shared memory before it
  const Bars<KIND> bars{sbase + L::BAR};
  volatile uint32_t* info = reinterpret_cast<volatile uint32_t*>(smem + L::INFO);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + L::SLOT);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  allow_join();
  if (threadIdx.x == 32 * L::NWARP) {              // while the sequence is looked up
    prefetch_tmap(&tm_k);
    prefetch_tmap(&tm_v);
  }
  const Block blk = block_of<L::ROWS, TN>(a);
  if (!blk.any) return;
  if (sbase & 1023u) {                            // the operands' swizzle needs it
    if (threadIdx.x == 0) set_error(a.err, ERR_BOUNDS);
    return;
  }
  const int ntile = blk.ntile;
  const int nrow = min(L::R, (blk.rows - blk.row0 + TM - 1) / TM);   // row tiles that hold rows
  const int nstream = L::R > 1 ? nrow : L::NS;
  int* err = a.err + 1;

  if (threadIdx.x == 0) {
    mbar_init(bars.q_full(), L::TWARP * nrow);
    for (int s = 0; s < L::NST; ++s) {
      mbar_init(bars.full(s), 1);
      mbar_init(bars.empty(s), 1);
    }
    for (int i = 0; i < L::NS; ++i) {
      mbar_init(bars.s_full(i), 1);
      mbar_init(bars.s_free(i), L::TWARP);       // one arrival per softmax warp
      mbar_init(bars.p_full(i), L::TWARP);
      mbar_init(bars.pv_done(i), 1);
    }
    mbar_init(bars.fin(), 1);
    info[L::NST] = 0;
    fence_mbar_init();
  }
  const int page_size = 1 << a.c.page_shift;
  const int box = min(page_size, TN);             // rows of one copy
  const int box_shift = min(a.c.page_shift, 7);
  const int nbox = TN >> box_shift;

  // The first global loads start before the barrier of the block: the producer's table entries
  // (lanes 0-7 copy a tile's boxes of K, lanes 8-15 those of V), the softmax warps' rows of Q.
  const int* table = a.c.table + blk.b * a.c.table_stride;
  const int my = lane & 7;
  const bool mine = lane < 16 && my < nbox;
  auto slot_of = [&](int it) { return (blk.t_begin + it) * TN + (my << box_shift); };
  auto lookup = [&](int it) {
    const int slot = slot_of(it);
    return mine && it < ntile && slot < blk.len ? table[slot >> a.c.page_shift] : -1;
  };
  constexpr bool QUAD = L::QUAD;
  constexpr int CH = 8 / L::HALVES;               // 16-byte chunks of Q: each warp of a pair one half of a row
  const int stream = warp / L::TWARP;
  const int half = QUAD ? 0 : (warp >> 2) & 1;
  const int r = threadIdx.x & 127;                // row in the tile = TMEM lane
  const int row = blk.row0 + (QUAD ? lane : (L::R > 1 ? stream * TM : 0) + r);
  const bool real = warp < L::NWARP && row < blk.rows;
  const int token = real ? row / a.group : 0;
  const int head = blk.h * a.group + (real ? row - token * a.group : 0);
  const int at = blk.seq.first + token;
  int first_page = -1;
  uint4 qrow[CH];
  if (warp == L::NWARP) first_page = lookup(0);
  if (warp < L::NWARP && (L::R > 1 || stream == 0)) {
    const uint4* src = reinterpret_cast<const uint4*>(
        static_cast<const __nv_bfloat16*>(a.q.p) + at * a.q.st + head * a.q.sh) + CH * half;
#pragma unroll
    for (int c = 0; c < CH; ++c) qrow[c] = real ? __ldg(src + c) : make_uint4(0, 0, 0, 0);
  }
  if (warp == 0) tmem_alloc<L::COLS>(smem_u32(tmem_slot));
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  if (warp == L::NWARP) {
    // ------------------------------------------------------------ TMA producer
    int next = first_page;
    int issued = 0;
    for (int it = 0; it < ntile; ++it) {
      const int s = it % L::NST;
      const int raw = next;
      next = lookup(it + 1);
      if (it >= L::NST && !wait_all(bars.empty(s), ((it / L::NST) - 1) & 1, err)) break;
      const int slot = slot_of(it);
      const bool want = mine && slot < blk.len;
      const int page = want ? page_of(a, raw) : -1;
      const uint32_t good = __ballot_sync(0xffffffffu, page >= 0);
      if (__any_sync(0xffffffffu, want && page < 0) && lane == 0) {
        set_error(a.err, ERR_BOUNDS);
        info[L::NST] = 1;
      }
      if (lane == 0) {
        info[s] = good & 0xffu;
        mbar_expect_tx(bars.full(s), __popc(good) * box * 128);
      }
      __syncwarp();
      if (page >= 0) {
        const int y = ((page * a.c.heads + blk.h) << a.c.page_shift) + (slot & (page_size - 1));
        const uint32_t dst = sbase + L::KV + s * L::STAGE + (lane >= 8 ? L::TILE : 0) + (my << box_shift) * 128;
        tma_load_2d(dst, lane >= 8 ? &tm_v : &tm_k, 0, y, bars.full(s));
      }
      __syncwarp();
      ++issued;
    }
    // drain: every issued copy has landed before the block may exit
    for (int it = max(0, issued - L::NST); it < issued; ++it)
      mbar_wait(bars.full(it % L::NST), (it / L::NST) & 1, err);
  } else if (warp == L::NWARP + 1) {
    // ------------------------------------------------------------ MMA issuer
    // Stream i's n-th tile is j = first_i + n * STEP.  S of tile n and then O += P V of tile n - 1,
    // stream after stream: the fixed order keeps the streams' softmax out of step.
    if (ntile > 0) {
      const bool leader = elect_one();
      const uint64_t dq0 = sdesc_sw128(sbase, 16, 1024);
      const uint64_t dk0 = sdesc_sw128(sbase + L::KV, 16, 1024);
      const uint64_t dv0 = sdesc_sw128(sbase + L::KV + L::TILE, 8192, 1024);
      constexpr uint32_t ST16 = L::STAGE >> 4;
      const int most = (ntile + L::STEP - 1) / L::STEP;
      bool ok = wait_all(bars.q_full(), 0, err);
      for (int n = 0; ok && n <= most; ++n) {
        for (int i = 0; i < nstream; ++i) {
          const int j = (L::R > 1 ? 0 : i) + n * L::STEP, s = j % L::NST;
          if (j < ntile) {
            if (L::R == 1 || i == 0) {
              ok = wait_all(bars.full(s), (j / L::NST) & 1, err);
              if (!ok) break;
              const int kb = (blk.t_begin + j) * TN;
              const uint32_t bits = info[s];
              if (kb + TN > blk.len || bits != (1u << nbox) - 1u) {
                // rows of V without a key
                for (int r = lane; r < TN; r += 32)
                  if (kb + r >= blk.len || !((bits >> (r >> box_shift)) & 1u)) {
                    uint4* p = reinterpret_cast<uint4*>(smem + L::KV + s * L::STAGE + L::TILE + r * 128);
#pragma unroll
                    for (int c = 0; c < 8; ++c) p[c] = make_uint4(0, 0, 0, 0);
                  }
                fence_async_smem();
                __syncwarp();
              }
            }
            // S = Q K^T as soon as the softmax warps hold S of tile n - 1
            if (n > 0) {
              ok = wait_all(bars.s_free(i), (n - 1) & 1, err);
              if (!ok) break;
            }
            tc_fence_after();
            if (leader) {
              const uint64_t dq = dq0 + (L::R > 1 ? i : 0) * (QTILE >> 4), dk = dk0 + s * ST16;
#pragma unroll
              for (int ks = 0; ks < 4; ++ks)
                mma_bf16_ss(tmem + TN * i, dq + 2 * ks, dk + 2 * ks, L::IDESC_QK, ks > 0 ? 1u : 0u);
              mma_commit(bars.s_full(i));
            }
            __syncwarp();
          }
          const int jp = j - L::STEP, sp = (jp + L::NST) % L::NST;
          if (n > 0 && jp < ntile) {
            // O += P V of tile n - 1
            ok = wait_all(bars.p_full(i), (n - 1) & 1, err);
            if (!ok) break;
            tc_fence_after();
            if (leader) {
              const uint64_t dv = dv0 + sp * ST16;
#pragma unroll
              for (int ks = 0; ks < TN / 16; ++ks)
                mma_bf16_ts(tmem + L::TO + 64 * i, tmem + L::TP + TN / 2 * i + 8 * ks, dv + ks * 128, L::IDESC_PV,
                            (n > 1 || ks > 0) ? 1u : 0u);
              mma_commit(bars.pv_done(i));
              if (L::R == 1 || i == nstream - 1) mma_commit(bars.empty(sp));
            }
            __syncwarp();
          }
        }
      }
      if (leader) mma_commit(bars.fin());
      __syncwarp();
      mbar_wait(bars.fin(), 0, err);
    }
  } else if (warp < L::TWARP * nstream) {
    // ------------------------------------------------------------ softmax
    constexpr int NC = QUAD ? 1 : 2;               // 32-key chunks of a tile that a thread takes
    const int i = stream;
    const int first = L::R > 1 ? 0 : i;
    const int count = first < ntile ? (ntile - first + L::STEP - 1) / L::STEP : 0;
    const int c0 = QUAD ? 32 * warp : 64 * half;   // first of its keys
    const int pair_bar = 2 + (warp & 3) + 4 * i;   // both warps of these 32 rows
    float* xch = reinterpret_cast<float*>(smem + L::XCH) + i * TM + r;
    const int lim = real ? row_limit(a, blk, token) : 0x7fffffff;    // rows without a query need no mask
    const uint32_t lane_off = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t tS = tmem + lane_off + TN * i + c0;
    const uint32_t tO = tmem + lane_off + L::TO + 64 * i;
    const uint32_t tP = tmem + lane_off + L::TP + TN / 2 * i;
    const float sl2 = a.scale_log2;
    if (L::R > 1 || i == 0) {
      // this row of Q, into the 128-byte swizzle of the operand
#pragma unroll
      for (int c = 0; c < CH; ++c)
        *reinterpret_cast<uint4*>(smem + (L::R > 1 ? i : 0) * QTILE + swz(r, CH * half + c)) = qrow[c];
      if constexpr (QUAD) {
        // P of the other quarters' keys stays zero
        uint32_t z[32];
#pragma unroll
        for (int e = 0; e < 32; ++e) z[e] = 0;
        tmem_st32(tP, z);
        tmem_st32(tP + 32, z);
        tmem_wait_st();
      }
      fence_async_smem();
      tc_fence_before();
      warp_arrive(bars.q_full());
    }
    float m = -INFINITY, l = 0.f;
    bool ok = true;
    // a wait that ran out skips the later waits, not the steps: the two warps of a pair
    // meet at the same barriers whatever either of them saw
    for (int n = 0; n < count; ++n) {
      const int j = first + n * L::STEP;
      const int kb = (blk.t_begin + j) * TN + c0;
      ok = ok && wait_all(bars.s_full(i), n & 1, err);
      tc_fence_after();
      const bool bad = info[L::NST] != 0;          // some box had no page
      uint32_t v[32 * NC];
#pragma unroll
      for (int c = 0; c < NC; ++c) tmem_ld32(tS + 32 * c, v + 32 * c);
      tmem_wait_ld();
      tie<32 * NC>(v);
      tc_fence_before();
      warp_arrive(bars.s_free(i));
      const bool masked = __any_sync(0xffffffffu, kb + 32 * NC > lim || bad);
      if (masked) {
        // keys of the tile that this row sees: below its limit, in pages that exist (a stage's
        // valid boxes are read in its barrier's phase; it is not refilled before this tile's product)
        uint32_t boxes = ~0u;
        if (bad) {
          ok = ok && wait_all(bars.full(j % L::NST), (j / L::NST) & 1, err);
          boxes = info[j % L::NST];
        }
#pragma unroll
        for (int c = 0; c < NC; ++c) {
          const int left = lim - kb - 32 * c;
          uint32_t msk = left >= 32 ? ~0u : (left <= 0 ? 0u : (1u << left) - 1u);
          // 16-key groups: no box is smaller
          if (!((boxes >> ((c0 + 32 * c) >> box_shift)) & 1u)) msk &= 0xffff0000u;
          if (!((boxes >> ((c0 + 32 * c + 16) >> box_shift)) & 1u)) msk &= 0x0000ffffu;
          apply_mask(v + 32 * c, msk);
        }
      }
      float mx = row_max<32 * NC>(v);
      // move the reference max only when a row's max grew by more than 2^8
      bool grow = (m == -INFINITY) ? (mx != -INFINITY) : ((mx - m) * sl2 > RESCALE_LOG2);
      grow = QUAD ? __any_sync(0xffffffffu, grow) : pair_any(pair_bar, grow);
      float alpha = 1.f;
      if (grow) {
        if constexpr (!QUAD) {
          // the maximum of both halves: a row's weights share one reference
          if (half == 0) *xch = mx;
          named_bar(pair_bar, 64);
          if (half == 1) *xch = mx = fmaxf(mx, *xch);
          named_bar(pair_bar, 64);
          if (half == 0) mx = *xch;
        }
        const float m_new = fmaxf(m, mx);
        const bool had = m != -INFINITY;             // a row without a key so far has nothing in O
        const bool need = had ? (m_new - m) * sl2 > RESCALE_LOG2 : m_new != -INFINITY;
        if (need) {
          alpha = had ? ex2((m - m_new) * sl2) : 0.f;
          m = m_new;
        }
        l *= alpha;
        // by a factor of 0 too: past a rise of 126 (log2 units) nothing of O is left
        grow = __any_sync(0xffffffffu, need && had);
      }
      // P (and O) are free once the previous tile's product has completed
      if (n > 0) {
        ok = ok && wait_all(bars.pv_done(i), (n - 1) & 1, err);
        tc_fence_after();
        if (grow) {
          // each warp of a pair scales its half of the channels
#pragma unroll 1
          for (int c = 0; c < 8 / L::HALVES; ++c) {
            uint32_t w[8];
            tmem_ld8(tO + 32 * half + 8 * c, w);
            tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 8; ++e) w[e] = __float_as_uint(__uint_as_float(w[e]) * alpha);
            tmem_st8(tO + 32 * half + 8 * c, w);
          }
        }
      }
      const float mb = (m == -INFINITY) ? 0.f : m * sl2;
      float l0 = 0.f, l1 = 0.f;
      // Weights are rounded to bf16 (half a step is 2^-8) for the product, since both of its operands are
      // of one type and the values are bf16; their sum takes them in 32 bits.  The error of an output is
      // that of its own rounding once more: 0.0023 of the result's norm against 0.0016 with exact weights.
      auto weights = [&](auto mixed) {
#pragma unroll
        for (int c = 0; c < NC; ++c) {
          uint32_t pk[16];
#pragma unroll
          for (int e = 0; e < 32; e += 2) {
            float p0, p1;
            if (decltype(mixed)::value && ((e / 2) * FMA_PAIRS) % 16 < FMA_PAIRS)
              exp2_pair_fma(v[32 * c + e], v[32 * c + e + 1], sl2, -mb, l0, l1, p0, p1);
            else
              exp2_pair(v[32 * c + e], v[32 * c + e + 1], sl2, -mb, l0, l1, p0, p1);
            pk[e >> 1] = pack_bf16(p0, p1);
          }
          tmem_st16(tP + (c0 >> 1) + 16 * c, pk);
        }
      };
      if (QUAD || masked) weights(std::false_type{});
      else weights(std::true_type{});
      l += l0 + l1;
      tmem_wait_st();
      tc_fence_before();
      warp_arrive(bars.p_full(i));
    }
    if (ok && count > 0) ok = mbar_wait(bars.pv_done(i), (count - 1) & 1, err);
    ok = __all_sync(0xffffffffu, ok);
    tc_fence_after();
    constexpr int NE = 64 / L::HALVES;             // channels that a thread holds at the end
    float o[NE];
    if (ok && count > 0) {
#pragma unroll
      for (int c = 0; c < NE / 32; ++c) {
        uint32_t w[32];
        tmem_ld32(tO + 32 * (half + c), w);
        tmem_wait_ld();
#pragma unroll
        for (int e = 0; e < 32; ++e) o[32 * c + e] = __uint_as_float(w[e]);
      }
    } else {
#pragma unroll
      for (int e = 0; e < NE; ++e) o[e] = 0.f;
    }
    if constexpr (!QUAD) {
      // the sum of both halves
      if (half == 0) *xch = l;
      named_bar(pair_bar, 64);
      if (half == 1) *xch = l = l + *xch;
      named_bar(pair_bar, 64);
      if (half == 0) l = *xch;
    }
    if constexpr (L::R > 1) {
      if (real) write_row(a, blk, at, head, 32 * half, o, m, l);
    } else {
      // Join the streams (or the quarters) of each row.  The ring is idle once all of them are here:
      // every copy has been consumed by a product that has completed.
      float* part = reinterpret_cast<float*>(smem + L::KV);
      constexpr int PARTS = QUAD ? 4 : L::NS;      // parts of a row
      constexpr int PROWS = QUAD ? 32 : TM;        // rows
      named_bar(1, 32 * L::NWARP);
      if (real && (QUAD || i > 0)) {
        float* mine = part + (QUAD ? threadIdx.x : r) * PITCH;
#pragma unroll
        for (int e = 0; e < NE; ++e) mine[32 * half + e] = o[e];
        if (half == 0) {
          mine[64] = m;
          mine[65] = l;
        }
      }
      named_bar(1, 32 * L::NWARP);
      if constexpr (QUAD) {
        // four threads per row, sixteen channels each
        const int rr = threadIdx.x >> 2, e0 = (threadIdx.x & 3) * 16;
        const int row_r = blk.row0 + rr;
        if (row_r < blk.rows) {
          float mx = -INFINITY;
#pragma unroll
          for (int w = 0; w < PARTS; ++w) mx = fmaxf(mx, part[(PROWS * w + rr) * PITCH + 64]);
          const float mu = (mx == -INFINITY) ? 0.f : mx;
          float ls = 0.f, os[16];
#pragma unroll
          for (int e = 0; e < 16; ++e) os[e] = 0.f;
#pragma unroll
          for (int w = 0; w < PARTS; ++w) {
            const float* p = part + (PROWS * w + rr) * PITCH;
            const float f = ex2((p[64] - mu) * sl2);
            ls = fmaf(f, p[65], ls);
#pragma unroll
            for (int e = 0; e < 16; ++e) os[e] = fmaf(f, p[e0 + e], os[e]);
          }
          const int tk = row_r / a.group;
          write_row(a, blk, blk.seq.first + tk, blk.h * a.group + row_r - tk * a.group, e0, os, mx, ls);
        }
      } else if (i == 0 && real) {
        const float* p = part + r * PITCH;
        const float mx = fmaxf(m, p[64]);
        const float mu = (mx == -INFINITY) ? 0.f : mx;
        const float f0 = ex2((m - mu) * sl2), f1 = ex2((p[64] - mu) * sl2);
        l = fmaf(f1, p[65], f0 * l);
#pragma unroll
        for (int e = 0; e < NE; ++e) o[e] = fmaf(f1, p[32 * half + e], f0 * o[e]);
        write_row(a, blk, at, head, 32 * half, o, mx, l);
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 0) tmem_dealloc<L::COLS>(tmem);
}

// ---- fp32 ---------------------------------------------------------------------
// 64 rows by 64 keys per step, 256 threads as 16 x 16: thread (ty, tx) holds 4 rows by
// 4 keys (tx + 16 i) of S and the same rows by channels 4 tx .. of O.  Scores take two channels in
// one instruction (their operands lie side by side; in P V they would have to be moved together,
// which made it 13 % slower).  512 queries of 37 heads over 8192 keys, 296 full blocks: 34
// TFLOP/s, 46 % of the FMA pipe (33 with single products); 4 or 8 rows by 8 keys per thread, which
// read half the shared memory (32 % of its rate instead of 62 %), reached 33 as well: what is left is
// the warps' waits for each step's loads and for the softmax between the two products.
constexpr int FK = 64;                    // keys per tile
constexpr int FP = 68;                    // row pitch in floats: 16-byte reads of 16 rows meet no bank twice
constexpr int TR = 64;
// two products and sums in one instruction
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("{\n .reg .b64 a, b, c;\n mov.b64 a, {%2, %3};\n mov.b64 b, {%4, %5};\n mov.b64 c, {%6, %7};\n"
      " fma.rn.f32x2 a, a, b, c;\n mov.b64 {%0, %1}, a;\n}\n"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return d;
}
// four channels of a row's result, or of this split's part
__device__ __forceinline__ void write_f32(const CacheAttnArgs& a, const Block& blk, int at, int head, int e0, float4 o,
                                          float m, float l) {
  if (a.n_split == 1) {
    const float inv = l > 0.f ? 1.f / l : (l == l ? 0.f : l);        // a NaN stays one
    *reinterpret_cast<float4*>(static_cast<float*>(a.out.p) + at * a.out.st + head * a.out.sh + e0) =
        make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv);
    if (a.lse && e0 == 0)
      a.lse[static_cast<long long>(head) * a.n_tokens + at] = l == 0.f ? -INFINITY : (m * a.scale_log2 + log2f(l)) * LN2;
  } else {
    const long long pr = (static_cast<long long>(blk.split) * a.n_tokens + at) * a.q.heads + head;
    if (blk.ntile > 0) *reinterpret_cast<float4*>(a.part_o + pr * D + e0) = o;
    if (e0 == 0) *reinterpret_cast<float2*>(a.part_ml + pr * 2) = make_float2(m, l);
  }
}

struct FLay {
  static constexpr int Q = 0;
  static constexpr int K = Q + TR * FP * 4;               // two buffers of K, two of V
  static constexpr int V = K + 2 * FK * FP * 4;
  static constexpr int P = V + 2 * FK * FP * 4;
  static constexpr int OK = P + TR * FP * 4;              // keys that exist, two buffers
  static constexpr int BYTES = OK + 2 * FK * 4;
};

__global__ void __launch_bounds__(256, 2) cache_attn_f32_kernel(const __grid_constant__ CacheAttnArgs a) {
  using L = FLay;
  constexpr int R = TR / 16;
  extern __shared__ __align__(1024) uint8_t smem[];
  float* sq = reinterpret_cast<float*>(smem + L::Q);
  float* sp = reinterpret_cast<float*>(smem + L::P);
  float* sk = reinterpret_cast<float*>(smem + L::K);
  float* sv = reinterpret_cast<float*>(smem + L::V);
  int* skey = reinterpret_cast<int*>(smem + L::OK);
  allow_join();
  const Block blk = block_of<TR, FK>(a);
  if (!blk.any) return;
  const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
  const int page_size = 1 << a.c.page_shift;

  for (int i = tid; i < TR * 16; i += 256) {
    const int r = i >> 4, c = i & 15, row = blk.row0 + r;
    float4 w = make_float4(0.f, 0.f, 0.f, 0.f);
    if (row < blk.rows) {
      const int token = row / a.group, head = blk.h * a.group + row - token * a.group;
      w = __ldg(reinterpret_cast<const float4*>(static_cast<const float*>(a.q.p) +
                                                (blk.seq.first + token) * a.q.st + head * a.q.sh) + c);
    }
    *reinterpret_cast<float4*>(sq + r * FP + 4 * c) = w;
  }
  // keys and values of a tile; rows without a key are zero
  auto load = [&](int it, int buf) {
    const int kb = (blk.t_begin + it) * FK;
    for (int i = tid; i < FK * 16; i += 256) {
      const int r = i >> 4, c = i & 15, slot = kb + r;
      int page = -1;
      if (slot < blk.len) {
        page = page_of(a, __ldg(a.c.table + blk.b * a.c.table_stride + (slot >> a.c.page_shift)));
        if (page < 0 && c == 0) set_error(a.err, ERR_BOUNDS);
      }
      const long long off =
          (((static_cast<long long>(max(page, 0)) * a.c.heads + blk.h) << a.c.page_shift) + (slot & (page_size - 1))) * D +
          4 * c;
      const int bytes = page >= 0 ? 16 : 0;
      cp_async16(smem_u32(sk + (buf * FK + r) * FP + 4 * c), static_cast<const float*>(a.c.k) + off, bytes);
      cp_async16(smem_u32(sv + (buf * FK + r) * FP + 4 * c), static_cast<const float*>(a.c.v) + off, bytes);
      if (c == 0) skey[buf * FK + r] = page >= 0;
    }
  };
  int lim[R];
#pragma unroll
  for (int i = 0; i < R; ++i) {
    const int row = blk.row0 + ty * R + i;
    lim[i] = row < blk.rows ? row_limit(a, blk, row / a.group) : 0;
  }
  float m[R], l[R], o[R][4];
#pragma unroll
  for (int i = 0; i < R; ++i) {
    m[i] = -INFINITY;
    l[i] = 0.f;
#pragma unroll
    for (int e = 0; e < 4; ++e) o[i][e] = 0.f;
  }
  if (blk.ntile > 0) load(0, 0);
  cp_async_commit();
  for (int j = 0; j < blk.ntile; ++j) {
    const int buf = j & 1;
    if (j + 1 < blk.ntile) load(j + 1, buf ^ 1);
    cp_async_commit();
    cp_async_wait<1>();
    __syncthreads();
    const float* k = sk + buf * FK * FP;
    const float* v = sv + buf * FK * FP;
    float s[R][4];
    float2 s2[R][4];
#pragma unroll
    for (int i = 0; i < R; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) s2[i][e] = make_float2(0.f, 0.f);
#pragma unroll 4
    for (int d = 0; d < D; d += 4) {
      float4 kv[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) kv[e] = *reinterpret_cast<const float4*>(k + (tx + 16 * e) * FP + d);
#pragma unroll
      for (int i = 0; i < R; ++i) {
        const float4 q = *reinterpret_cast<const float4*>(sq + (ty * R + i) * FP + d);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          s2[i][e] = fma2(make_float2(q.x, q.y), make_float2(kv[e].x, kv[e].y), s2[i][e]);
          s2[i][e] = fma2(make_float2(q.z, q.w), make_float2(kv[e].z, kv[e].w), s2[i][e]);
        }
      }
    }
    const int kb = (blk.t_begin + j) * FK;
    float scale[R];
#pragma unroll
    for (int i = 0; i < R; ++i) {
      float mx = -INFINITY;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int key = tx + 16 * e;
        s[i][e] = s2[i][e].x + s2[i][e].y;
        if (kb + key >= lim[i] || !skey[buf * FK + key]) s[i][e] = -INFINITY;
        mx = fmaxf(mx, s[i][e]);
      }
#pragma unroll
      for (int w = 1; w < 16; w <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, w));
      const float mn = fmaxf(m[i], mx);
      const float mu = mn == -INFINITY ? 0.f : mn;
      const float alpha = exp2f((m[i] - mu) * a.scale_log2);
      m[i] = mn;
      float sum = 0.f;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float p = exp2f((s[i][e] - mu) * a.scale_log2);
        sum += p;
        sp[(ty * R + i) * FP + tx + 16 * e] = p;
      }
#pragma unroll
      for (int w = 1; w < 16; w <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, w);
      l[i] = fmaf(l[i], alpha, sum);
      scale[i] = alpha;
    }
    __syncwarp();                      // a row's P is written and read by one half-warp
    // a tile's sums on their own, then into O: a long cache's are not one chain of additions
    float w[R][4];
#pragma unroll
    for (int i = 0; i < R; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) w[i][e] = 0.f;
#pragma unroll 2
    for (int c = 0; c < FK; c += 4) {
      float4 vv[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) vv[e] = *reinterpret_cast<const float4*>(v + (c + e) * FP + 4 * tx);
#pragma unroll
      for (int i = 0; i < R; ++i) {
        const float4 p = *reinterpret_cast<const float4*>(sp + (ty * R + i) * FP + c);
        const float pe[4] = {p.x, p.y, p.z, p.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          w[i][0] = fmaf(pe[e], vv[e].x, w[i][0]);
          w[i][1] = fmaf(pe[e], vv[e].y, w[i][1]);
          w[i][2] = fmaf(pe[e], vv[e].z, w[i][2]);
          w[i][3] = fmaf(pe[e], vv[e].w, w[i][3]);
        }
      }
    }
#pragma unroll
    for (int i = 0; i < R; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[i][e] = fmaf(o[i][e], scale[i], w[i][e]);
    __syncthreads();                   // the buffer is refilled in the next step
  }
#pragma unroll
  for (int i = 0; i < R; ++i) {
    const int row = blk.row0 + ty * R + i;
    if (row >= blk.rows) continue;
    const int token = row / a.group, head = blk.h * a.group + row - token * a.group;
    const int at = blk.seq.first + token;
    write_f32(a, blk, at, head, 4 * tx, make_float4(o[i][0], o[i][1], o[i][2], o[i][3]), m[i], l[i]);
  }
}

// Few rows: bound by reading the cache.  A warp streams steps of N x 2 keys on its own: a half-warp
// holds a key's 64 channels, four per lane, as loaded from memory; a row's scores of a step are
// partial products of each lane, summed and dealt out over the 16 lanes in one exchange (N values:
// 8 shuffles for 8 keys), so that lane c ends with the score of key 2 (c / (16 / N)) + half; the
// weights are handed back by shuffles for O += p V.  Each warp has its own running maximum and
// sums; the block's eight warps are joined at the end.  A step's keys lie in one page.  16 rows by
// 64 keys through shared memory (one row a thread) read 1.6 TB/s where this reads 5.4 (48
// sequences of 9728 tokens, single new ones, 4 key heads and 16 query heads: 0.96 GB in 175 to 180 us;
// one query head for each key head 152 us, 6.3 TB/s; eight, in tiles of 8 rows, 371 us, 2.6 TB/s:
// bound by the rows' products and exchanges).
template <int R, int N>
__global__ void __launch_bounds__(256, 2) cache_attn_f32_few_kernel(const __grid_constant__ CacheAttnArgs a) {
  constexpr int KEYS = 2 * N, WARPS = 8, PART = 66;
  __shared__ float parts[WARPS][R][PART];
  allow_join();
  const Block blk = block_of<R, FK>(a);
  if (!blk.any) return;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, half = lane >> 4, c = lane & 15;
  const int page_size = 1 << a.c.page_shift;
  const int* table = a.c.table + blk.b * a.c.table_stride;
  float4 q[R], o[R];
  float m[R], l[R];
  int lim[R];
#pragma unroll
  for (int i = 0; i < R; ++i) {
    const int row = blk.row0 + i;
    o[i] = q[i] = make_float4(0.f, 0.f, 0.f, 0.f);
    m[i] = -INFINITY;
    l[i] = 0.f;
    lim[i] = 0;
    if (row < blk.rows) {
      const int token = row / a.group, head = blk.h * a.group + row - token * a.group;
      q[i] = __ldg(reinterpret_cast<const float4*>(static_cast<const float*>(a.q.p) +
                                                   (blk.seq.first + token) * a.q.st + head * a.q.sh) + c);
      lim[i] = row_limit(a, blk, token);
    }
  }
  const int k0 = blk.t_begin * FK, k1 = min((blk.t_begin + blk.ntile) * FK, blk.len);
  int raw = k0 + warp * KEYS < k1 ? __ldg(table + ((k0 + warp * KEYS) >> a.c.page_shift)) : -1;
  for (int kb = k0 + warp * KEYS; kb < k1; kb += WARPS * KEYS) {
    const int page = page_of(a, raw);
    if (page < 0 && lane == 0) set_error(a.err, ERR_BOUNDS);
    const int after = kb + WARPS * KEYS;
    if (after < k1) raw = __ldg(table + (after >> a.c.page_shift));
    const long long row =
        ((static_cast<long long>(max(page, 0)) * a.c.heads + blk.h) << a.c.page_shift) + (kb & (page_size - 1)) + half;
    const float4* pk = reinterpret_cast<const float4*>(static_cast<const float*>(a.c.k) + row * D) + c;
    const float4* pv = reinterpret_cast<const float4*>(static_cast<const float*>(a.c.v) + row * D) + c;
    float4 k[N], v[N];
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const bool there = page >= 0 && kb + 2 * i + half < blk.len;
      k[i] = there ? __ldg(pk + 32 * i) : make_float4(0.f, 0.f, 0.f, 0.f);
    }
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const bool there = page >= 0 && kb + 2 * i + half < blk.len;
      v[i] = there ? __ldg(pv + 32 * i) : make_float4(0.f, 0.f, 0.f, 0.f);
    }
    const int key = kb + 2 * (c / (16 / N)) + half;          // whose score this lane ends with
#pragma unroll
    for (int i = 0; i < R; ++i) {
      if (i > 0 && blk.row0 + i >= blk.rows) break;          // the whole block
      float s[N];
#pragma unroll
      for (int e = 0; e < N; ++e)
        s[e] = fmaf(q[i].x, k[e].x, fmaf(q[i].y, k[e].y, fmaf(q[i].z, k[e].z, q[i].w * k[e].w)));
      // sum over the half-warp's lanes; each exchange halves the values that a lane keeps
      int x = 8;
#pragma unroll
      for (int n = N / 2; n > 0; n >>= 1, x >>= 1) {
        const bool up = (c & x) != 0;
#pragma unroll
        for (int e = 0; e < n; ++e) {
          const float give = up ? s[e] : s[e + n];
          s[e] = (up ? s[e + n] : s[e]) + __shfl_xor_sync(0xffffffffu, give, x);
        }
      }
      for (; x > 0; x >>= 1) s[0] += __shfl_xor_sync(0xffffffffu, s[0], x);
      float sc = page >= 0 && key < lim[i] ? s[0] : -INFINITY;
      float mx = sc;
#pragma unroll
      for (int w = 16 / N; w < 32; w <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, w));
      const float mn = fmaxf(m[i], mx), mu = mn == -INFINITY ? 0.f : mn;
      const float alpha = exp2f((m[i] - mu) * a.scale_log2);
      const float p = exp2f((sc - mu) * a.scale_log2);
      m[i] = mn;
      l[i] = fmaf(l[i], alpha, p);
      o[i].x *= alpha;
      o[i].y *= alpha;
      o[i].z *= alpha;
      o[i].w *= alpha;
#pragma unroll
      for (int e = 0; e < N; ++e) {
        const float pe = __shfl_sync(0xffffffffu, p, (half << 4) | (e * (16 / N)));
        o[i].x = fmaf(pe, v[e].x, o[i].x);
        o[i].y = fmaf(pe, v[e].y, o[i].y);
        o[i].z = fmaf(pe, v[e].z, o[i].z);
        o[i].w = fmaf(pe, v[e].w, o[i].w);
      }
    }
  }
#pragma unroll
  for (int i = 0; i < R; ++i) {
    // the two halves' sums of O; l over the lanes of different keys
    o[i].x += __shfl_xor_sync(0xffffffffu, o[i].x, 16);
    o[i].y += __shfl_xor_sync(0xffffffffu, o[i].y, 16);
    o[i].z += __shfl_xor_sync(0xffffffffu, o[i].z, 16);
    o[i].w += __shfl_xor_sync(0xffffffffu, o[i].w, 16);
#pragma unroll
    for (int w = 16 / N; w < 32; w <<= 1) l[i] += __shfl_xor_sync(0xffffffffu, l[i], w);
    if (half == 0) {
      float* p = parts[warp][i] + 4 * c;
      p[0] = o[i].x;
      p[1] = o[i].y;
      p[2] = o[i].z;
      p[3] = o[i].w;
    }
    if (lane == 0) {
      parts[warp][i][64] = m[i];
      parts[warp][i][65] = l[i];
    }
  }
  __syncthreads();
  const int i = threadIdx.x >> 4, e0 = 4 * (threadIdx.x & 15), row = blk.row0 + i;
  if (i >= R || row >= blk.rows) return;
  float mx = -INFINITY;
#pragma unroll
  for (int w = 0; w < WARPS; ++w) mx = fmaxf(mx, parts[w][i][64]);
  const float mu = mx == -INFINITY ? 0.f : mx;
  float ls = 0.f, os[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int w = 0; w < WARPS; ++w) {
    const float f = exp2f((parts[w][i][64] - mu) * a.scale_log2);
    ls = fmaf(f, parts[w][i][65], ls);
#pragma unroll
    for (int e = 0; e < 4; ++e) os[e] = fmaf(f, parts[w][i][e0 + e], os[e]);
  }
  const int token = row / a.group, head = blk.h * a.group + row - token * a.group;
  write_f32(a, blk, blk.seq.first + token, head, e0, make_float4(os[0], os[1], os[2], os[3]), mx, ls);
}

// ---- joining the splits ---------------------------------------------------------
// o = sum_s 2^((m_s - m) c) o_s / sum_s 2^((m_s - m) c) l_s.  Sixteen lanes hold the 64
// channels of a part; TPR / 16 such groups take a row's parts in turn, each with a
// running maximum, and are joined at the end.  Few parts: 32 threads a row; many (one
// token over a long cache): 128, since the parts' loads are what takes the time (one warp
// with a part at a time took 30 us for 100 parts).  A split that saw no key has l = 0
// and wrote no o; what lies there is not used.
template <typename T, int TPR>
__global__ void __launch_bounds__(128) cache_join_kernel(const __grid_constant__ CacheAttnArgs a) {
  constexpr int G = TPR / 16, RPB = 128 / TPR;
  const int lane = threadIdx.x & 31, sub = threadIdx.x % TPR, g = sub >> 4, e0 = 4 * (sub & 15);
  const long long rows = static_cast<long long>(a.n_tokens) * a.q.heads;
  const long long row = static_cast<long long>(blockIdx.x) * RPB + threadIdx.x / TPR;
  bool real = row < rows;
  const int at = real ? static_cast<int>(row / a.q.heads) : 0;
  const int head = real ? static_cast<int>(row - static_cast<long long>(at) * a.q.heads) : 0;
  // the row's sequence: rows of none, and of a refused one, stay as they are
  if (real) {
    int lo = 0, hi = a.c.batch;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (a.cu[mid] <= at) lo = mid; else hi = mid;
    }
    real = a.cu[lo] <= at && a.cu[lo + 1] > at && sequence_of(a, lo).ok;
  }
  float m = -INFINITY, l = 0.f;
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
  wait_for_parts();
  if (real) {
    constexpr int B = 4;
    for (int s0 = g; s0 < a.n_split; s0 += G * B) {
      float2 ml[B];
      float4 ov[B];
#pragma unroll
      for (int b = 0; b < B; ++b) {
        const int s = min(s0 + b * G, a.n_split - 1);
        ml[b] = *reinterpret_cast<const float2*>(a.part_ml + (s * rows + row) * 2);
        ov[b] = *reinterpret_cast<const float4*>(a.part_o + (s * rows + row) * D + e0);
      }
#pragma unroll
      for (int b = 0; b < B; ++b) {
        if (s0 + b * G >= a.n_split || ml[b].y == 0.f) continue;
        const float mn = fmaxf(m, ml[b].x), mu = mn == -INFINITY ? 0.f : mn;
        const float f0 = ex2((m - mu) * a.scale_log2), f1 = ex2((ml[b].x - mu) * a.scale_log2);
        m = mn;
        l = fmaf(f1, ml[b].y, f0 * l);
        o.x = fmaf(f1, ov[b].x, f0 * o.x);
        o.y = fmaf(f1, ov[b].y, f0 * o.y);
        o.z = fmaf(f1, ov[b].z, f0 * o.z);
        o.w = fmaf(f1, ov[b].w, f0 * o.w);
      }
    }
  }
  auto merge = [&](float m1, float l1, float4 o1) {
    const float mn = fmaxf(m, m1), mu = mn == -INFINITY ? 0.f : mn;
    const float f0 = ex2((m - mu) * a.scale_log2), f1 = ex2((m1 - mu) * a.scale_log2);
    m = mn;
    l = fmaf(f1, l1, f0 * l);
    o.x = fmaf(f1, o1.x, f0 * o.x);
    o.y = fmaf(f1, o1.y, f0 * o.y);
    o.z = fmaf(f1, o1.z, f0 * o.z);
    o.w = fmaf(f1, o1.w, f0 * o.w);
  };
  // the warp's two groups
  {
    const float m1 = __shfl_xor_sync(0xffffffffu, m, 16), l1 = __shfl_xor_sync(0xffffffffu, l, 16);
    float4 o1;
    o1.x = __shfl_xor_sync(0xffffffffu, o.x, 16);
    o1.y = __shfl_xor_sync(0xffffffffu, o.y, 16);
    o1.z = __shfl_xor_sync(0xffffffffu, o.z, 16);
    o1.w = __shfl_xor_sync(0xffffffffu, o.w, 16);
    merge(m1, l1, o1);
  }
  if constexpr (TPR == 128) {
    __shared__ float4 so[4][16];
    __shared__ float2 sml[4];
    const int w = threadIdx.x >> 5;
    if (lane < 16) so[w][lane] = o;
    if (lane == 0) sml[w] = make_float2(m, l);
    __syncthreads();
    if (threadIdx.x >= 16) return;
#pragma unroll
    for (int k = 1; k < 4; ++k) merge(sml[k].x, sml[k].y, so[k][lane]);
  } else if (lane >= 16) {
    return;
  }
  if (!real) return;
  const float inv = l > 0.f ? 1.f / l : (l == l ? 0.f : l);
  T* out = static_cast<T*>(a.out.p) + at * a.out.st + head * a.out.sh + e0;
  if constexpr (sizeof(T) == 2)
    *reinterpret_cast<uint2*>(out) = make_uint2(pack_bf16(o.x * inv, o.y * inv), pack_bf16(o.z * inv, o.w * inv));
  else
    *reinterpret_cast<float4*>(out) = make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv);
  if (a.lse && e0 == 0)
    a.lse[static_cast<long long>(head) * a.n_tokens + at] =
        l == 0.f ? -INFINITY : (m * a.scale_log2 + log2f(l)) * LN2;
}

// ---- host -------------------------------------------------------------------------
// a pool of pages as [rows][64] with boxes of one page (at most a tile's keys)
bool pool_map(CUtensorMap* m, const void* base, const PagedCache& c, int keys) {
  EncodeTiledFn fn = encode_fn();
  if (!fn) return false;
  const int page = 1 << c.page_shift;
  const cuuint64_t dims[2] = {64, static_cast<cuuint64_t>(c.num_pages) * c.heads * page};
  const cuuint64_t strides[1] = {128};
  const cuuint32_t box[2] = {64, static_cast<cuuint32_t>(page < keys ? page : keys)};
  const cuuint32_t estr[2] = {1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(base), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// dynamic shared memory above the default needs the attribute, once per device
template <typename F>
cudaError_t allow_smem(F* kernel, int bytes, std::atomic<unsigned long long>& done) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 64 && ((done.load(std::memory_order_relaxed) >> dev) & 1)) return cudaSuccess;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess && dev < 64) done.fetch_or(1ull << dev, std::memory_order_relaxed);
  return e;
}

template <int KIND>
cudaError_t launch_tc(const CacheAttnArgs& a, dim3 blocks, cudaStream_t st) {
  using L = Lay<KIND>;
  static std::atomic<unsigned long long> done{0};
  cudaError_t e = allow_smem(cache_attn_kernel<KIND>, L::BYTES, done);
  if (e != cudaSuccess) return e;
  CUtensorMap mk, mv;
  if (!pool_map(&mk, a.c.k, a.c, L::TK) || !pool_map(&mv, a.c.v, a.c, L::TK)) return cudaErrorInvalidValue;
  cache_attn_kernel<KIND><<<blocks, L::NTHREADS, L::BYTES, st>>>(mk, mv, a);
  return cudaGetLastError();
}

cudaError_t launch_join(void (*kernel)(CacheAttnArgs), const CacheAttnArgs& a, long long blocks, cudaStream_t st) {
  cudaLaunchAttribute early;
  early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  early.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t c;
  memset(&c, 0, sizeof(c));
  c.gridDim = dim3(static_cast<unsigned>(blocks));
  c.blockDim = dim3(128);
  c.stream = st;
  c.attrs = &early;
  c.numAttrs = 1;
  return cudaLaunchKernelEx(&c, kernel, a);
}

cudaError_t launch_f32(const CacheAttnArgs& a, dim3 blocks, cudaStream_t st) {
  static std::atomic<unsigned long long> done{0};
  cudaError_t e = allow_smem(cache_attn_f32_kernel, FLay::BYTES, done);
  if (e != cudaSuccess) return e;
  cache_attn_f32_kernel<<<blocks, 256, FLay::BYTES, st>>>(a);
  return cudaGetLastError();
}

}  // namespace

CacheAttnPlan plan_cache_attn(bool fp32, int batch, int kv_heads, int q_heads, long long n_tokens, int max_new,
                              long long max_len) {
  CacheAttnPlan p;
  const long long most = n_tokens < max_new ? n_tokens : max_new;
  const long long rows = most * (q_heads / kv_heads);
  // Per variant: rows and keys of a tile, blocks that run at once, and times in us: a key tile of a
  // block alone and with all SMs at work, a block's start.  The times, and those of rounds and join
  // below, are fitted to a sweep of 650 calls of drawn sizes with 1 to 96 parts each: the chosen
  // number of parts takes 3 to 4 % longer than the best one in the mean (one part: 60 %).
  struct Cost {
    int tile, keys, slots;
    double alone, busy, start;
  };
  static const Cost costs[] = {{256, 128, 148, 1.3, 2.3, 4.5},      // ROW_TILES
                               {128, 128, 148, 0.7, 0.8, 5.0},      // ONE_TILE
                               {32, 128, 296, 0.9, 2.3, 5.5},       // QUARTERS
                               {64, 64, 296, 5.9, 10.0, 3.0},       // F32_64
                               {8, 64, 296, 2.4, 3.5, 3.0},         // F32_8
                               {4, 64, 296, 0.95, 2.6, 3.5}};       // F32_4
  p.kind = fp32 ? (rows <= 4 ? F32_4 : rows <= 24 ? F32_8 : F32_64) : (rows <= 32 ? QUARTERS : rows <= 128 ? ONE_TILE : ROW_TILES);
  const Cost& c = costs[p.kind];
  if (max_len > 0x7fffffff) max_len = 0x7fffffff;          // no sequence is longer
  p.row_tiles = static_cast<int>((rows + c.tile - 1) / c.tile);
  if (p.row_tiles < 1) p.row_tiles = 1;
  const long long ktiles = (max_len + c.keys - 1) / c.keys;
  long long ns = 1, most_splits = ktiles;
  if (most_splits > 128) most_splits = 128;
  if (most_splits > 1) {
    // The blocks that have rows (a block with one of its two row tiles takes four fifths of the
    // time), and of their keys what several sequences of different lengths have on average: the
    // lengths are on the device.
    const int half = p.kind == ROW_TILES ? 2 : 1;
    const double group = static_cast<double>(q_heads) / kv_heads;
    const long long units = (rows * half + c.tile - 1) / c.tile;
    double blocks = static_cast<double>(units / half) + (units % half ? 0.8 : 0.0);
    blocks *= batch;
    if (batch > 1) blocks = fmin(blocks, fmax(n_tokens * group / c.tile + 0.5 * batch, batch));
    blocks *= kv_heads;
    const double mean = batch > 1 ? 0.9 : 1.0;
    double best = 1e30;
    // (more than a round and a half of blocks: their order evens them out, and parts only cost)
    for (long long n = 1; n <= most_splits && (n == 1 || blocks < 1.5 * c.slots); ++n) {
      const double chunk = ceil(static_cast<double>(ktiles) / n);
      const double run = blocks * (mean * n + (n > 1 ? 0.5 * (1.0 - mean) : 1.0 - mean));       // blocks with keys
      const double r = run / c.slots;
      const double rounds = r <= 1.0 ? 1.0 : batch > 1 ? fmin(r + 0.3, 1.0 + 2.1 * (r - 1.0)) : ceil(r);
      const double tile_us = c.alone + (c.busy - c.alone) * (r < 1.0 ? r : 1.0);
      // joining: a launch, and the parts written and read once
      const double join = n > 1 ? 2.0 + n * (0.07 + n_tokens * q_heads * 1e-4) : 0.0;
      const double t = rounds * (chunk * tile_us + 0.5 * c.start) + 0.5 * c.start + join;
      if (t < best * 0.95) {
        best = t;
        ns = n;
      }
    }
  }
  p.tiles_per_split = static_cast<int>(ktiles > 0 ? (ktiles + ns - 1) / ns : 1);
  p.n_split = static_cast<int>(ktiles > 0 ? (ktiles + p.tiles_per_split - 1) / p.tiles_per_split : 1);
  p.bytes = p.n_split > 1 ? static_cast<size_t>(p.n_split) * n_tokens * q_heads * (D + 2) * sizeof(float) : 0;
  return p;
}

cudaError_t launch_cache_attn(const CacheAttnArgs& a, bool fp32, int kind, cudaStream_t st) {
  const dim3 blocks(static_cast<unsigned>(a.c.batch) * a.c.heads, a.row_tiles, a.n_split);
  cudaError_t e;
  switch (kind) {
    case ROW_TILES: e = launch_tc<ROW_TILES>(a, blocks, st); break;
    case ONE_TILE: e = launch_tc<ONE_TILE>(a, blocks, st); break;
    case QUARTERS: e = launch_tc<QUARTERS>(a, blocks, st); break;
    case F32_64: e = launch_f32(a, blocks, st); break;
    case F32_8:
      cache_attn_f32_few_kernel<8, 4><<<blocks, 256, 0, st>>>(a);
      e = cudaGetLastError();
      break;
    case F32_4:
      cache_attn_f32_few_kernel<4, 8><<<blocks, 256, 0, st>>>(a);
      e = cudaGetLastError();
      break;
    default: return cudaErrorInvalidValue;
  }
  if (e != cudaSuccess || a.n_split == 1) return e;
  const long long rows = static_cast<long long>(a.n_tokens) * a.q.heads;
  if (a.n_split > 8)
    return fp32 ? launch_join(cache_join_kernel<float, 128>, a, rows, st)
                : launch_join(cache_join_kernel<__nv_bfloat16, 128>, a, rows, st);
  return fp32 ? launch_join(cache_join_kernel<float, 32>, a, (rows + 3) / 4, st)
              : launch_join(cache_join_kernel<__nv_bfloat16, 32>, a, (rows + 3) / 4, st);
}

}  // namespace gsa
