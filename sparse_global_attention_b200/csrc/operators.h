// Host-side launch interface of the operators around the layer (internal).
#pragma once
#include "gsa_kernels.h"

namespace gsa {

// one strided set of rows (64 contiguous elements per outer, token, head)
struct Rows {
  void* p;
  long long so, st, sh;      // strides in elements
  int heads;                 // 0: absent
};

struct RopeTable {
  unsigned long long f[32];  // turns per unit of position of each channel pair, modulo 1, in 2^-64
};

enum NormMode : int { NORM_NONE = 0, NORM_LAYER = 1, NORM_RMS = 2 };

// ---- paged cache ------------------------------------------------------------
struct PagedCache {
  void *k, *v;               // [num_pages][heads][1 << page_shift][64]
  const int* table;          // [batch][max_pages]
  long long table_stride;
  int num_pages, page_shift, heads, batch, max_pages;
};

// ---- norm + rotation --------------------------------------------------------
struct NormRopeArgs {
  Rows in[3], out[3];        // q, k, v
  const void* w[2];          // weights and biases of q and k (bias may be null)
  const void* b[2];
  const int* pos;            // [tokens][axes] per outer entry
  long long pos_so;
  long long n_outer, n_tokens;
  float eps;
  RopeTable rope;
  // appending to a cache: k (in[1]) and v (in[2]) go to the places of packed tokens
  // (n_outer 1), out[1] and out[2] being the pools with their head strides
  PagedCache c;
  const int *cu, *start;
  int* err;                  // bounds word
};
cudaError_t launch_append(const NormRopeArgs& a, bool fp32, int norm, int axes, cudaStream_t st);
cudaError_t launch_norm_rope(const NormRopeArgs& a, bool fp32, int norm, int axes, cudaStream_t st);

// blocks of the backward, two per SM (each writes one row of partial sums)
constexpr int NORM_BWD_BLOCKS = 148 * 2;

struct NormRopeBwdArgs {
  Rows in[2], dout[3], din[3];
  const void* w[2];
  const int* pos;
  long long pos_so;
  long long n_outer, n_tokens;
  float eps;
  RopeTable rope;
  float* part;               // [2][NORM_BWD_BLOCKS][128]: weight and bias sums of q and k per block
  int blocks[3];             // blocks of each tensor (set by the launcher)
  float* dw[2];
  float* db[2];
};
cudaError_t launch_norm_rope_bwd(const NormRopeBwdArgs& a, bool fp32, bool grad_fp32, int norm, int axes,
                                 cudaStream_t st);

// ---- attention over the paged cache --------------------------------------------
struct CacheAttnArgs {
  PagedCache c;
  Rows q, out;               // rows of n_tokens tokens (so unused)
  const int *cu, *len;
  int n_tokens, max_new;
  int group;                 // query heads per key head
  int causal;
  float scale_log2;          // softmax scale * log2(e)
  int row_tiles;             // query tiles of a sequence and key head (of max_new tokens)
  int n_split;               // 1: final output; > 1: partials
  int tiles_per_split;       // key tiles per split; the last split takes what is left
  float* lse;                // optional [q heads][n_tokens]
  float* part_o;             // [n_split][n_tokens * q heads][64] unnormalised
  float* part_ml;            // [n_split][n_tokens * q heads][2] max in raw score units, sum
  int* err;                  // bounds word, timeout word
};
struct CacheAttnPlan {
  int kind;                  // kernel variant
  int row_tiles, n_split, tiles_per_split;
  size_t bytes;              // workspace
};
CacheAttnPlan plan_cache_attn(bool fp32, int batch, int kv_heads, int q_heads, long long n_tokens, int max_new,
                              long long max_len);
cudaError_t launch_cache_attn(const CacheAttnArgs& a, bool fp32, int kind, cudaStream_t st);

// the sequence of the new tokens [cu[b], cu[b + 1]) and its cached length, checked
struct Sequence {
  int first, n, len;
  bool ok;
};
__device__ __forceinline__ Sequence sequence_of(const CacheAttnArgs& a, int b) {
  Sequence s;
  s.first = a.cu[b];
  s.n = a.cu[b + 1] - s.first;
  s.len = a.len[b];
  s.ok = s.first >= 0 && s.n >= 0 && s.n <= a.max_new && s.first <= a.n_tokens - s.n && s.len >= 0;
  return s;
}

}  // namespace gsa
