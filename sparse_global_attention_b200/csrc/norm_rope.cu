// Per-head norm of queries and keys with the position rotation in one pass,
// its gradients, and the same pass writing keys (and values) into a paged cache.
//
// A row is the 64 channels of one (token, head).  Eight lanes hold a row, eight
// channels each, so a warp works on four heads of a token at a time with one
// 16-byte (bf16) access per lane, and every sum over a row is three shuffles.
// Mean and variance come from the row in registers (the variance from the
// centred values), the rotation pairs are a lane exchange (channel i with i + 32:
// lane ^ 4; i with i + 16 inside a half: lane ^ 2), everything in fp32 with one
// rounding at the store.  One warp takes one token: its 32 angles are computed
// once, one per lane, and serve all heads.  An angle is reduced to a part of a
// turn in 64 bits (position times turns per position, minus the nearest whole
// number), so positions far into a stream lose nothing; what is left goes to
// sincospif.
#include "gsa_common.cuh"
#include "operators.h"

namespace gsa {

namespace {

constexpr int NTHR = 256;
constexpr int WARPS = NTHR / 32;

// eight consecutive channels, kept as loaded until they are used
template <typename T> struct Raw8;
template <> struct Raw8<__nv_bfloat16> {
  uint4 u;
  __device__ __forceinline__ void load(const void* p) { u = __ldcs(reinterpret_cast<const uint4*>(p)); }
  __device__ __forceinline__ void zero() { u = make_uint4(0, 0, 0, 0); }
  __device__ __forceinline__ void get(float* f) const {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = __uint_as_float(w[i] << 16);
      f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
  __device__ __forceinline__ void put(const float* f) {
    u = make_uint4(pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3]), pack_bf16(f[4], f[5]), pack_bf16(f[6], f[7]));
  }
  __device__ __forceinline__ void store(void* p) const { *reinterpret_cast<uint4*>(p) = u; }
};
template <> struct Raw8<float> {
  float4 a, b;
  __device__ __forceinline__ void load(const void* p) {
    a = __ldcs(reinterpret_cast<const float4*>(p));
    b = __ldcs(reinterpret_cast<const float4*>(p) + 1);
  }
  __device__ __forceinline__ void zero() { a = b = make_float4(0.f, 0.f, 0.f, 0.f); }
  __device__ __forceinline__ void get(float* f) const {
    f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w; f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
  }
  __device__ __forceinline__ void put(const float* f) {
    a = make_float4(f[0], f[1], f[2], f[3]);
    b = make_float4(f[4], f[5], f[6], f[7]);
  }
  __device__ __forceinline__ void store(void* p) const {
    reinterpret_cast<float4*>(p)[0] = a;
    reinterpret_cast<float4*>(p)[1] = b;
  }
};

__device__ __forceinline__ float row_sum(float v) {      // over the eight lanes of a row
  v += __shfl_xor_sync(0xffffffffu, v, 1);
  v += __shfl_xor_sync(0xffffffffu, v, 2);
  v += __shfl_xor_sync(0xffffffffu, v, 4);
  return v;
}

// cos and sin of this lane's eight channels for a token at positions p0, p1
template <int AXES>
struct Turn {
  float c[8], s[8];          // s carries the sign of the channel's place in its pair
  __device__ __forceinline__ void set(double f, long long p0, long long p1, int lane) {
    const long long p = (AXES == 2 && lane >= 16) ? p1 : p0;
    double t = static_cast<double>(p) * f;
    t -= rint(t);
    float sn, cs;
    sincospif(static_cast<float>(2.0 * t), &sn, &cs);
    const int ch = lane & 7;
    const int from = AXES == 2 ? 16 * (ch >> 2) + 8 * (ch & 1) : 8 * (ch & 3);
    const bool first = AXES == 2 ? (ch & 2) == 0 : ch < 4;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      c[e] = __shfl_sync(0xffffffffu, cs, from + e);
      const float v = __shfl_sync(0xffffffffu, sn, from + e);
      s[e] = first ? -v : v;
    }
  }
  // rotate by the angle (DIR = 1) or back (DIR = -1)
  template <int DIR>
  __device__ __forceinline__ void apply(float* y) const {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float o = __shfl_xor_sync(0xffffffffu, y[e], AXES == 2 ? 2 : 4);
      y[e] = DIR > 0 ? fmaf(o, s[e], y[e] * c[e]) : fmaf(-o, s[e], y[e] * c[e]);
    }
  }
};
template <>
struct Turn<0> {
  __device__ __forceinline__ void set(double, long long, long long, int) {}
  template <int DIR>
  __device__ __forceinline__ void apply(float*) const {}
};

// turns per unit of position of this lane's channel pair
template <int AXES>
__device__ __forceinline__ double lane_freq(const RopeTable& r, int lane) {
  if constexpr (AXES == 0) return 0.0;
  return r.f[AXES == 2 ? (lane & 15) : lane];
}

// normalised row (no weight); returns the row's factor
template <int NORM>
__device__ __forceinline__ float norm_row(float* x, float eps) {
  if constexpr (NORM == NORM_NONE) return 1.f;
  if constexpr (NORM == NORM_LAYER) {
    float s = 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) s += x[e];
    const float mean = row_sum(s) * (1.f / D);
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] -= mean;
  }
  float q = 0.f;
#pragma unroll
  for (int e = 0; e < 8; ++e) q = fmaf(x[e], x[e], q);
  const float r = 1.f / sqrtf(row_sum(q) * (1.f / D) + eps);
#pragma unroll
  for (int e = 0; e < 8; ++e) x[e] *= r;
  return r;
}

// weight and bias of a lane's eight channels
template <typename T, int NORM>
struct Affine {
  float w[8], b[8];
  __device__ __forceinline__ void load(const void* wp, const void* bp, int ch) {
    Raw8<T> r;
    r.load(static_cast<const T*>(wp) + 8 * ch);
    r.get(w);
    if constexpr (NORM == NORM_LAYER) {
      r.zero();
      if (bp) r.load(static_cast<const T*>(bp) + 8 * ch);
      r.get(b);
    }
  }
  __device__ __forceinline__ void apply(float* x) const {
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = NORM == NORM_LAYER ? fmaf(x[e], w[e], b[e]) : x[e] * w[e];
  }
};
template <typename T>
struct Affine<T, NORM_NONE> {
  __device__ __forceinline__ void load(const void*, const void*, int) {}
  __device__ __forceinline__ void apply(float*) const {}
};

__device__ __forceinline__ void split_token(long long g, long long n_tokens, long long& o, long long& t) {
  if (g <= 0xffffffffll && n_tokens <= 0xffffffffll) {
    const uint32_t q = static_cast<uint32_t>(g) / static_cast<uint32_t>(n_tokens);
    o = q;
    t = static_cast<uint32_t>(g) - q * static_cast<uint32_t>(n_tokens);
  } else {
    o = g / n_tokens;
    t = g - o * n_tokens;
  }
}

// the heads of one token, 4 U at a time: load, fn(row in registers), store
template <typename TI, typename TO, int U, typename F>
__device__ __forceinline__ void each_row(const TI* in, long long in_sh, TO* out, long long out_sh, int heads, int lane,
                                         F fn) {
  const int r = lane >> 3, ch = lane & 7;
#pragma unroll 1
  for (int h0 = 0; h0 < heads; h0 += 4 * U) {
    Raw8<TI> raw[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int h = h0 + 4 * u + r;
      if (h < heads) raw[u].load(in + h * in_sh + 8 * ch);
      else raw[u].zero();
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int h = h0 + 4 * u + r;
      if (h0 + 4 * u >= heads) break;      // the whole warp
      float x[8];
      raw[u].get(x);
      fn(x);
      Raw8<TO> w;
      w.put(x);
      if (h < heads) w.store(out + h * out_sh + 8 * ch);
    }
  }
}

// blockIdx.y: 0 queries, 1 keys, 2 values (carried along)
template <typename T, int NORM, int AXES>
__global__ void __launch_bounds__(NTHR) norm_rope_kernel(const __grid_constant__ NormRopeArgs a) {
  constexpr int U = sizeof(T) == 2 ? 4 : 2;
  const int role = blockIdx.y;
  const Rows in = a.in[role], out = a.out[role];
  if (in.heads == 0) return;
  const int lane = threadIdx.x & 31;
  const T* src = static_cast<const T*>(in.p);
  T* dst = static_cast<T*>(out.p);
  const long long total = a.n_outer * a.n_tokens, step = static_cast<long long>(gridDim.x) * WARPS;
  Affine<T, NORM> af;
  if (role < 2) af.load(a.w[role], a.b[role], lane & 7);
  const double f = lane_freq<AXES>(a.rope, lane);
  for (long long g = static_cast<long long>(blockIdx.x) * WARPS + (threadIdx.x >> 5); g < total; g += step) {
    long long o, t;
    split_token(g, a.n_tokens, o, t);
    const T* pi = src + o * in.so + t * in.st;
    T* po = dst + o * out.so + t * out.st;
    if (role == 2) {
      each_row<T, T, U>(pi, in.sh, po, out.sh, in.heads, lane, [](float*) {});
      continue;
    }
    Turn<AXES> turn;
    if constexpr (AXES > 0) {
      const int* p = a.pos + o * a.pos_so + t * AXES;
      turn.set(f, p[0], AXES == 2 ? p[AXES - 1] : 0, lane);
    }
    each_row<T, T, U>(pi, in.sh, po, out.sh, in.heads, lane, [&](float* x) {
      norm_row<NORM>(x, a.eps);
      af.apply(x);
      turn.template apply<1>(x);
    });
  }
}

// Gradients: with g the output gradient turned back and h the normalised row,
// db += g, dw += g h, u = g w, dx = r (u - mean(u) - h mean(u h)) (RMS: without
// mean(u)).  A block's weight sums go to its own row of `part`; a second kernel
// adds those in a fixed order.
template <typename T, typename G, int NORM, int AXES>
__global__ void __launch_bounds__(NTHR) norm_rope_bwd_kernel(const __grid_constant__ NormRopeBwdArgs a) {
  constexpr int U = 2;
  const int role = blockIdx.y;
  const Rows gin = a.dout[role], gout = a.din[role];
  if (gin.heads == 0) return;
  const int lane = threadIdx.x & 31, r = lane >> 3, ch = lane & 7;
  const long long total = a.n_outer * a.n_tokens, step = static_cast<long long>(gridDim.x) * WARPS;
  const double f = lane_freq<AXES>(a.rope, lane);
  Affine<T, NORM == NORM_NONE ? NORM_NONE : NORM_RMS> af;
  const int xr = role < 2 ? role : 0;
  const Rows xin = a.in[xr];
  if (role < 2) af.load(a.w[role], nullptr, ch);
  float dw[8], db[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) dw[e] = db[e] = 0.f;
  for (long long g = static_cast<long long>(blockIdx.x) * WARPS + (threadIdx.x >> 5); g < total; g += step) {
    long long o, t;
    split_token(g, a.n_tokens, o, t);
    const G* pg = static_cast<const G*>(gin.p) + o * gin.so + t * gin.st;
    G* po = static_cast<G*>(gout.p) + o * gout.so + t * gout.st;
    if (role == 2) {
      each_row<G, G, U>(pg, gin.sh, po, gout.sh, gin.heads, lane, [](float*) {});
      continue;
    }
    const T* px = static_cast<const T*>(xin.p) + o * xin.so + t * xin.st;
    Turn<AXES> turn;
    if constexpr (AXES > 0) {
      const int* p = a.pos + o * a.pos_so + t * AXES;
      turn.set(f, p[0], AXES == 2 ? p[AXES - 1] : 0, lane);
    }
#pragma unroll 1
    for (int h0 = 0; h0 < gin.heads; h0 += 4 * U) {
      Raw8<G> rg[U];
      Raw8<T> rx[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int h = h0 + 4 * u + r;
        rg[u].zero();
        rx[u].zero();
        if (h < gin.heads) {
          rg[u].load(pg + h * gin.sh + 8 * ch);
          if constexpr (NORM != NORM_NONE) rx[u].load(px + h * xin.sh + 8 * ch);
        }
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int h = h0 + 4 * u + r;
        if (h0 + 4 * u >= gin.heads) break;
        float d[8];
        rg[u].get(d);
        turn.template apply<-1>(d);
        if constexpr (NORM != NORM_NONE) {
          float x[8];
          rx[u].get(x);
          const float rs = norm_row<NORM>(x, a.eps);
          float su = 0.f, sh = 0.f;
          const bool real = h < gin.heads;
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            if (real) {
              db[e] += d[e];
              dw[e] = fmaf(d[e], x[e], dw[e]);
            }
            d[e] *= af.w[e];
            su += d[e];
            sh = fmaf(d[e], x[e], sh);
          }
          const float mh = row_sum(sh) * (1.f / D);
          const float mu = NORM == NORM_LAYER ? row_sum(su) * (1.f / D) : 0.f;
#pragma unroll
          for (int e = 0; e < 8; ++e) d[e] = rs * (d[e] - mu - x[e] * mh);
        }
        Raw8<G> w;
        w.put(d);
        if (h < gin.heads) w.store(po + h * gout.sh + 8 * ch);
      }
    }
  }
  if constexpr (NORM != NORM_NONE) {
    if (role == 2 || !a.part) return;
    __shared__ float sums[WARPS][128];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      dw[e] += __shfl_xor_sync(0xffffffffu, dw[e], 8);
      dw[e] += __shfl_xor_sync(0xffffffffu, dw[e], 16);
      db[e] += __shfl_xor_sync(0xffffffffu, db[e], 8);
      db[e] += __shfl_xor_sync(0xffffffffu, db[e], 16);
      if (r == 0) {
        sums[threadIdx.x >> 5][8 * ch + e] = dw[e];
        sums[threadIdx.x >> 5][64 + 8 * ch + e] = db[e];
      }
    }
    __syncthreads();
    if (threadIdx.x < 128) {
      float v = 0.f;
#pragma unroll
      for (int w = 0; w < WARPS; ++w) v += sums[w][threadIdx.x];
      a.part[(static_cast<long long>(role) * a.n_part + blockIdx.x) * 128 + threadIdx.x] = v;
    }
  }
}

// one block per tensor: column c of [n_part][128], eight interleaved chains
__global__ void __launch_bounds__(1024) norm_rope_sum_kernel(const float* part, int n_part, float* dw0, float* db0,
                                                             float* dw1, float* db1) {
  __shared__ float sums[8][128];
  const int col = threadIdx.x & 127, grp = threadIdx.x >> 7, role = blockIdx.x;
  float v = 0.f;
  for (int i = grp; i < n_part; i += 8) v += part[(static_cast<long long>(role) * n_part + i) * 128 + col];
  sums[grp][col] = v;
  __syncthreads();
  if (grp == 0) {
#pragma unroll
    for (int i = 1; i < 8; ++i) v += sums[i][col];
    float* out = col < 64 ? (role ? dw1 : dw0) : (role ? db1 : db0);
    if (out) out[col & 63] = v;
  }
}

// last index i in [0, n] with cu[i] <= t (cu[0] <= t), by all lanes of a warp
__device__ __forceinline__ int find_sequence(const int* cu, int n, long long t, int lane) {
  int lo = 0;
  while (n > 0) {
    const int step = (n + 31) >> 5;
    const int at = min((lane + 1) * step, n);
    const bool le = cu[lo + at] <= t;
    const int cnt = __popc(__ballot_sync(0xffffffffu, le));
    const int skip = cnt * step;
    if (skip >= n) return lo + n;
    lo += skip;
    n = min(step, n - skip) - 1;
  }
  return lo;
}

// blockIdx.y: 0 keys (normed and rotated), 1 values; one warp per token
template <typename T, int NORM, int AXES>
__global__ void __launch_bounds__(NTHR) append_kernel(const __grid_constant__ AppendArgs a) {
  constexpr int U = sizeof(T) == 2 ? 4 : 2;
  const int role = blockIdx.y;
  const Rows in = a.in[role];
  const int lane = threadIdx.x & 31;
  const long long step = static_cast<long long>(gridDim.x) * WARPS;
  Affine<T, NORM> af;
  if (role == 0) af.load(a.w, a.b, lane & 7);
  const double f = lane_freq<AXES>(a.rope, lane);
  const int page_size = 1 << a.c.page_shift;
  for (long long t = static_cast<long long>(blockIdx.x) * WARPS + (threadIdx.x >> 5); t < a.n_tokens; t += step) {
    if (a.cu[0] > t) continue;
    const int b = find_sequence(a.cu, a.c.batch, t, lane);
    if (b >= a.c.batch) continue;                       // behind the last sequence
    const int first = a.cu[b];
    const long long place = static_cast<long long>(a.start[b]) + (t - first);
    int page = -1;
    if (first <= t && a.cu[b + 1] > t && a.start[b] >= 0 && (place >> a.c.page_shift) < a.c.max_pages)
      page = a.c.table[b * a.c.table_stride + (place >> a.c.page_shift)];
    if (page < 0 || page >= a.c.num_pages) {
      if (lane == 0) set_error(a.err, ERR_BOUNDS);
      continue;
    }
    const long long row = (static_cast<long long>(page) * a.c.heads << a.c.page_shift) + (place & (page_size - 1));
    const T* pi = static_cast<const T*>(in.p) + t * in.st;
    T* po = static_cast<T*>(role ? a.c.v : a.c.k) + row * D;
    const long long osh = static_cast<long long>(page_size) * D;
    if (role == 1) {
      each_row<T, T, U>(pi, in.sh, po, osh, in.heads, lane, [](float*) {});
      continue;
    }
    Turn<AXES> turn;
    if constexpr (AXES > 0) {
      long long p0 = place, p1 = 0;
      if (a.pos) {
        p0 = a.pos[t * AXES];
        p1 = a.pos[t * AXES + AXES - 1];
      }
      turn.set(f, p0, p1, lane);
    }
    each_row<T, T, U>(pi, in.sh, po, osh, in.heads, lane, [&](float* x) {
      norm_row<NORM>(x, a.eps);
      af.apply(x);
      turn.template apply<1>(x);
    });
  }
}

int blocks_for(long long tokens, int most) {
  const long long b = (tokens + WARPS - 1) / WARPS;
  return static_cast<int>(b < most ? b : most);
}

}  // namespace

// instantiate for the call's norm and number of axes
#define GSA_BY_NORM_AXES(CALL)                                              \
  switch (norm * 3 + axes) {                                                \
    case 0: CALL(0, 0); break;                                              \
    case 1: CALL(0, 1); break;                                              \
    case 2: CALL(0, 2); break;                                              \
    case 3: CALL(1, 0); break;                                              \
    case 4: CALL(1, 1); break;                                              \
    case 5: CALL(1, 2); break;                                              \
    case 6: CALL(2, 0); break;                                              \
    case 7: CALL(2, 1); break;                                              \
    case 8: CALL(2, 2); break;                                              \
    default: return cudaErrorInvalidValue;                                  \
  }

cudaError_t launch_norm_rope(const NormRopeArgs& a, bool fp32, int norm, int axes, cudaStream_t st) {
  const dim3 grid(blocks_for(a.n_outer * a.n_tokens, 1 << 16), a.in[2].heads ? 3 : 2);
#define GSA_CALL(N, A)                                                                                      \
  (fp32 ? norm_rope_kernel<float, N, A><<<grid, NTHR, 0, st>>>(a)                                           \
        : norm_rope_kernel<__nv_bfloat16, N, A><<<grid, NTHR, 0, st>>>(a))
  GSA_BY_NORM_AXES(GSA_CALL)
#undef GSA_CALL
  return cudaGetLastError();
}

cudaError_t launch_norm_rope_bwd(const NormRopeBwdArgs& in, bool fp32, bool grad_fp32, int norm, int axes,
                                 cudaStream_t st) {
  NormRopeBwdArgs a = in;
  a.n_part = blocks_for(a.n_outer * a.n_tokens, NORM_BWD_BLOCKS);
  if (a.n_part > 0) {
    const dim3 grid(a.n_part, a.dout[2].heads ? 3 : 2);
#define GSA_CALL(N, A)                                                                                      \
  (fp32 ? norm_rope_bwd_kernel<float, float, N, A><<<grid, NTHR, 0, st>>>(a)                                \
        : grad_fp32 ? norm_rope_bwd_kernel<__nv_bfloat16, float, N, A><<<grid, NTHR, 0, st>>>(a)            \
                    : norm_rope_bwd_kernel<__nv_bfloat16, __nv_bfloat16, N, A><<<grid, NTHR, 0, st>>>(a))
    GSA_BY_NORM_AXES(GSA_CALL)
#undef GSA_CALL
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  if (a.part && norm != NORM_NONE)
    // a tensor that is left out has no sums to write (its pointers are null)
    norm_rope_sum_kernel<<<2, 1024, 0, st>>>(a.part, a.n_part, a.dw[0], a.db[0], a.dw[1], a.db[1]);
  return cudaGetLastError();
}

cudaError_t launch_append(const AppendArgs& a, bool fp32, int norm, int axes, cudaStream_t st) {
  const dim3 grid(blocks_for(a.n_tokens, 1 << 16), 2);
#define GSA_CALL(N, A)                                                                                      \
  (fp32 ? append_kernel<float, N, A><<<grid, NTHR, 0, st>>>(a)                                              \
        : append_kernel<__nv_bfloat16, N, A><<<grid, NTHR, 0, st>>>(a))
  GSA_BY_NORM_AXES(GSA_CALL)
#undef GSA_CALL
  return cudaGetLastError();
}

}  // namespace gsa
