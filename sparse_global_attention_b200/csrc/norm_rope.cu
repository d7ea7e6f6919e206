// Per-head norm of queries and keys with the position rotation in one pass,
// its gradients, and the same pass writing keys (and values) into a paged cache.
//
// A row is the 64 channels of one (token, head).  Eight lanes hold a row and every sum over a
// row is three shuffles.  A warp works on four heads of a token at a time (a quad) or, in large
// calls, on four tokens.  A lane holds four channels and the four that the rotation pairs them with
// (i and i + 32, or i and i + 16 inside a half), so the rotation needs no exchange, and
// the arithmetic runs on pairs of channels (packed fp32: the passes are near the issue
// limit, 1,800 instructions a token of 16 heads in the one-channel form with exchanged
// partners took 123 us where the bytes take 78).  Mean and variance come from the row in
// registers (the variance from the centred values), everything is fp32 with one rounding
// at the store.  The 32 angles of a token are computed once and serve all
// its heads.  An angle is a part of a turn in 64-bit fixed point (position times turns per
// position modulo 2^64 is one integer product, off by less than 2^-28 of a turn: make_table
// has the derivation), so positions far into a stream lose nothing; its upper half goes to
// sincospif, whose argument keeps 2^-26 of a turn.
//
// Bound by HBM.  Each warp loads the rows of four heads a lane before it works on them; a grid
// of what the SMs hold keeps the tokens in flight together, so that the rows of each head are
// written side by side (128 frames of 1296 tokens and 16 heads, 2.04 GB: 363 us, 5.6 TB/s; in
// quads 396 us, in quads with a block for every eight tokens 503 us).
#include "gsa_common.cuh"
#include "operators.h"

namespace gsa {

namespace {

constexpr int NTHR = 256;
constexpr int WARPS = NTHR / 32;
constexpr int FWD_BLOCKS = 148 * 3;      // of the forward at the most: what the SMs hold

// ---- pairs of channels ----------------------------------------------------------
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 d;
  asm("{\n .reg .b64 a, b;\n mov.b64 a, {%2, %3};\n mov.b64 b, {%4, %5};\n add.rn.f32x2 a, a, b;\n"
      " mov.b64 {%0, %1}, a;\n}\n"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  float2 d;
  asm("{\n .reg .b64 a, b;\n mov.b64 a, {%2, %3};\n mov.b64 b, {%4, %5};\n mul.rn.f32x2 a, a, b;\n"
      " mov.b64 {%0, %1}, a;\n}\n"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("{\n .reg .b64 a, b, c;\n mov.b64 a, {%2, %3};\n mov.b64 b, {%4, %5};\n mov.b64 c, {%6, %7};\n"
      " fma.rn.f32x2 a, a, b, c;\n mov.b64 {%0, %1}, a;\n}\n"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return d;
}
__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }

// a lane's eight channels: 0..3 and, in 4..7, the ones that the rotation pairs with them
struct Lane8 {
  float2 v[4];
};

// four channels, kept as loaded until they are used
template <typename T> struct Raw4;
template <> struct Raw4<__nv_bfloat16> {
  uint2 u;
  __device__ __forceinline__ void load(const void* p) { u = __ldcg(static_cast<const uint2*>(p)); }
  __device__ __forceinline__ void zero() { u = make_uint2(0, 0); }
  __device__ __forceinline__ void get(float2* f) const {
    f[0] = make_float2(__uint_as_float(u.x << 16), __uint_as_float(u.x & 0xffff0000u));
    f[1] = make_float2(__uint_as_float(u.y << 16), __uint_as_float(u.y & 0xffff0000u));
  }
  __device__ __forceinline__ void put(const float2* f) {
    u = make_uint2(pack_bf16(f[0].x, f[0].y), pack_bf16(f[1].x, f[1].y));
  }
  __device__ __forceinline__ void store(void* p) const { __stcs(static_cast<uint2*>(p), u); }
};
template <> struct Raw4<float> {
  float4 u;
  __device__ __forceinline__ void load(const void* p) { u = __ldcg(static_cast<const float4*>(p)); }
  __device__ __forceinline__ void zero() { u = make_float4(0.f, 0.f, 0.f, 0.f); }
  __device__ __forceinline__ void get(float2* f) const {
    f[0] = make_float2(u.x, u.y);
    f[1] = make_float2(u.z, u.w);
  }
  __device__ __forceinline__ void put(const float2* f) { u = make_float4(f[0].x, f[0].y, f[1].x, f[1].y); }
  __device__ __forceinline__ void store(void* p) const { __stcs(static_cast<float4*>(p), u); }
};
template <typename T>
struct Raw8 {
  Raw4<T> a, b;
  __device__ __forceinline__ void get(Lane8& x) const {
    a.get(x.v);
    b.get(x.v + 2);
  }
  __device__ __forceinline__ void put(const Lane8& x) {
    a.put(x.v);
    b.put(x.v + 2);
  }
};

// first channel of a lane, and the distance to its partners
template <int AXES>
struct Chan {
  static constexpr int APART = AXES == 0 ? 4 : (AXES == 1 ? 32 : 16);
  __device__ static __forceinline__ int first(int c) {
    return AXES == 0 ? 8 * c : (AXES == 1 ? 4 * c : 32 * (c >> 2) + 4 * (c & 3));
  }
};

__device__ __forceinline__ float row_sum(float v) {      // over the eight lanes of a row
  v += __shfl_xor_sync(0xffffffffu, v, 1);
  v += __shfl_xor_sync(0xffffffffu, v, 2);
  v += __shfl_xor_sync(0xffffffffu, v, 4);
  return v;
}
__device__ __forceinline__ float sum8(float2 a, float2 b, float2 c, float2 d) {
  const float2 s = add2(add2(a, b), add2(c, d));
  return row_sum(s.x + s.y);
}

// cos and sin of this lane's four pairs for a token at positions p0, p1
template <int AXES>
struct Turn {
  float2 c[2], s[2], ns[2];
  __device__ __forceinline__ void set(unsigned long long f, int p0, int p1, int lane) {
    const long long p = AXES == 2 && lane >= 16 ? p1 : p0;
    const long long turn = static_cast<long long>(static_cast<unsigned long long>(p) * f);      // modulo a turn
    float sn, cs;
    sincospif(static_cast<float>(static_cast<int>(turn >> 32)) * 4.656612873077393e-10f, &sn, &cs);   // 2^-31 half turns
    const int from = 4 * (lane & 7);
    float* cp = reinterpret_cast<float*>(c);
    float* sp = reinterpret_cast<float*>(s);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      cp[e] = __shfl_sync(0xffffffffu, cs, from + e);
      sp[e] = __shfl_sync(0xffffffffu, sn, from + e);
    }
#pragma unroll
    for (int k = 0; k < 2; ++k) ns[k] = make_float2(-s[k].x, -s[k].y);
  }
  // the lane's own four pairs, f their turns per unit: every group of eight lanes has a token of its own
  __device__ __forceinline__ void set_own(const unsigned long long* f, int p0, int p1, int lane) {
    const long long p = AXES == 2 && (lane & 4) ? p1 : p0;
    float* cp = reinterpret_cast<float*>(c);
    float* sp = reinterpret_cast<float*>(s);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const long long turn = static_cast<long long>(static_cast<unsigned long long>(p) * f[e]);
      sincospif(static_cast<float>(static_cast<int>(turn >> 32)) * 4.656612873077393e-10f, &sp[e], &cp[e]);
    }
#pragma unroll
    for (int k = 0; k < 2; ++k) ns[k] = make_float2(-s[k].x, -s[k].y);
  }
  // rotate by the angle (DIR = 1) or back (DIR = -1)
  template <int DIR>
  __device__ __forceinline__ void apply(Lane8& y) const {
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const float2 a = y.v[k], b = y.v[2 + k];
      y.v[k] = fma2(b, DIR > 0 ? ns[k] : s[k], mul2(a, c[k]));
      y.v[2 + k] = fma2(a, DIR > 0 ? s[k] : ns[k], mul2(b, c[k]));
    }
  }
};
template <>
struct Turn<0> {
  __device__ __forceinline__ void set(unsigned long long, int, int, int) {}
  __device__ __forceinline__ void set_own(const unsigned long long*, int, int, int) {}
  template <int DIR>
  __device__ __forceinline__ void apply(Lane8&) const {}
};

// turns per unit of position, in 2^-64, of the lane's own four pairs
template <int AXES>
__device__ __forceinline__ void own_freq(const RopeTable& t, int lane, unsigned long long (&f)[4]) {
#pragma unroll
  for (int e = 0; e < 4; ++e) f[e] = AXES == 0 ? 0 : t.f[(4 * (lane & 7) + e) & (AXES == 2 ? 15 : 31)];
}
// and of the pair whose angle this lane computes for the others
template <int AXES>
__device__ __forceinline__ unsigned long long lane_freq(const RopeTable& r, int lane) {
  if constexpr (AXES == 0) return 0;
  return r.f[AXES == 2 ? (lane & 15) : lane];
}

// normalised row (no weight); returns the row's factor
template <int NORM>
__device__ __forceinline__ float norm_row(Lane8& x, float eps) {
  if constexpr (NORM == NORM_NONE) return 1.f;
  if constexpr (NORM == NORM_LAYER) {
    const float2 nm = both(sum8(x.v[0], x.v[1], x.v[2], x.v[3]) * (-1.f / D));
#pragma unroll
    for (int k = 0; k < 4; ++k) x.v[k] = add2(x.v[k], nm);
  }
  float2 q = mul2(x.v[0], x.v[0]);
#pragma unroll
  for (int k = 1; k < 4; ++k) q = fma2(x.v[k], x.v[k], q);
  const float r = rsqrtf(fmaf(row_sum(q.x + q.y), 1.f / D, eps));
  const float2 rr = both(r);
#pragma unroll
  for (int k = 0; k < 4; ++k) x.v[k] = mul2(x.v[k], rr);
  return r;
}

// weight and bias of a lane's eight channels
template <typename T, int NORM>
struct Affine {
  Lane8 w, b;
  __device__ __forceinline__ void load(const void* wp, const void* bp, int first, int apart) {
    Raw8<T> r;
    r.a.load(static_cast<const T*>(wp) + first);
    r.b.load(static_cast<const T*>(wp) + first + apart);
    r.get(w);
    if constexpr (NORM == NORM_LAYER) {
      r.a.zero();
      r.b.zero();
      if (bp) {
        r.a.load(static_cast<const T*>(bp) + first);
        r.b.load(static_cast<const T*>(bp) + first + apart);
      }
      r.get(b);
    }
  }
  __device__ __forceinline__ void apply(Lane8& x) const {
#pragma unroll
    for (int k = 0; k < 4; ++k) x.v[k] = NORM == NORM_LAYER ? fma2(x.v[k], w.v[k], b.v[k]) : mul2(x.v[k], w.v[k]);
  }
};
template <typename T>
struct Affine<T, NORM_NONE> {
  __device__ __forceinline__ void load(const void*, const void*, int, int) {}
  __device__ __forceinline__ void apply(Lane8&) const {}
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

// element of new token t of sequence b in a pool (head 0), -1 if it has no page; and its place in its
// sequence.  `tell`: the thread that records what is wrong.
__device__ __forceinline__ long long place_row(const NormRopeArgs& a, int b, long long t, bool tell, int& place) {
  const PagedCache& c = a.c;
  const int first = a.cu[b], start = a.start[b];
  const long long at = static_cast<long long>(start) + (t - first);
  int page = -1;
  if (first <= t && a.cu[b + 1] > t && start >= 0 && (at >> c.page_shift) < c.max_pages)
    page = c.table[b * c.table_stride + (at >> c.page_shift)];
  if (page < 0 || page >= c.num_pages) {
    if (tell) set_error(a.err, ERR_BOUNDS);
    return -1;
  }
  place = static_cast<int>(at);
  return ((static_cast<long long>(page) * c.heads << c.page_shift) + (at & ((1 << c.page_shift) - 1))) * D;
}
// a token of the whole warp
__device__ __forceinline__ long long paged_row(const NormRopeArgs& a, long long t, int lane, int& place) {
  if (a.cu[0] > t) return -1;
  const int b = find_sequence(a.cu, a.c.batch, t, lane);
  return b >= a.c.batch ? -1 : place_row(a, b, t, lane == 0, place);      // -1: behind the last sequence
}
// a token of this lane's group
__device__ __forceinline__ long long paged_row_of(const NormRopeArgs& a, long long t, bool tell, int& place) {
  if (a.cu[0] > t || a.cu[a.c.batch] <= t) return -1;
  int lo = 0, hi = a.c.batch;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (a.cu[mid] <= t) lo = mid; else hi = mid;
  }
  return place_row(a, lo, t, tell, place);
}

// What the rows do not show of cu: sequences that start before them, end behind them or have a negative
// length.  The last block looks, after its own items.
__device__ __forceinline__ void check_sequences(const NormRopeArgs& a) {
  if (blockIdx.x != gridDim.x - 1) return;
  for (int b = threadIdx.x; b < a.c.batch; b += NTHR) {
    const int first = a.cu[b], end = a.cu[b + 1];
    if (first < 0 || end < first || end > a.n_tokens) set_error(a.err, ERR_BOUNDS);
  }
}

// An item is up to U quads of one token: `left` heads from `head` on.
struct Item {
  long long o, t;
  int head;
  __device__ __forceinline__ void at(long long it, int batches, int heads_per, long long n_tokens) {
    long long g = it;
    int hb = 0;
    if (batches > 1) {
      long long b;
      split_token(it, batches, g, b);
      hb = static_cast<int>(b);
    }
    head = hb * heads_per;
    split_token(g, n_tokens, o, t);
  }
};

// Items of q, then of k, then of v (carried along), over all warps of the grid.  PAGED: rows go to
// the cache instead of `out` (tokens packed, outer 1).
template <typename T, int NORM, int AXES, bool PAGED>
__global__ void __launch_bounds__(NTHR, 3) norm_rope_kernel(const __grid_constant__ NormRopeArgs a) {
  constexpr int U = sizeof(T) == 2 ? 4 : 2;
  const int lane = threadIdx.x & 31, r = lane >> 3;
  const int c0 = Chan<AXES>::first(lane & 7);
  constexpr int APART = Chan<AXES>::APART;
  const long long tokens = a.n_outer * a.n_tokens;
  const long long step = static_cast<long long>(gridDim.x) * WARPS;
  long long item = static_cast<long long>(blockIdx.x) * WARPS + (threadIdx.x >> 5);
  const unsigned long long f = lane_freq<AXES>(a.rope, lane);
  long long end = 0;                                       // first item behind the tensor
#pragma unroll 1
  for (int role = PAGED ? 1 : 0; role < 3; ++role) {
    const Rows in = a.in[role], out = a.out[role];
    if (in.heads == 0) continue;
    const int batches = (in.heads + 4 * U - 1) / (4 * U);
    const long long begin = end;
    end += tokens * batches;
    if (item >= end) continue;                             // this warp has none of it
    Affine<T, NORM> af;
    if (role < 2) af.load(a.w[role], a.b[role], c0, APART);
    const T* src = static_cast<const T*>(in.p) + r * in.sh + c0;
    T* dst = static_cast<T*>(out.p) + r * out.sh + c0;
#pragma unroll 1
    for (; item < end; item += step) {
      Item it;
      it.at(item - begin, batches, 4 * U, a.n_tokens);
      const T* pi = src + it.o * in.so + it.t * in.st + it.head * in.sh;
      Raw8<T> raw[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (it.head + 4 * u + r < in.heads) {
          raw[u].a.load(pi + 4 * u * in.sh);
          raw[u].b.load(pi + 4 * u * in.sh + APART);
        }
      }
      int p0 = 0, p1 = 0;
      long long at;
      if constexpr (PAGED) {
        at = paged_row(a, it.t, lane, p0);                 // the token's place in a pool
        if (at < 0) continue;
      } else {
        at = it.o * out.so + it.t * out.st;
      }
      T* po = dst + at + it.head * out.sh;
      Turn<AXES> turn;
      if (AXES > 0 && role < 2) {
        if (a.pos) {
          const int* q = a.pos + it.o * a.pos_so + it.t * AXES;
          p0 = q[0];
          if constexpr (AXES == 2) p1 = q[1];
        }
        turn.set(f, p0, p1, lane);
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (it.head + 4 * u >= in.heads) break;            // the whole warp
        if (role < 2) {
          Lane8 x;
          raw[u].get(x);
          norm_row<NORM>(x, a.eps);
          af.apply(x);
          turn.template apply<1>(x);
          raw[u].put(x);
        }
        if (it.head + 4 * u + r < in.heads) {
          raw[u].a.store(po + 4 * u * out.sh);
          raw[u].b.store(po + 4 * u * out.sh + APART);
        }
      }
    }
  }
  if constexpr (PAGED) check_sequences(a);
}

// Large calls: each group of eight lanes takes a token of its own and goes through its heads four at a
// time, with its own angles (four a lane).  No lane is left without a row whatever the heads are, and
// the angles cost a token, not a head; but a warp holds four tokens and has to go through all their
// heads, which makes small calls longer.  launch_fwd has the rule between the two and its figures.
// Three blocks an SM: two, with the next rows on their way while a warp works on these, took 378 us
// for the 128 frames where this takes 364, items of at most eight heads 387.
template <typename T, int NORM, int AXES, bool PAGED>
__global__ void __launch_bounds__(NTHR, 3) norm_rope_group_kernel(const __grid_constant__ NormRopeArgs a) {
  const int lane = threadIdx.x & 31, r = lane >> 3;
  const int c0 = Chan<AXES>::first(lane & 7);
  constexpr int APART = Chan<AXES>::APART;
  const long long tokens = a.n_outer * a.n_tokens, items = (tokens + 3) >> 2;
  const long long step = static_cast<long long>(gridDim.x) * WARPS;
  long long item = static_cast<long long>(blockIdx.x) * WARPS + (threadIdx.x >> 5);
  unsigned long long f[4];
  own_freq<AXES>(a.rope, lane, f);
  long long end = 0;                                       // first item behind the tensor
#pragma unroll 1
  for (int role = PAGED ? 1 : 0; role < 3; ++role) {
    const Rows in = a.in[role], out = a.out[role];
    if (in.heads == 0) continue;
    const long long begin = end;
    end += items;
    if (item >= end) continue;                             // this warp has none of it
    Affine<T, NORM> af;
    if (role < 2) af.load(a.w[role], a.b[role], c0, APART);
    const T* src = static_cast<const T*>(in.p) + c0;
    T* dst = static_cast<T*>(out.p) + c0;
#pragma unroll 1
    for (; item < end; item += step) {
      const long long g = 4 * (item - begin) + r;
      const bool real = g < tokens;
      long long o, t;
      split_token(real ? g : 0, a.n_tokens, o, t);
      const T* pi = src + o * in.so + t * in.st;
      Raw8<T> raw[4];
      const auto fetch = [&](int h0) {
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          raw[u].a.zero();
          raw[u].b.zero();
          if (h0 + u < in.heads && real) {
            raw[u].a.load(pi + (h0 + u) * in.sh);
            raw[u].b.load(pi + (h0 + u) * in.sh + APART);
          }
        }
      };
      fetch(0);
      int p0 = 0, p1 = 0;
      long long at = 0;
      if constexpr (PAGED) at = real ? paged_row_of(a, t, (lane & 7) == 0, p0) : -1;
      else at = o * out.so + t * out.st;
      Turn<AXES> turn;
      if (AXES > 0 && role < 2) {
        if (a.pos) {
          const int* q = a.pos + o * a.pos_so + t * AXES;
          p0 = q[0];
          if constexpr (AXES == 2) p1 = q[1];
        }
        turn.set_own(f, p0, p1, lane);
      }
#pragma unroll 1
      for (int h0 = 0;;) {
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          if (h0 + u >= in.heads) break;                   // the whole warp
          if (role < 2) {
            Lane8 x;
            raw[u].get(x);
            norm_row<NORM>(x, a.eps);
            af.apply(x);
            turn.template apply<1>(x);
            raw[u].put(x);
          }
          if (real && (!PAGED || at >= 0)) {
            T* po = dst + at + (h0 + u) * out.sh;
            raw[u].a.store(po);
            raw[u].b.store(po + APART);
          }
        }
        if ((h0 += 4) >= in.heads) break;
        fetch(h0);
      }
    }
  }
  if constexpr (PAGED) check_sequences(a);
}

// Gradients: with g the output gradient turned back and h the normalised row,
// db += g, dw += g h, u = g w, dx = r (u - mean(u) - h mean(u h)) (RMS: without
// mean(u)).  Blocks are dealt to the tensors by their bytes; a block's weight sums
// go to its own row of `part`, and a second kernel adds those in a fixed order.
// GROUPS: a token per group of lanes and two of its heads at a time, else two quads of a token; the
// next two rows of a lane are on their way while it works on these.
template <typename T, typename G, int NORM, int AXES, bool GROUPS>
__global__ void __launch_bounds__(NTHR, 2) norm_rope_bwd_kernel(const __grid_constant__ NormRopeBwdArgs a) {
  constexpr int U = 2;
  constexpr bool NORMED = NORM != NORM_NONE;
  const int lane = threadIdx.x & 31, r = lane >> 3;
  const int c0 = Chan<AXES>::first(lane & 7);
  constexpr int APART = Chan<AXES>::APART;
  asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
  int blk = blockIdx.x, role = 0;
  while (blk >= a.blocks[role]) blk -= a.blocks[role++];
  const Rows gin = a.dout[role], gout = a.din[role];
  const Rows xin = a.in[role < 2 ? role : 0];
  constexpr int NEXT = GROUPS ? 1 : 4, OFF = GROUPS ? 0 : 1;      // heads from one row of a lane to its next; of lanes
  const int batches = (gin.heads + NEXT * U - 1) / (NEXT * U);
  const long long tokens = a.n_outer * a.n_tokens, step = static_cast<long long>(a.blocks[role]) * WARPS;
  const long long items = GROUPS ? (tokens + 3) >> 2 : tokens * batches;
  unsigned long long f[GROUPS ? 4 : 1];
  if constexpr (GROUPS) own_freq<AXES>(a.rope, lane, f);
  else f[0] = lane_freq<AXES>(a.rope, lane);
  Affine<T, NORMED ? NORM_RMS : NORM_NONE> af;
  if (role < 2) af.load(a.w[role], nullptr, c0, APART);
  Lane8 dw, db;
#pragma unroll
  for (int k = 0; k < 4; ++k) dw.v[k] = db.v[k] = both(0.f);
  const G* pg = static_cast<const G*>(gin.p) + OFF * r * gin.sh + c0;
  const T* px = static_cast<const T*>(xin.p) + OFF * r * xin.sh + c0;
  G* po = static_cast<G*>(gout.p) + OFF * r * gout.sh + c0;
  const bool with_x = NORMED && role < 2;

  Raw8<G> rg[U];
  Raw8<T> rx[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    rx[u].a.zero();
    rx[u].b.zero();
  }
  int p0 = 0, p1 = 0;
  Item it;
  bool mine = true;                                        // this lane's token is one
  long long item = static_cast<long long>(blk) * WARPS + (threadIdx.x >> 5);
  int batch = 0;                                           // GROUPS: of the item
  auto load = [&]() {
    if constexpr (GROUPS) {
      it.head = batch * U;
      if (batch == 0) {
        const long long g = 4 * item + r;
        mine = g < tokens;
        split_token(mine ? g : 0, a.n_tokens, it.o, it.t);
      }
    } else {
      it.at(item, batches, 4 * U, a.n_tokens);
    }
    const G* g = pg + it.o * gin.so + it.t * gin.st + it.head * gin.sh;
    const T* p = px + it.o * xin.so + it.t * xin.st + it.head * xin.sh;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      rg[u].a.zero();
      rg[u].b.zero();
      if (mine && it.head + NEXT * u + OFF * r < gin.heads) {
        rg[u].a.load(g + NEXT * u * gin.sh);
        rg[u].b.load(g + NEXT * u * gin.sh + APART);
        if (with_x) {
          rx[u].a.load(p + NEXT * u * xin.sh);
          rx[u].b.load(p + NEXT * u * xin.sh + APART);
        }
      }
    }
    if (AXES > 0 && role < 2 && batch == 0) {
      const int* q = a.pos + it.o * a.pos_so + it.t * AXES;
      p0 = q[0];
      if constexpr (AXES == 2) p1 = q[1];
    }
  };
  Turn<AXES> turn;
  bool more = item < items;
  if (more) load();
#pragma unroll 1
  while (more) {
    Raw8<G> ng[U];
    Raw8<T> nx[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      ng[u] = rg[u];
      nx[u] = rx[u];
    }
    const Item cur = it;
    const bool have = mine;
    if (role < 2 && batch == 0) {
      if constexpr (GROUPS) turn.set_own(f, p0, p1, lane);
      else turn.set(f[0], p0, p1, lane);
    }
    if (!GROUPS || ++batch == batches) {
      batch = 0;
      item += step;
    }
    more = item < items;
    if (more) load();
    G* p = po + cur.o * gout.so + cur.t * gout.st + cur.head * gout.sh;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (cur.head + NEXT * u >= gin.heads) break;         // the whole warp
      const bool real = have && cur.head + NEXT * u + OFF * r < gin.heads;
      if (role < 2) {
        Lane8 d;
        ng[u].get(d);                                      // zeros where there is no head
        turn.template apply<-1>(d);
        if constexpr (NORMED) {
          Lane8 x;
          nx[u].get(x);
          const float rs = norm_row<NORM>(x, a.eps);
          float2 sh = both(0.f);
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            if (real) {
              db.v[k] = add2(db.v[k], d.v[k]);
              dw.v[k] = fma2(d.v[k], x.v[k], dw.v[k]);
            }
            d.v[k] = mul2(d.v[k], af.w.v[k]);
            sh = fma2(d.v[k], x.v[k], sh);
          }
          const float2 nmh = both(row_sum(sh.x + sh.y) * (-1.f / D));
          const float mu = NORM == NORM_LAYER ? sum8(d.v[0], d.v[1], d.v[2], d.v[3]) * (-1.f / D) : 0.f;
          const float2 rr = both(rs), nmu = both(mu);
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            float2 v = fma2(x.v[k], nmh, d.v[k]);
            if constexpr (NORM == NORM_LAYER) v = add2(v, nmu);
            d.v[k] = mul2(v, rr);
          }
        }
        ng[u].put(d);
      }
      if (real) {
        ng[u].a.store(p + NEXT * u * gout.sh);
        ng[u].b.store(p + NEXT * u * gout.sh + APART);
      }
    }
  }
  if constexpr (NORMED) {
    if (role == 2 || !a.part) return;
    __shared__ float sums[WARPS][128];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int ch = c0 + (k & 1) * 2 + (k >> 1) * APART;
      float2 w = dw.v[k], b = db.v[k];
#pragma unroll
      for (int x = 8; x < 32; x <<= 1) {
        w.x += __shfl_xor_sync(0xffffffffu, w.x, x);
        w.y += __shfl_xor_sync(0xffffffffu, w.y, x);
        b.x += __shfl_xor_sync(0xffffffffu, b.x, x);
        b.y += __shfl_xor_sync(0xffffffffu, b.y, x);
      }
      if (r == 0) {
        sums[threadIdx.x >> 5][ch] = w.x;
        sums[threadIdx.x >> 5][ch + 1] = w.y;
        sums[threadIdx.x >> 5][64 + ch] = b.x;
        sums[threadIdx.x >> 5][64 + ch + 1] = b.y;
      }
    }
    __syncthreads();
    if (threadIdx.x < 128) {
      float v = 0.f;
#pragma unroll
      for (int w = 0; w < WARPS; ++w) v += sums[w][threadIdx.x];
      a.part[(static_cast<long long>(role) * NORM_BWD_BLOCKS + blk) * 128 + threadIdx.x] = v;
    }
  }
}

// one block per tensor: column c of the blocks' rows [blocks][128], eight interleaved chains of
// eight loads at a time; launched while the blocks still run (programmatic dependent launch)
__global__ void __launch_bounds__(1024) norm_rope_sum_kernel(const __grid_constant__ NormRopeBwdArgs a) {
  __shared__ float sums[8][128];
  const int col = threadIdx.x & 127, grp = threadIdx.x >> 7, role = blockIdx.x, n = a.blocks[role];
  const float* p = a.part + static_cast<long long>(role) * NORM_BWD_BLOCKS * 128 + col;
  asm volatile("griddepcontrol.wait;\n" ::: "memory");
  float v = 0.f;
  for (int i = grp; i < n; i += 64) {
    float x[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) x[k] = i + 8 * k < n ? p[(i + 8 * k) * 128] : 0.f;
#pragma unroll
    for (int k = 0; k < 8; ++k) v += x[k];
  }
  sums[grp][col] = v;
  __syncthreads();
  if (grp == 0) {
#pragma unroll
    for (int i = 1; i < 8; ++i) v += sums[i][col];
    float* out = col < 64 ? a.dw[role] : a.db[role];
    if (out) out[col & 63] = v;
  }
}

int blocks_for(long long items, int most) {
  const long long b = (items + WARPS - 1) / WARPS;
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
    default: break;                                                         \
  }                                                                         \
  return cudaErrorInvalidValue;

// Which of the two kernels: small calls last as long as their longest warp, which in groups goes
// through all heads one after the other and in quads has items / warps of them; measured even at
// about an eighth of the heads (16 heads: 1369 tokens, three tensors, 6.3 us in quads, 8.0 in groups;
// 3001 tokens, two tensors, 8.8 and 9.0; 8 heads 7.8 and 6.5, 2 heads 7.0 and 4.8, but 48 tokens of
// them 3.4 and 3.7).  Above that groups in 16 bits:
// 60,000 tokens of queries and keys, us in quads and in groups, 4 heads 54 and 26, 7 heads 67 and 43,
// 16 heads 92 and 90, 24 heads 170 and 130; three tensors of 16 heads with two axes, 165,888 tokens,
// 396 and 363.  In 32 bits a quad's lanes hold twice the bytes and the memory is the bound once they
// are full, so groups only where a quarter of the lanes or more would have no row: 4 heads 52 and 44,
// 10 heads 131 and 107, but 8 heads 75 and 83, 16 heads 153 and 166, 32 heads 300 and 332.
template <typename T, int NORM, int AXES, bool PAGED>
cudaError_t launch_fwd(const NormRopeArgs& a, cudaStream_t st) {
  constexpr int PER = 4 * (sizeof(T) == 2 ? 4 : 2);        // heads of an item of quads
  const long long tokens = a.n_outer * a.n_tokens;
  long long items = 0, tensors = 0, heads = 0, most = 0;
  for (int i = PAGED ? 1 : 0; i < 3; ++i) {
    heads += tokens * a.in[i].heads;
    items += tokens * ((a.in[i].heads + PER - 1) / PER);
    tensors += a.in[i].heads > 0;
    if (a.in[i].heads > most) most = a.in[i].heads;
  }
  if (8 * items > FWD_BLOCKS * WARPS * most && (sizeof(T) == 2 || 4 * heads <= 3 * PER * items))
    norm_rope_group_kernel<T, NORM, AXES, PAGED>
        <<<blocks_for(tensors * ((tokens + 3) / 4), FWD_BLOCKS), NTHR, 0, st>>>(a);
  else
    norm_rope_kernel<T, NORM, AXES, PAGED><<<blocks_for(items, FWD_BLOCKS), NTHR, 0, st>>>(a);
  return cudaGetLastError();
}

cudaError_t launch_norm_rope(const NormRopeArgs& a, bool fp32, int norm, int axes, cudaStream_t st) {
#define GSA_CALL(N, A) return fp32 ? launch_fwd<float, N, A, false>(a, st) : launch_fwd<__nv_bfloat16, N, A, false>(a, st)
  GSA_BY_NORM_AXES(GSA_CALL)
#undef GSA_CALL
}

// Quads or groups as in the forward; measured even at a quarter of the heads (us, queries and keys: 16
// heads, 3001 tokens 16.1 and 15.7, 8 heads 10.6 and 10.7, 2 heads 9.3 and 6.8; 700 tokens of 4 heads 6.1
// and 6.1, of 10 heads 8.6 and 9.1).  60,000 tokens in 16 bits: 2 heads 69 and 30, 8 heads 93 and 81, 16
// heads 188 and 151, 24 heads 277 and 220; three tensors of 16 heads with gradients in 32 bits and two
// axes, 217 and 197.  In 32 bits: 2 heads 77 and 35, 12 heads 203 and 184, but 16 heads 229 and 247.
template <typename T, typename G, int NORM, int AXES>
cudaError_t launch_bwd(NormRopeBwdArgs a, cudaStream_t st) {
  const long long tokens = a.n_outer * a.n_tokens;
  double bytes[3], all = 0.0;
  long long quads = 0, heads = 0, most = 0;
  for (int i = 0; i < 3; ++i) {
    bytes[i] = a.dout[i].heads * (2.0 * sizeof(G) + (i < 2 && NORM != NORM_NONE ? sizeof(T) : 0));
    all += bytes[i];
    quads += tokens * ((a.dout[i].heads + 7) / 8);
    heads += tokens * a.dout[i].heads;
    if (a.dout[i].heads > most) most = a.dout[i].heads;
  }
  const bool groups = 4 * quads > NORM_BWD_BLOCKS * WARPS * most && (sizeof(T) == 2 || 4 * heads <= 3 * 8 * quads);
  // blocks by each tensor's bytes, at most what has items
  int total = 0;
  for (int i = 0; i < 3; ++i) {
    a.blocks[i] = 0;
    if (tokens == 0 || a.dout[i].heads == 0) continue;
    const long long items = groups ? (tokens + 3) / 4 : tokens * ((a.dout[i].heads + 7) / 8);
    const int share = static_cast<int>(NORM_BWD_BLOCKS * bytes[i] / all);
    a.blocks[i] = blocks_for(items, share < 1 ? 1 : share);
    total += a.blocks[i];
  }
  if (total > 0) {
    if (groups) norm_rope_bwd_kernel<T, G, NORM, AXES, true><<<total, NTHR, 0, st>>>(a);
    else norm_rope_bwd_kernel<T, G, NORM, AXES, false><<<total, NTHR, 0, st>>>(a);
  }
  // a tensor that is left out has no sums to write (its pointers are null)
  if (a.part && NORM != NORM_NONE) {
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    cudaLaunchAttribute early;
    early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    early.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t c = {};
    c.gridDim = dim3(2);
    c.blockDim = dim3(1024);
    c.stream = st;
    c.attrs = &early;
    c.numAttrs = total > 0 ? 1 : 0;      // behind this call's blocks only
    return cudaLaunchKernelEx(&c, norm_rope_sum_kernel, a);
  }
  return cudaGetLastError();
}

cudaError_t launch_norm_rope_bwd(const NormRopeBwdArgs& a, bool fp32, bool grad_fp32, int norm, int axes,
                                 cudaStream_t st) {
#define GSA_CALL(N, A)                                                              \
  return fp32 ? launch_bwd<float, float, N, A>(a, st)                               \
              : grad_fp32 ? launch_bwd<__nv_bfloat16, float, N, A>(a, st)           \
                          : launch_bwd<__nv_bfloat16, __nv_bfloat16, N, A>(a, st)
  GSA_BY_NORM_AXES(GSA_CALL)
#undef GSA_CALL
}

cudaError_t launch_append(const NormRopeArgs& a, bool fp32, int norm, int axes, cudaStream_t st) {
#define GSA_CALL(N, A) return fp32 ? launch_fwd<float, N, A, true>(a, st) : launch_fwd<__nv_bfloat16, N, A, true>(a, st)
  GSA_BY_NORM_AXES(GSA_CALL)
#undef GSA_CALL
}

}  // namespace gsa
