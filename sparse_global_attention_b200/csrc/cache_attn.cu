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
// Warp roles: softmax warps (thread = row = TMEM lane), one TMA producer, one MMA
// issuer.  Variants by the rows of a sequence and key head:
//   two tiles of 128 rows per block (a chunk of tokens): every key tile that
//     arrives serves 256 rows, and one tile's exponentials run while the other's
//     products do;
//   one tile of 128 rows, two blocks per SM (a few tokens);
//   at most 32 rows (single tokens): the rows are repeated in the four 32-lane
//     quarters of TMEM and each of the four softmax warps takes 32 of a tile's 128
//     keys for all rows (its P is zero elsewhere), so no warp does four times the
//     exponentials; the quarters' sums are joined at the end.
// Rows of V that no key stands for (the cache's memory behind a sequence's last
// token, pages that do not exist) are zeroed in shared memory before the product,
// since 0 * NaN is NaN; scores of such keys are replaced, not added to.
//
// fp32 is a register-tiled kernel (64 or 16 rows by 64 keys) with the same split.
//
// All mbarrier waits are bounded; one that runs out records GSA_ERR_DEVICE_TIMEOUT.
#include <atomic>
#include <cuda.h>
#include <string.h>

#include "operators.h"
#include "tc_ptx.cuh"
#include "tc_softmax.cuh"

namespace gsa {

namespace {

using namespace tc;

constexpr int TM = 128;                  // rows per tensor-core tile
constexpr int TN = 128;                  // keys per tile
constexpr int TILE = TN * 128;           // bytes of one 128 x 64 bf16 tile
constexpr float RESCALE_LOG2 = 8.f;      // rescale O when the max grows by > 2^8
constexpr uint32_t IDESC_QK = idesc_bf16(128, 128, false);
constexpr uint32_t IDESC_PV = idesc_bf16(128, 64, true);
constexpr float LN2 = 0.6931471805599453f;

// kernel variants
enum Kind : int { TWO_TILES = 0, ONE_TILE = 1, QUARTERS = 2, F32_64 = 3, F32_16 = 4 };

template <int KIND>
struct Lay {
  static constexpr int NQ = KIND == TWO_TILES ? 2 : 1;
  static constexpr int NST = KIND == TWO_TILES ? 5 : 3;      // K/V ring depth
  static constexpr int ROWS = KIND == QUARTERS ? 32 : NQ * TM;
  static constexpr int NWARP = 4 * NQ;                       // softmax warps
  static constexpr int NTHREADS = 32 * (NWARP + 2);
  static constexpr int COLS = KIND == TWO_TILES ? 512 : 256; // TMEM columns
  static constexpr int TO = 128 * NQ, TP = TO + 64 * NQ;     // S_i at 128 i, O_i and P_i after
  static constexpr int KV = NQ * TILE;
  static constexpr int STAGE = 2 * TILE;
  static constexpr int BAR = KV + NST * STAGE;
  // q_full, full[NST], empty[NST], s_full[NQ], s_free[NQ], p_full[NQ], pv_done[NQ], fin
  static constexpr int NBAR = 2 + 2 * NST + 4 * NQ;
  static constexpr int INFO = BAR + NBAR * 8;                // valid boxes of each stage, "some are not"
  static constexpr int SLOT = INFO + 4 * (NST + 1);
  static constexpr int BYTES = SLOT + 16;
};
static_assert(2 * (Lay<QUARTERS>::BYTES + 1024) <= 228 * 1024, "two blocks per SM");
static_assert(4 * 32 * 66 * 4 <= Lay<QUARTERS>::NST * Lay<QUARTERS>::STAGE, "the quarters' sums fit the ring");

template <int KIND>
struct Bars {
  using L = Lay<KIND>;
  uint32_t base;
  __device__ uint32_t q_full() const { return base; }
  __device__ uint32_t full(int s) const { return base + 8 * (1 + s); }
  __device__ uint32_t empty(int s) const { return base + 8 * (1 + L::NST + s); }
  __device__ uint32_t s_full(int i) const { return base + 8 * (1 + 2 * L::NST + i); }
  __device__ uint32_t s_free(int i) const { return base + 8 * (1 + 2 * L::NST + L::NQ + i); }
  __device__ uint32_t p_full(int i) const { return base + 8 * (1 + 2 * L::NST + 2 * L::NQ + i); }
  __device__ uint32_t pv_done(int i) const { return base + 8 * (1 + 2 * L::NST + 3 * L::NQ + i); }
  __device__ uint32_t fin() const { return base + 8 * (1 + 2 * L::NST + 4 * L::NQ); }
};

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
  unsigned x = blockIdx.x;
  k.split = x % a.n_split;
  x /= a.n_split;
  const int tile = a.row_tiles - 1 - static_cast<int>(x % a.row_tiles);   // causal: the longest first
  x /= a.row_tiles;
  k.h = x % a.c.heads;
  k.b = x / a.c.heads;
  k.seq = sequence_of(a, k.b);
  const long long room = static_cast<long long>(a.c.max_pages) << a.c.page_shift;
  k.len = static_cast<int>(min(static_cast<long long>(k.seq.len), room));
  if (threadIdx.x == 0 && (!k.seq.ok || (k.len != k.seq.len && k.seq.n > 0))) set_error(a.err, ERR_BOUNDS);
  k.rows = k.seq.ok ? k.seq.n * a.group : 0;
  k.row0 = tile * TROWS;
  k.any = k.row0 < k.rows;
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

// page of slot `t` of sequence b, -1 if the pool has none such
__device__ __forceinline__ int page_of(const CacheAttnArgs& a, int raw) {
  return raw >= 0 && raw < a.c.num_pages ? raw : -1;
}

template <int KIND>
__global__ void __launch_bounds__(Lay<KIND>::NTHREADS, KIND == TWO_TILES ? 1 : 2)
    cache_attn_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                      const __grid_constant__ CacheAttnArgs a) {
  using L = Lay<KIND>;
  extern __shared__ __align__(1024) uint8_t smem[];
  const uint32_t sbase = smem_u32(smem);          // 1024-byte aligned: no static shared memory before it
  const Bars<KIND> bars{sbase + L::BAR};
  volatile uint32_t* info = reinterpret_cast<volatile uint32_t*>(smem + L::INFO);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + L::SLOT);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  const Block blk = block_of<L::ROWS, TN>(a);
  if (!blk.any) return;
  if (sbase & 1023u) {                            // the operands' swizzle needs it
    if (threadIdx.x == 0) set_error(a.err, ERR_BOUNDS);
    return;
  }
  const int nq = (L::NQ == 2 && blk.rows - blk.row0 > TM) ? 2 : 1;      // tiles that hold rows
  const int ntile = blk.ntile;
  int* err = a.err + 1;

  if (threadIdx.x == 0) {
    mbar_init(bars.q_full(), 4 * nq);
    for (int s = 0; s < L::NST; ++s) {
      mbar_init(bars.full(s), 1);
      mbar_init(bars.empty(s), 1);
    }
    for (int i = 0; i < L::NQ; ++i) {
      mbar_init(bars.s_full(i), 1);
      mbar_init(bars.s_free(i), 4);              // one arrival per softmax warp
      mbar_init(bars.p_full(i), 4);
      mbar_init(bars.pv_done(i), 1);
    }
    mbar_init(bars.fin(), 1);
    info[L::NST] = 0;
    fence_mbar_init();
  }
  if (warp == 0) tmem_alloc<L::COLS>(smem_u32(tmem_slot));
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  const int page_size = 1 << a.c.page_shift;
  const int box = min(page_size, TN);             // rows of one copy
  const int box_shift = min(a.c.page_shift, 7);
  const int nbox = TN >> box_shift;

  if (warp == L::NWARP) {
    // ------------------------------------------------------------ TMA producer
    // lanes 0-7 copy the tile's boxes of K, lanes 8-15 those of V
    if (ntile > 0) {
      const int* table = a.c.table + blk.b * a.c.table_stride;
      const int my = lane & 7;
      const bool mine = lane < 16 && my < nbox;
      auto slot_of = [&](int it) { return (blk.t_begin + it) * TN + (my << box_shift); };
      auto lookup = [&](int it) {
        const int slot = slot_of(it);
        return mine && it < ntile && slot < blk.len ? table[slot >> a.c.page_shift] : -1;
      };
      int next = lookup(0);
      int issued = 0;
      for (int it = 0; it < ntile; ++it) {
        const int s = it % L::NST;
        const int raw = next;
        next = lookup(it + 1);
        if (it >= L::NST &&
            !__all_sync(0xffffffffu, mbar_wait(bars.empty(s), ((it / L::NST) - 1) & 1, err)))
          break;
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
          const uint32_t dst = sbase + L::KV + s * L::STAGE + (lane >= 8 ? TILE : 0) + (my << box_shift) * 128;
          tma_load_2d(dst, lane >= 8 ? &tm_v : &tm_k, 0, y, bars.full(s));
        }
        __syncwarp();
        ++issued;
      }
      // drain: every issued copy has landed before the block may exit
      for (int it = max(0, issued - L::NST); it < issued; ++it)
        mbar_wait(bars.full(it % L::NST), (it / L::NST) & 1, err);
    }
  } else if (warp == L::NWARP + 1) {
    // ------------------------------------------------------------ MMA issuer
    if (ntile > 0) {
      const bool leader = elect_one();
      const uint64_t dq0 = sdesc_sw128(sbase, 16, 1024);
      const uint64_t dk0 = sdesc_sw128(sbase + L::KV, 16, 1024);
      const uint64_t dv0 = sdesc_sw128(sbase + L::KV + TILE, 8192, 1024);
      constexpr uint32_t T16 = TILE >> 4, ST16 = L::STAGE >> 4;
      bool ok = __all_sync(0xffffffffu, mbar_wait(bars.q_full(), 0, err));
      tc_fence_after();
      for (int j = 0; ok && j <= ntile; ++j) {
        if (j < ntile) {
          const int s = j % L::NST;
          ok = __all_sync(0xffffffffu, mbar_wait(bars.full(s), (j / L::NST) & 1, err));
          if (!ok) break;
          const int kb = (blk.t_begin + j) * TN;
          const uint32_t bits = info[s];
          if (kb + TN > blk.len || bits != (1u << nbox) - 1u) {
            // rows of V without a key
            for (int r = lane; r < TN; r += 32)
              if (kb + r >= blk.len || !((bits >> (r >> box_shift)) & 1u)) {
                uint4* p = reinterpret_cast<uint4*>(smem + L::KV + s * L::STAGE + TILE + r * 128);
#pragma unroll
                for (int c = 0; c < 8; ++c) p[c] = make_uint4(0, 0, 0, 0);
              }
            fence_async_smem();
            __syncwarp();
          }
          tc_fence_after();
        }
        const uint64_t dk = dk0 + (j % L::NST) * ST16;
        const uint64_t dv = dv0 + ((j + L::NST - 1) % L::NST) * ST16;
        for (int i = 0; i < nq && ok; ++i) {
          if (j < ntile) {
            // S_i = Q_i K_j^T as soon as the softmax warps hold S_i of tile j - 1
            if (j > 0) {
              ok = __all_sync(0xffffffffu, mbar_wait(bars.s_free(i), (j - 1) & 1, err));
              if (!ok) break;
              tc_fence_after();
            }
            if (leader) {
#pragma unroll
              for (int ks = 0; ks < 4; ++ks)
                mma_bf16_ss(tmem + 128 * i, dq0 + i * T16 + 2 * ks, dk + 2 * ks, IDESC_QK, ks > 0 ? 1u : 0u);
              mma_commit(bars.s_full(i));
            }
            __syncwarp();
          }
          if (j > 0) {
            // O_i += P_i V_{j-1}
            ok = __all_sync(0xffffffffu, mbar_wait(bars.p_full(i), (j - 1) & 1, err));
            if (!ok) break;
            tc_fence_after();
            if (leader) {
#pragma unroll
              for (int ks = 0; ks < TN / 16; ++ks)
                mma_bf16_ts(tmem + L::TO + 64 * i, tmem + L::TP + 64 * i + 8 * ks, dv + ks * 128, IDESC_PV,
                            (j > 1 || ks > 0) ? 1u : 0u);
              mma_commit(bars.pv_done(i));
            }
            __syncwarp();
          }
        }
        if (ok && j > 0 && leader) mma_commit(bars.empty((j - 1) % L::NST));
        __syncwarp();
      }
      if (leader) mma_commit(bars.fin());
      __syncwarp();
      mbar_wait(bars.fin(), 0, err);
    }
  } else if (warp < 4 * nq) {
    // ------------------------------------------------------------ softmax
    constexpr bool QUAD = KIND == QUARTERS;
    constexpr int NC = QUAD ? 1 : 4;               // 32-key chunks of a tile that a thread takes
    const int qi = warp >> 2;
    const int c0 = QUAD ? 32 * (warp & 3) : 0;     // first of its keys
    const int row = blk.row0 + (QUAD ? lane : qi * TM + (threadIdx.x & 127));
    const bool real = row < blk.rows;
    const int token = real ? row / a.group : 0;
    const int head = blk.h * a.group + (real ? row - token * a.group : 0);
    const int lim = real ? row_limit(a, blk, token) : 0x7fffffff;    // rows without a query need no mask
    const uint32_t lane_off = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t tS = tmem + lane_off + 128 * qi + c0;
    const uint32_t tO = tmem + lane_off + L::TO + 64 * qi;
    const uint32_t tP = tmem + lane_off + L::TP + 64 * qi;
    const float sl2 = a.scale_log2;
    // this row of Q, into the 128-byte swizzle of the operand
    if (ntile > 0) {
      uint4 w[8];
      const uint4* src = reinterpret_cast<const uint4*>(
          static_cast<const __nv_bfloat16*>(a.q.p) + (blk.seq.first + token) * a.q.st + head * a.q.sh);
#pragma unroll
      for (int c = 0; c < 8; ++c) w[c] = real ? __ldg(src + c) : make_uint4(0, 0, 0, 0);
      const int r = threadIdx.x & 127;
#pragma unroll
      for (int c = 0; c < 8; ++c) *reinterpret_cast<uint4*>(smem + qi * TILE + swz(r, c)) = w[c];
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
    for (int j = 0; j < ntile; ++j) {
      ok = __all_sync(0xffffffffu, mbar_wait(bars.s_full(qi), j & 1, err));
      if (!ok) break;
      tc_fence_after();
      const int kb = (blk.t_begin + j) * TN + c0;
      const uint32_t bad = info[L::NST];
      uint32_t v[32 * NC];
      if constexpr (QUAD) {
        tmem_ld32(tS, v);
      } else {
        tmem_ld64(tS, v);
        tmem_ld64(tS + 64, v + 64);
      }
      tmem_wait_ld();
      tc_fence_before();
      warp_arrive(bars.s_free(qi));
      if (bad) {
        // some box of this block had no page: the stage's valid boxes, from its barrier's phase
        ok = __all_sync(0xffffffffu, mbar_wait(bars.full(j % L::NST), (j / L::NST) & 1, err));
        if (!ok) break;
        const uint32_t bits = info[j % L::NST];
#pragma unroll
        for (int c = 0; c < NC; ++c) {
          uint32_t msk = 0;
          for (int e = 0; e < 32; ++e) msk |= ((bits >> ((c0 + 32 * c + e) >> box_shift)) & 1u) << e;
          apply_mask(v + 32 * c, msk);
        }
      }
      if (__any_sync(0xffffffffu, kb + 32 * NC > lim)) {
#pragma unroll
        for (int c = 0; c < NC; ++c) {
          const int left = lim - kb - 32 * c;
          apply_mask(v + 32 * c, left >= 32 ? ~0u : (left <= 0 ? 0u : (1u << left) - 1u));
        }
      }
      float mx = max32(v);
#pragma unroll
      for (int c = 1; c < NC; ++c) mx = fmaxf(mx, max32(v + 32 * c));
      // move the reference max only when a row's max grew by more than 2^8
      const float m_new = fmaxf(m, mx);
      const bool need = (m == -INFINITY) ? (m_new != -INFINITY) : ((m_new - m) * sl2 > RESCALE_LOG2);
      float alpha = 1.f;
      if (need) {
        alpha = (m == -INFINITY) ? 0.f : ex2((m - m_new) * sl2);
        m = m_new;
      }
      l *= alpha;
      // P (and O) are free once the previous tile's product has completed
      if (j > 0) {
        ok = __all_sync(0xffffffffu, mbar_wait(bars.pv_done(qi), (j - 1) & 1, err));
        if (!ok) break;
        tc_fence_after();
        if (__any_sync(0xffffffffu, need && alpha != 0.f)) {
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            uint32_t w[32];
            tmem_ld32(tO + 32 * c, w);
            tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 32; ++e) w[e] = __float_as_uint(__uint_as_float(w[e]) * alpha);
            tmem_st32(tO + 32 * c, w);
          }
        }
      }
      const float mb = (m == -INFINITY) ? 0.f : m * sl2;
      float l0 = 0.f, l1 = 0.f;
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        uint32_t pk[16];
#pragma unroll
        for (int e = 0; e < 32; e += 2) {
          float p0, p1;
          exp2_pair(v[32 * c + e], v[32 * c + e + 1], sl2, -mb, l0, l1, p0, p1);
          pk[e >> 1] = pack_bf16(p0, p1);
        }
        tmem_st16(tP + (c0 >> 1) + 16 * c, pk);
      }
      l += l0 + l1;
      tmem_wait_st();
      tc_fence_before();
      warp_arrive(bars.p_full(qi));
    }
    if (ok && ntile > 0) ok = mbar_wait(bars.pv_done(qi), (ntile - 1) & 1, err);
    ok = __all_sync(0xffffffffu, ok);
    tc_fence_after();
    float o[64];
    if (ok && ntile > 0) {
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        uint32_t v[32];
        tmem_ld32(tO + 32 * c, v);
        tmem_wait_ld();
#pragma unroll
        for (int e = 0; e < 32; ++e) o[32 * c + e] = __uint_as_float(v[e]);
      }
    } else {
#pragma unroll
      for (int e = 0; e < 64; ++e) o[e] = 0.f;
    }
    const int at = blk.seq.first + token;
    const long long prow = (static_cast<long long>(blk.split) * a.n_tokens + at) * a.q.heads + head;
    __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(a.out.p) + at * a.out.st + head * a.out.sh;
    if constexpr (QUAD) {
      // join the four quarters: the ring is idle, every copy has been consumed
      constexpr int PITCH = 66;
      float* part = reinterpret_cast<float*>(smem + L::KV);
      float* mineq = part + threadIdx.x * PITCH;
      if (real) {
#pragma unroll
        for (int e = 0; e < 64; ++e) mineq[e] = o[e];
        mineq[64] = m;
        mineq[65] = l;
      }
      named_bar(1, 128);
      // four threads per row, sixteen channels each
      const int r = threadIdx.x >> 2, e0 = (threadIdx.x & 3) * 16;
      const int row_r = blk.row0 + r;
      if (row_r < blk.rows) {
        float mx = -INFINITY;
#pragma unroll
        for (int w = 0; w < 4; ++w) mx = fmaxf(mx, part[(32 * w + r) * PITCH + 64]);
        const float mu = (mx == -INFINITY) ? 0.f : mx;
        float ls = 0.f, os[16];
#pragma unroll
        for (int e = 0; e < 16; ++e) os[e] = 0.f;
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          const float* p = part + (32 * w + r) * PITCH;
          const float f = ex2((p[64] - mu) * sl2);
          ls = fmaf(f, p[65], ls);
#pragma unroll
          for (int e = 0; e < 16; ++e) os[e] = fmaf(f, p[e0 + e], os[e]);
        }
        const int tk = row_r / a.group;
        const int hd = blk.h * a.group + row_r - tk * a.group;
        const int tat = blk.seq.first + tk;
        if (a.n_split == 1) {
          const float inv = ls > 0.f ? 1.f / ls : (ls == ls ? 0.f : ls);
          __nv_bfloat16* d = static_cast<__nv_bfloat16*>(a.out.p) + tat * a.out.st + hd * a.out.sh + e0;
#pragma unroll
          for (int e = 0; e < 16; e += 8)
            *reinterpret_cast<uint4*>(d + e) =
                make_uint4(pack_bf16(os[e] * inv, os[e + 1] * inv), pack_bf16(os[e + 2] * inv, os[e + 3] * inv),
                           pack_bf16(os[e + 4] * inv, os[e + 5] * inv), pack_bf16(os[e + 6] * inv, os[e + 7] * inv));
          if (a.lse && e0 == 0)
            a.lse[static_cast<long long>(hd) * a.n_tokens + tat] =
                ls == 0.f ? -INFINITY : (mu * sl2 + log2f(ls)) * LN2;
        } else {
          const long long pr = (static_cast<long long>(blk.split) * a.n_tokens + tat) * a.q.heads + hd;
          if (ntile > 0) {
#pragma unroll
            for (int e = 0; e < 16; e += 4)
              *reinterpret_cast<float4*>(a.part_o + pr * D + e0 + e) =
                  make_float4(os[e], os[e + 1], os[e + 2], os[e + 3]);
          }
          if (e0 == 0) *reinterpret_cast<float2*>(a.part_ml + pr * 2) = make_float2(mx, ls);
        }
      }
    } else if (real) {
      if (a.n_split == 1) {
        const float inv = l > 0.f ? 1.f / l : (l == l ? 0.f : l);     // a NaN stays one
#pragma unroll
        for (int e = 0; e < 64; e += 8)
          *reinterpret_cast<uint4*>(dst + e) =
              make_uint4(pack_bf16(o[e] * inv, o[e + 1] * inv), pack_bf16(o[e + 2] * inv, o[e + 3] * inv),
                         pack_bf16(o[e + 4] * inv, o[e + 5] * inv), pack_bf16(o[e + 6] * inv, o[e + 7] * inv));
        if (a.lse)
          a.lse[static_cast<long long>(head) * a.n_tokens + at] = l == 0.f ? -INFINITY : (m * sl2 + log2f(l)) * LN2;
      } else {
        if (ntile > 0) {
#pragma unroll
          for (int e = 0; e < 64; e += 4)
            *reinterpret_cast<float4*>(a.part_o + prow * D + e) = make_float4(o[e], o[e + 1], o[e + 2], o[e + 3]);
        }
        *reinterpret_cast<float2*>(a.part_ml + prow * 2) = make_float2(m, l);
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 0) tmem_dealloc<L::COLS>(tmem);
}

// ---- fp32 ---------------------------------------------------------------------
// TR rows by 64 keys per step, 256 threads as 16 x 16: thread (ty, tx) holds
// TR / 16 rows by 4 keys (tx + 16 i) of S and the same rows by channels 4 tx .. of O.
constexpr int FK = 64;                    // keys per tile
constexpr int FP = 68;                    // row pitch in floats: 16-byte reads of 16 rows meet no bank twice
template <int TR>
struct FLay {
  static constexpr int Q = 0;
  static constexpr int K = Q + TR * FP * 4;               // two buffers of K, two of V
  static constexpr int V = K + 2 * FK * FP * 4;
  static constexpr int P = V + 2 * FK * FP * 4;
  static constexpr int OK = P + TR * FP * 4;              // keys that exist, two buffers
  static constexpr int BYTES = OK + 2 * FK * 4;
};

template <int TR>
__global__ void __launch_bounds__(256, 2) cache_attn_f32_kernel(const __grid_constant__ CacheAttnArgs a) {
  using L = FLay<TR>;
  constexpr int R = TR / 16;
  extern __shared__ __align__(1024) uint8_t smem[];
  float* sq = reinterpret_cast<float*>(smem + L::Q);
  float* sp = reinterpret_cast<float*>(smem + L::P);
  float* sk = reinterpret_cast<float*>(smem + L::K);
  float* sv = reinterpret_cast<float*>(smem + L::V);
  int* skey = reinterpret_cast<int*>(smem + L::OK);
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
#pragma unroll
    for (int i = 0; i < R; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) s[i][e] = 0.f;
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
          s[i][e] = fmaf(q.x, kv[e].x, s[i][e]);
          s[i][e] = fmaf(q.y, kv[e].y, s[i][e]);
          s[i][e] = fmaf(q.z, kv[e].z, s[i][e]);
          s[i][e] = fmaf(q.w, kv[e].w, s[i][e]);
        }
      }
    }
    const int kb = (blk.t_begin + j) * FK;
#pragma unroll
    for (int i = 0; i < R; ++i) {
      float mx = -INFINITY;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int key = tx + 16 * e;
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
#pragma unroll
      for (int e = 0; e < 4; ++e) o[i][e] *= alpha;
    }
    __syncwarp();                      // a row's P is written and read by one half-warp
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
          o[i][0] = fmaf(pe[e], vv[e].x, o[i][0]);
          o[i][1] = fmaf(pe[e], vv[e].y, o[i][1]);
          o[i][2] = fmaf(pe[e], vv[e].z, o[i][2]);
          o[i][3] = fmaf(pe[e], vv[e].w, o[i][3]);
        }
      }
    }
    __syncthreads();                   // the buffer is refilled in the next step
  }
#pragma unroll
  for (int i = 0; i < R; ++i) {
    const int row = blk.row0 + ty * R + i;
    if (row >= blk.rows) continue;
    const int token = row / a.group, head = blk.h * a.group + row - token * a.group;
    const int at = blk.seq.first + token;
    if (a.n_split == 1) {
      const float inv = l[i] > 0.f ? 1.f / l[i] : (l[i] == l[i] ? 0.f : l[i]);
      *reinterpret_cast<float4*>(static_cast<float*>(a.out.p) + at * a.out.st + head * a.out.sh + 4 * tx) =
          make_float4(o[i][0] * inv, o[i][1] * inv, o[i][2] * inv, o[i][3] * inv);
      if (a.lse && tx == 0)
        a.lse[static_cast<long long>(head) * a.n_tokens + at] =
            l[i] == 0.f ? -INFINITY : (m[i] * a.scale_log2 + log2f(l[i])) * LN2;
    } else {
      const long long pr = (static_cast<long long>(blk.split) * a.n_tokens + at) * a.q.heads + head;
      if (blk.ntile > 0)
        *reinterpret_cast<float4*>(a.part_o + pr * D + 4 * tx) = make_float4(o[i][0], o[i][1], o[i][2], o[i][3]);
      if (tx == 0) *reinterpret_cast<float2*>(a.part_ml + pr * 2) = make_float2(m[i], l[i]);
    }
  }
}

// ---- joining the splits ---------------------------------------------------------
// o = sum_s 2^((m_s - m) c) o_s / sum_s 2^((m_s - m) c) l_s.  One warp per row
// (token, head), two channels per lane; a split that saw no key has l = 0 and no o.
template <typename T>
__global__ void __launch_bounds__(128) cache_join_kernel(const __grid_constant__ CacheAttnArgs a) {
  const int lane = threadIdx.x & 31;
  const long long rows = static_cast<long long>(a.n_tokens) * a.q.heads;
  const long long row = static_cast<long long>(blockIdx.x) * 4 + (threadIdx.x >> 5);
  if (row >= rows) return;
  const int at = static_cast<int>(row / a.q.heads), head = static_cast<int>(row - static_cast<long long>(at) * a.q.heads);
  // the row's sequence: rows of none, and of a refused one, stay as they are
  int lo = 0, hi = a.c.batch;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (a.cu[mid] <= at) lo = mid; else hi = mid;
  }
  if (a.cu[lo] > at || a.cu[lo + 1] <= at) return;
  if (!sequence_of(a, lo).ok) return;
  float mx = -INFINITY;
  for (int s = lane; s < a.n_split; s += 32) {
    const float2 ml = *reinterpret_cast<const float2*>(a.part_ml + (s * rows + row) * 2);
    if (ml.y != 0.f) mx = fmaxf(mx, ml.x);
  }
#pragma unroll
  for (int w = 16; w > 0; w >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, w));
  const float mu = (mx == -INFINITY) ? 0.f : mx;
  float l = 0.f, o0 = 0.f, o1 = 0.f;
#pragma unroll 4
  for (int s = 0; s < a.n_split; ++s) {
    const float2 ml = *reinterpret_cast<const float2*>(a.part_ml + (s * rows + row) * 2);
    if (ml.y == 0.f) continue;
    const float2 ov = *reinterpret_cast<const float2*>(a.part_o + (s * rows + row) * D + 2 * lane);
    const float w = ex2((ml.x - mu) * a.scale_log2);
    l = fmaf(w, ml.y, l);
    o0 = fmaf(w, ov.x, o0);
    o1 = fmaf(w, ov.y, o1);
  }
  const float inv = l > 0.f ? 1.f / l : (l == l ? 0.f : l);
  T* out = static_cast<T*>(a.out.p) + at * a.out.st + head * a.out.sh + 2 * lane;
  if constexpr (sizeof(T) == 2) *reinterpret_cast<uint32_t*>(out) = pack_bf16(o0 * inv, o1 * inv);
  else *reinterpret_cast<float2*>(out) = make_float2(o0 * inv, o1 * inv);
  if (a.lse && lane == 0)
    a.lse[static_cast<long long>(head) * a.n_tokens + at] = l == 0.f ? -INFINITY : (mu * a.scale_log2 + log2f(l)) * LN2;
}

// ---- host -------------------------------------------------------------------------
// a pool of pages as [rows][64] with boxes of one page (at most 128 rows)
bool pool_map(CUtensorMap* m, const void* base, const PagedCache& c) {
  EncodeTiledFn fn = encode_fn();
  if (!fn) return false;
  const int page = 1 << c.page_shift;
  const cuuint64_t dims[2] = {64, static_cast<cuuint64_t>(c.num_pages) * c.heads * page};
  const cuuint64_t strides[1] = {128};
  const cuuint32_t box[2] = {64, static_cast<cuuint32_t>(page < TN ? page : TN)};
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
cudaError_t launch_tc(const CacheAttnArgs& a, unsigned blocks, cudaStream_t st) {
  using L = Lay<KIND>;
  static std::atomic<unsigned long long> done{0};
  cudaError_t e = allow_smem(cache_attn_kernel<KIND>, L::BYTES, done);
  if (e != cudaSuccess) return e;
  CUtensorMap mk, mv;
  if (!pool_map(&mk, a.c.k, a.c) || !pool_map(&mv, a.c.v, a.c)) return cudaErrorInvalidValue;
  cache_attn_kernel<KIND><<<blocks, L::NTHREADS, L::BYTES, st>>>(mk, mv, a);
  return cudaGetLastError();
}

template <int TR>
cudaError_t launch_f32(const CacheAttnArgs& a, unsigned blocks, cudaStream_t st) {
  static std::atomic<unsigned long long> done{0};
  cudaError_t e = allow_smem(cache_attn_f32_kernel<TR>, FLay<TR>::BYTES, done);
  if (e != cudaSuccess) return e;
  cache_attn_f32_kernel<TR><<<blocks, 256, FLay<TR>::BYTES, st>>>(a);
  return cudaGetLastError();
}

}  // namespace

CacheAttnPlan plan_cache_attn(bool fp32, int batch, int kv_heads, int q_heads, long long n_tokens, int max_new,
                              long long max_len) {
  CacheAttnPlan p;
  const long long most = n_tokens < max_new ? n_tokens : max_new;
  const long long rows = most * (q_heads / kv_heads);
  int tile, keys, slots, least;      // rows and keys per tile, blocks that run at once, key tiles worth a split
  if (fp32) {
    p.kind = rows <= 16 ? F32_16 : F32_64;
    tile = rows <= 16 ? 16 : 64;
    keys = FK;
    slots = 296;
    least = 4;
  } else if (rows <= 32) {
    p.kind = QUARTERS;
    tile = 32;
    keys = TN;
    slots = 296;
    least = 4;
  } else if (rows <= 128) {
    p.kind = ONE_TILE;
    tile = 128;
    keys = TN;
    slots = 296;
    least = 4;
  } else {
    p.kind = TWO_TILES;
    tile = 256;
    keys = TN;
    slots = 148;
    least = 16;
  }
  p.row_tiles = static_cast<int>((rows + tile - 1) / tile);
  if (p.row_tiles < 1) p.row_tiles = 1;
  const long long blocks = static_cast<long long>(batch) * kv_heads * p.row_tiles;
  const long long ktiles = (max_len + keys - 1) / keys;
  long long ns = 1, most_splits = ktiles / least;
  if (most_splits > 128) most_splits = 128;
  if (blocks < 2 * slots && most_splits > 1) {
    // the fewest splits that fill the last wave best
    double best = 0.0;
    const long long top = (4 * slots + blocks - 1) / blocks;
    for (long long n = 1; n <= most_splits && n <= top; ++n) {
      const long long tot = blocks * n;
      const double eff = static_cast<double>(tot) / static_cast<double>(slots * ((tot + slots - 1) / slots));
      if (eff > best + 0.02) {
        best = eff;
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
  const unsigned blocks = static_cast<unsigned>(a.c.batch) * a.c.heads * a.row_tiles * a.n_split;
  cudaError_t e;
  switch (kind) {
    case TWO_TILES: e = launch_tc<TWO_TILES>(a, blocks, st); break;
    case ONE_TILE: e = launch_tc<ONE_TILE>(a, blocks, st); break;
    case QUARTERS: e = launch_tc<QUARTERS>(a, blocks, st); break;
    case F32_64: e = launch_f32<64>(a, blocks, st); break;
    case F32_16: e = launch_f32<16>(a, blocks, st); break;
    default: return cudaErrorInvalidValue;
  }
  if (e != cudaSuccess || a.n_split == 1) return e;
  const long long rows = static_cast<long long>(a.n_tokens) * a.q.heads;
  const unsigned grid = static_cast<unsigned>((rows + 3) / 4);
  if (fp32) cache_join_kernel<float><<<grid, 128, 0, st>>>(a);
  else cache_join_kernel<__nv_bfloat16><<<grid, 128, 0, st>>>(a);
  return cudaGetLastError();
}

}  // namespace gsa
