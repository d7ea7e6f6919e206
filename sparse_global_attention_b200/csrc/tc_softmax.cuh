// Softmax steps of the tensor-core attention kernels (a thread owns a row of
// S) and the host side of their tensor maps.
#pragma once
#include <cuda.h>

#include "tc_ptx.cuh"

namespace gsa {
namespace tc {

// one arrival per warp, after every lane's preceding work (fences included)
__device__ __forceinline__ void warp_arrive(uint32_t bar) {
  __syncwarp();
  if ((threadIdx.x & 31) == 0) mbar_arrive(bar);
}

// Two exponentials of the softmax with packed fp32x2 arithmetic (one FFMA2
// for both arguments, one FADD2 for both running sums): half the FMA-pipe
// issue slots of the scalar form, and exactly its roundings.
__device__ __forceinline__ void exp2_pair(uint32_t s0, uint32_t s1, float sl2, float nmb, float& l0, float& l1,
                                          float& p0, float& p1) {
  float x0, x1;
  asm("{\n .reg .b64 a, b, c, d;\n"
      " mov.b64 a, {%2, %3};\n mov.b64 b, {%4, %4};\n mov.b64 c, {%5, %5};\n"
      " fma.rn.f32x2 d, a, b, c;\n mov.b64 {%0, %1}, d;\n}\n"
      : "=f"(x0), "=f"(x1)
      : "r"(s0), "r"(s1), "f"(sl2), "f"(nmb));
  p0 = ex2(x0);
  p1 = ex2(x1);
  asm("{\n .reg .b64 a, b;\n"
      " mov.b64 a, {%0, %1};\n mov.b64 b, {%2, %3};\n add.rn.f32x2 a, a, b;\n mov.b64 {%0, %1}, a;\n}\n"
      : "+f"(l0), "+f"(l1)
      : "f"(p0), "f"(p1));
}

// max of 32 values with 4 independent chains
__device__ __forceinline__ float max32(const uint32_t* v) {
  float m0 = __uint_as_float(v[0]), m1 = __uint_as_float(v[1]), m2 = __uint_as_float(v[2]),
        m3 = __uint_as_float(v[3]);
#pragma unroll
  for (int e = 4; e < 32; e += 4) {
    m0 = fmaxf(m0, __uint_as_float(v[e]));
    m1 = fmaxf(m1, __uint_as_float(v[e + 1]));
    m2 = fmaxf(m2, __uint_as_float(v[e + 2]));
    m3 = fmaxf(m3, __uint_as_float(v[e + 3]));
  }
  return fmaxf(fmaxf(m0, m1), fmaxf(m2, m3));
}

__device__ __forceinline__ void apply_mask(uint32_t* v, uint32_t msk) {
#pragma unroll
  for (int e = 0; e < 32; ++e) v[e] = ((msk >> e) & 1u) ? v[e] : 0xff800000u;   // -inf
}

__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,"
      "%14,%15,%16};\n" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
      "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}

// ---- tensor maps (host) --------------------------------------------------------
typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                  const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

inline EncodeTiledFn encode_fn() {
  static EncodeTiledFn fn = nullptr;
  if (!fn) {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<EncodeTiledFn>(p);
  }
  return fn;
}

}  // namespace tc
}  // namespace gsa
