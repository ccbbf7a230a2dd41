// Device code shared by the 8-bit serving kernels (tokens.cu, int8_mm.cu):
// typed element access, the token quantizer's arithmetic, the products'
// epilogue.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "common.cuh"

namespace gptq {

// ------------------------------------------------------------ element access
template <typename T>
__device__ __forceinline__ float to_f32(T x);
template <>
__device__ __forceinline__ float to_f32<float>(float x) { return x; }
template <>
__device__ __forceinline__ float to_f32<__half>(__half x) { return __half2float(x); }
template <>
__device__ __forceinline__ float to_f32<__nv_bfloat16>(__nv_bfloat16 x) { return __bfloat162float(x); }
template <typename T>
__device__ __forceinline__ T from_f32(float x);
template <>
__device__ __forceinline__ float from_f32<float>(float x) { return x; }
template <>
__device__ __forceinline__ __half from_f32<__half>(float x) { return __float2half_rn(x); }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float x) { return __float2bfloat16_rn(x); }

// Eight consecutive elements as loaded; left elements (>= 1) lie inside the
// row, those past its end read as zero.  vec: the address is 16-byte aligned.
template <typename T>
struct Raw8 {
  alignas(16) T v[8];
};
template <typename T>
__device__ __forceinline__ Raw8<T> load8(const T* __restrict__ p, int left, bool vec) {
  Raw8<T> r;
  if (vec && left >= 8) {
#pragma unroll
    for (int i = 0; i < (int)sizeof(T) / 2; ++i)
      reinterpret_cast<uint4*>(r.v)[i] = reinterpret_cast<const uint4*>(p)[i];
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) r.v[i] = i < left ? p[i] : from_f32<T>(0.f);
  }
  return r;
}
template <typename T>
__device__ __forceinline__ void store8(T* __restrict__ p, const float* v, int left, bool vec) {
  Raw8<T> r;
#pragma unroll
  for (int i = 0; i < 8; ++i) r.v[i] = from_f32<T>(v[i]);
  if (vec && left >= 8) {
#pragma unroll
    for (int i = 0; i < (int)sizeof(T) / 2; ++i)
      reinterpret_cast<uint4*>(p)[i] = reinterpret_cast<const uint4*>(r.v)[i];
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < left) p[i] = r.v[i];
  }
}

// ------------------------------------------------------------ tensor cores
// Instruction descriptor of kind::i8: 32-bit integer accumulator (bits 4-5 =
// 2), both operands signed (bits 7-9 and 10-12 = 1) and K-major, N >> 3 at
// bits 17-22, M >> 4 at bits 24-28.
__host__ __device__ constexpr uint32_t idesc_i8(uint32_t M, uint32_t N) {
  return (2u << 4) | (1u << 7) | (1u << 10) | ((N >> 3) << 17) | ((M >> 4) << 24);
}

__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ uint32_t map_to_rank(uint32_t addr, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}

// ------------------------------------------------------------ token quantizer
// s = RN(max |x| RN(1/127)), code = clamp(rint(RN(x / s)), -127, 127), fp32.
// top: the bit pattern of the row's largest magnitude, where NaN and infinity
// sort above every finite value and give s = NaN and codes of zero.  The
// quotient comes from quot_rn (five operations instead of a divide) while s
// is in its range; an x too small for that range has |x / s| < 1/2 either
// way, its code is 0.
struct TokenScale {
  float scale, inv;
  bool some, fast;
  __device__ __forceinline__ explicit TokenScale(uint32_t top) {
    const bool finite = top < 0x7f800000u;
    scale = finite ? __uint_as_float(top) * (1.f / 127.f) : __uint_as_float(0x7fc00000u);
    some = finite && scale > 0.f;
    fast = scale >= 0x1p-60f && scale <= 0x1p60f;
    inv = fast ? __frcp_rn(scale) : 0.f;
  }
  __device__ __forceinline__ int code(float x) const {
    if (!some) return 0;
    const int c = __float2int_rn(fast ? quot_rn(x, scale, inv) : __fdiv_rn(x, scale));
    return min(127, max(-127, c));
  }
};

// ------------------------------------------------------------------ epilogue
// The gate's activation in fp32.  tanh's gelu is written through the logistic
// function, 0.5 (1 + tanh z) = 1 / (1 + exp(-2 z)), so both need one
// exponential and one quotient (__expf and __fdividef: a few units in the
// last place of fp32).
__device__ __forceinline__ float activate(float g, int act) {
  if (act == GPTQ_ACT_GELU) return 0.5f * g * (1.f + erff(g * 0.70710678118654752f));
  const float z = act == GPTQ_ACT_SILU ? g : 1.5957691216057308f * fmaf(0.044715f * g * g, g, g);
  return __fdividef(g, 1.f + __expf(-z));
}

// One product's value from its exact integer sum.
__device__ __forceinline__ float scaled(int acc, int zero, int tsum, float tscale, float wscale) {
  return (float)(acc - zero * tsum) * tscale * wscale;
}

}  // namespace gptq
