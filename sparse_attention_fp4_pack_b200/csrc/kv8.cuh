// Helpers shared by the kernels of the paged 8-bit KV cache (kv8.cu, kv8_attn.cu).
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "csa2_device.cuh"

namespace csa2 {

// log2 of a power of two.
inline int log2_of(int v) {
  int n = 0;
  while ((1 << n) < v) ++n;
  return n;
}

// Two fp32 -> two E4M3 bytes (lo in bits 7..0), round to nearest even, saturating at 448.
__device__ __forceinline__ uint32_t e4m3x2_sat(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

// Two E4M3 bytes -> f16x2, exact.
__device__ __forceinline__ uint32_t f16x2_of_e4m3x2(uint32_t b) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"((uint16_t)b));
  return r;
}

// 4 E4M3 bytes -> 4 fp32, exact.
__device__ __forceinline__ void e4m3x4_f32(uint32_t w, float* x) {
  uint32_t lo, hi;
  asm("{\n\t.reg .b16 a, b;\n\t"
      "mov.b32 {a, b}, %2;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, a;\n\t"
      "cvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
      : "=r"(lo), "=r"(hi)
      : "r"(w));
  const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&lo));
  const float2 b = __half22float2(*reinterpret_cast<const __half2*>(&hi));
  x[0] = a.x;
  x[1] = a.y;
  x[2] = b.x;
  x[3] = b.y;
}

// 8 16-bit elements -> fp32.
template <typename T>
__device__ __forceinline__ void unpack8(uint4 w, float (&x)[8]);
template <>
__device__ __forceinline__ void unpack8<__nv_bfloat16>(uint4 w, float (&x)[8]) {
  const uint32_t v[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = bf16_lo(v[i]);
    x[2 * i + 1] = bf16_hi(v[i]);
  }
}
template <>
__device__ __forceinline__ void unpack8<__half>(uint4 w, float (&x)[8]) {
  const uint32_t v[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&v[i]));
    x[2 * i] = f.x;
    x[2 * i + 1] = f.y;
  }
}

}  // namespace csa2
