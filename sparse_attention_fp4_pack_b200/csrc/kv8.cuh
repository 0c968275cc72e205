// Helpers shared by the kernels of the paged 8-bit KV cache (kv8.cu, kv8_attn.cu).
#pragma once

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

}  // namespace csa2
