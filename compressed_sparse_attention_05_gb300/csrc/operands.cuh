// Attention operands on the tensor cores: dequantisation of MXFP4 and FP8 codes to
// fp16 pairs, and the register-level pieces of the softmax (exp2, reductions).
#pragma once

#include <cuda_fp16.h>

#include "common.cuh"

namespace csa2 {

__device__ __forceinline__ uint32_t word_of(const uint4& v, int i) {
  return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w;
}
// Two E2M1 codes (one byte, even channel in the low nibble) -> f16x2, low half first.
__device__ __forceinline__ uint32_t e2m1x2_f16x2(uint32_t byte) {
  uint32_t r;
  asm("{ .reg .b8 t; cvt.u8.u32 t, %1; cvt.rn.f16x2.e2m1x2 %0, t; }" : "=r"(r) : "r"(byte));
  return r;
}
// Eight E2M1 codes (a word, channel 0 in the low nibble) -> four f16x2.  The bytes are named
// as such: extracting them with shifts would cost as much again (72 against 112 cycles per
// 32 channels and warp pair, conversion and scaling).
__device__ __forceinline__ void e2m1x8_f16x8(uint32_t w, uint32_t& a, uint32_t& b, uint32_t& c, uint32_t& d) {
  asm("{ .reg .b8 x0, x1, x2, x3;\n mov.b32 {x0, x1, x2, x3}, %4;\n cvt.rn.f16x2.e2m1x2 %0, x0;\n"
      " cvt.rn.f16x2.e2m1x2 %1, x1;\n cvt.rn.f16x2.e2m1x2 %2, x2;\n cvt.rn.f16x2.e2m1x2 %3, x3; }"
      : "=r"(a), "=r"(b), "=r"(c), "=r"(d)
      : "r"(w));
}
// Two E4M3 codes (low 16 bits, first code in the low byte) -> f16x2, low half first (exact).
__device__ __forceinline__ uint32_t e4m3x2_f16x2(uint32_t pair) {
  uint32_t r;
  asm("{ .reg .b16 t; cvt.u16.u32 t, %1; cvt.rn.f16x2.e4m3x2 %0, t; }" : "=r"(r) : "r"(pair));
  return r;
}
__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t prmt(uint32_t a, uint32_t b, uint32_t sel) {
  uint32_t r;
  asm("prmt.b32 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(sel));
  return r;
}
// (lo, hi) fp32 -> f16x2 (round to nearest even), lo in the low half.
__device__ __forceinline__ uint32_t f32x2_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
// The same, with the largest finite value in the place of infinity and of what would round to it.
__device__ __forceinline__ uint32_t f32x2_f16x2_finite(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.satfinite.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
// (lo, hi) fp32 -> bf16x2 (round to nearest even), lo in the low half.
__device__ __forceinline__ uint32_t f32x2_bf16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ float f16_lo(uint32_t h2) { return __half2float(__ushort_as_half((unsigned short)(h2 & 0xFFFFu))); }
__device__ __forceinline__ float f16_hi(uint32_t h2) { return __half2float(__ushort_as_half((unsigned short)(h2 >> 16))); }
// Two window codes -> f16x2 of bf16(fp32(e4m3 * scale)) (the window operand).
template <bool kFinite = false>
__device__ __forceinline__ uint32_t win2_f16x2(uint32_t pair, float sc) {
  const uint32_t e = e4m3x2_f16x2(pair);
  const uint32_t bf = f32x2_bf16x2(f16_lo(e) * sc, f16_hi(e) * sc);
  const float lo = __uint_as_float(bf << 16), hi = __uint_as_float(bf & 0xFFFF0000u);
  return kFinite ? f32x2_f16x2_finite(lo, hi) : f32x2_f16x2(lo, hi);
}
__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// Reduction (max or sum) over the 32 lanes of each of 16 columns; lane L
// ends with column L & 15.  v is consumed.
template <bool kMax>
__device__ __forceinline__ float reduce16(float (&v)[16], int lane) {
#pragma unroll
  for (int j = 0; j < 16; ++j) {
    const float o = __shfl_xor_sync(0xffffffffu, v[j], 16);
    v[j] = kMax ? fmaxf(v[j], o) : v[j] + o;
  }
#pragma unroll
  for (int w = 8; w >= 1; w >>= 1) {
    const bool upper = (lane & w) != 0;
#pragma unroll
    for (int j = 0; j < w; ++j) {
      const float send = upper ? v[j] : v[j + w];
      const float keep = upper ? v[j + w] : v[j];
      const float got = __shfl_xor_sync(0xffffffffu, send, w);
      v[j] = kMax ? fmaxf(keep, got) : keep + got;
    }
  }
  return v[0];
}

}  // namespace csa2
