// e4m3 rows with power-of-two block scales: shared by the row quantizer and
// the FP8 GEMM epilogues.
#pragma once

#include <cuda_fp16.h>

#include "common.cuh"

namespace moeq {

constexpr int kFp8Block = 128;   // elements per scale of FP8 rows (and weight block edge)

// Exponent e of the scale 2^e of a block with largest finite magnitude amax:
// the smallest e >= -126 with amax <= 448 * 2^e (448 = 1.75 * 2^8 is the
// largest e4m3 value); 0 for a block of zeros. Taken from the bits of amax, so
// it is exact, and x * 2^-e then rounds once, in the conversion to e4m3.
__device__ __forceinline__ int fp8_block_exp(float amax) {
  const uint32_t b = __float_as_uint(amax);
  if (b == 0u) return 0;
  const int e = static_cast<int>(b >> 23) - 127 - 8 + ((b & 0x7fffffu) > 0x600000u ? 1 : 0);
  return e < -126 ? -126 : e;
}

// 2^e for -126 <= e <= 127.
__device__ __forceinline__ float exp2_int(int e) {
  return __uint_as_float(static_cast<uint32_t>(e + 127) << 23);
}

// E8M0 scale 2^(X - 127): X = 0 is the subnormal 2^-127, X = 255 is NaN.
__device__ __forceinline__ float e8m0_to_float(int X) {
  if (X == 0) return __uint_as_float(0x00400000u);
  return X == 255 ? __uint_as_float(0x7fffffffu) : exp2_int(X - 127);
}

// Four floats to e4m3 (nearest even), a in the lowest byte; magnitudes above
// 448 saturate, NaN stays NaN.
__device__ __forceinline__ uint32_t cvt_e4m3x4(float a, float b, float c, float d) {
  uint16_t lo, hi;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(b), "f"(a));
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(d), "f"(c));
  return static_cast<uint32_t>(lo) | (static_cast<uint32_t>(hi) << 16);
}

// Two e4m3 values (low byte first) to half precision, exactly.
__device__ __forceinline__ float2 e4m3x2_to_float2(uint32_t two) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<uint16_t>(two)));
  const __half2 hh = *reinterpret_cast<const __half2*>(&h);
  return __half22float2(hh);
}

// Magnitude of a finite value, 0 for NaN and infinities.
__device__ __forceinline__ float finite_abs(float v) {
  const float a = fabsf(v);
  return a < INFINITY ? a : 0.0f;
}

// An infinity as NaN (e4m3 has no infinity, and the conversion would give 448).
__device__ __forceinline__ float inf_to_nan(float v) {
  return fabsf(v) < INFINITY ? v : __uint_as_float(0x7fffffffu);
}

}  // namespace moeq
