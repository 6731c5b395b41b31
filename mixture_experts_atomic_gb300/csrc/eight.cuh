// Rows in 8-bit floating point: e4m3 values (three bits of mantissa, largest
// 448) with an fp32 scale for each 128 columns of a row.
//
//   s = 2^ceil(log2(max|v| / 448))     q = e4m3(v / s), to nearest, ties to even
//
// The scale is a power of two, so that dividing by it is exact and the values
// round once, as e4m3 does at any scale; what a power of two leaves unused of
// the range, one binade at most, is at its small end (the least normal value is
// 2^-14 to 2^-15 of the block's largest, the least of all 2^-17 to 2^-18).  Whoever reads rows takes any fp32 scale.
//
// A NaN or an infinity makes the scale NaN, and with it the block: e4m3 has no
// infinity, and the conversion would make it 448.  The largest magnitude is
// taken of the bit patterns, in which both are above every number.
#pragma once

#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <stdint.h>

namespace moeblaze {

constexpr int kBlock8 = 128;

struct Rows8 {
  uint8_t* q;
  float* s;
};

__host__ __device__ inline int blocks8(int d) { return (d + kBlock8 - 1) / kBlock8; }

__device__ __forceinline__ uint32_t abs_bits(float v) { return __float_as_uint(v) & 0x7fffffffu; }

struct Scale8 {
  float s, inv;  // 2^k and 2^-k
};
// of a block whose largest magnitude has these bits: m 2^e is at most 448 2^k
// = 1.75 2^(8 + k) for k = e - 8, or one more where m > 1.75.  Below 2^-118 k
// stays at -126, the least normal number's, so that 2^-k is finite.
__device__ __forceinline__ Scale8 scale8(uint32_t bits) {
  if (bits >= 0x7f800000u) return Scale8{__uint_as_float(0x7fffffffu), 0.f};
  const int k = max((int)(bits >> 23) - 8 + ((bits & 0x7fffffu) > 0x600000u ? 1 : 0), 1);
  return Scale8{__uint_as_float((uint32_t)k << 23), __uint_as_float((uint32_t)(254 - k) << 23)};
}

// the same for fp16: the largest comes to 2^14 or more
__device__ __forceinline__ Scale8 scale16(uint32_t bits) {
  if (bits >= 0x7f800000u) return Scale8{__uint_as_float(0x7fffffffu), 0.f};
  const int k = max((int)(bits >> 23) - 14, 1);
  return Scale8{__uint_as_float((uint32_t)k << 23), __uint_as_float((uint32_t)(254 - k) << 23)};
}

// four values, the first in the low byte
__device__ __forceinline__ uint32_t e4m3x4(const float* v, float inv) {
  const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(v[0] * inv, v[1] * inv), __NV_SATFINITE, __NV_E4M3);
  const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(v[2] * inv, v[3] * inv), __NV_SATFINITE, __NV_E4M3);
  return lo | hi << 16;
}

// the values of four e4m3 bytes, times s
__device__ __forceinline__ void e4m3_values(uint32_t u, float s, float* v) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(u >> (16 * i)), __NV_E4M3);
    const float2 f = __half22float2(__half2(h));
    v[2 * i] = f.x * s;
    v[2 * i + 1] = f.y * s;
  }
}

}  // namespace moeblaze
