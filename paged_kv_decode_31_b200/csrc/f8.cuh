// f8.cuh -- arithmetic of the 8-bit cache: conversions between fp32 / fp16
// pairs and the 8-bit floating types, the power-of-two block scales, and the
// splits that let 8-bit tensor-core operands carry 16-bit values.
//
// The cache holds e4m3 values; a value's block and KV head have a scale 2^e,
// kept as the byte e + 127 (E8M0), with e in [kScaleExpMin, kScaleExpMax].
#pragma once

#include <cuda_fp16.h>

#include <cstdint>

namespace pkv {

constexpr int kErrScale = 32;  // PKV_DEVERR_SCALE in pagedkv.h
constexpr int kScaleExpMin = -63, kScaleExpMax = 63;
constexpr int kScaleByteMin = kScaleExpMin + 127, kScaleByteMax = kScaleExpMax + 127;

// 2^(byte - 127) and 2^(127 - byte) for a scale byte in range.
__device__ __forceinline__ float scale_of(int byte) { return __int_as_float(byte << 23); }
__device__ __forceinline__ float inv_scale_of(int byte) { return __int_as_float((254 - byte) << 23); }

// Two values to 8 bits, the first in the low byte; round to nearest even,
// values past the largest finite one saturate, NaN stays NaN.
__device__ __forceinline__ uint32_t e4m3x2_of(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint32_t e5m2x2_of(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e5m2x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint32_t e4m3x2_of(__half2 v) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(r) : "r"(*reinterpret_cast<uint32_t *>(&v)));
  return r;
}
// Back to fp16: exact (every e4m3 value is an fp16 value).
__device__ __forceinline__ __half2 half2_of_e4m3x2(uint32_t v) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(static_cast<uint16_t>(v)));
  return *reinterpret_cast<__half2 *>(&r);
}
// A query row enters K Q^T as two 8-bit operands of one scale: the row times
// 2^k, k chosen so that its largest magnitude lies in [128, 256), is
// hi + lo with hi = e4m3(x) and lo = e5m2(x - hi).  A bf16 value has 8
// significant bits, hi takes the first 4 and the remainder (at most 8 units of
// the last bit) needs 3, which e5m2 has: the sum is exact for every element
// down to 2^-13 of the row's largest, and within 2^-21 of that largest below
// (where hi is subnormal).
struct Split2 {
  uint32_t hi, lo;  // two elements each, packed
};
__device__ __forceinline__ Split2 split_q(float x0, float x1) {
  Split2 s;
  s.hi = e4m3x2_of(x0, x1);
  const float2 h = __half22float2(half2_of_e4m3x2(s.hi));
  s.lo = e5m2x2_of(__fsub_rn(x0, h.x), __fsub_rn(x1, h.y));
  return s;
}

// A probability in [0, 256] enters P V as two e4m3 operands, hi = e4m3(p) and
// mid = e4m3(16 (p - hi)), whose products are accumulated apart and joined as
// hi + mid / 16 in fp32.  hi leaves at most 2^-4 of p's power of two, mid keeps
// 4 bits of that: p is off by at most 2^-9 relative (5.9e-4 rms), half of what
// rounding P to bf16 would do and a quarter of a bf16 output's own half step;
// below 2^-6 by at most 2^-14, half of mid's smallest step.  (The differences
// are taken from p rounded to fp16, 2^-11, which is below all of that.)
struct SplitP {
  uint32_t hi, mid;
};
__device__ __forceinline__ SplitP split_p(float p0, float p1) {
  SplitP s;
  const __half2 r = __floats2half2_rn(p0, p1);
  s.hi = e4m3x2_of(r);
  s.mid = e4m3x2_of(__hmul2(__hsub2(r, half2_of_e4m3x2(s.hi)), __floats2half2_rn(16.f, 16.f)));
  return s;
}
constexpr float kMidScale = 0.0625f;

}  // namespace pkv
