// f8.cuh -- arithmetic of the 8-bit cache: conversions between fp32 / fp16
// pairs and the 8-bit floating types, the power-of-two block scales, and the
// splits that let 8-bit tensor-core operands carry 16-bit values.
//
// The cache holds e4m3 values; a value's block and KV head have a scale 2^e,
// kept as the byte e + 127 (E8M0), with e in [kScaleExpMin, kScaleExpMax].  The
// attention kernels take any two of these beside each other in one row.
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
__device__ __forceinline__ uint32_t e5m2x2_of(__half2 v) {
  uint16_t r;
  asm("cvt.rn.satfinite.e5m2x2.f16x2 %0, %1;" : "=h"(r) : "r"(*reinterpret_cast<uint32_t *>(&v)));
  return r;
}
// Back to fp16: exact (every e4m3 or e5m2 value is an fp16 value).
__device__ __forceinline__ __half2 half2_of_e4m3x2(uint32_t v) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(static_cast<uint16_t>(v)));
  return *reinterpret_cast<__half2 *>(&r);
}
__device__ __forceinline__ __half2 half2_of_e5m2x2(uint32_t v) {
  uint32_t r;
  asm("cvt.rn.f16x2.e5m2x2 %0, %1;" : "=r"(r) : "h"(static_cast<uint16_t>(v)));
  return *reinterpret_cast<__half2 *>(&r);
}
// A query row enters K Q^T as two e4m3 operands whose products are accumulated
// apart and joined in fp32 as hi + lo / 16: the row times 2^k, k chosen so that
// its largest magnitude lies in [128, 256), is taken apart as hi = e4m3(x) and
// lo = e4m3(16 (x - hi)).  A bf16 value has 8 significant bits, hi takes the
// first 4 and lo holds the rest: exact for every element down to 2^-13 of the
// row's largest, and within 2^-21 of that largest below.
struct Split2 {
  uint32_t hi, lo;  // two elements each, packed
};
__device__ __forceinline__ Split2 split_q(float x0, float x1) {
  Split2 s;
  s.hi = e4m3x2_of(x0, x1);
  const float2 h = __half22float2(half2_of_e4m3x2(s.hi));
  s.lo = e4m3x2_of(__fmul_rn(__fsub_rn(x0, h.x), 16.f), __fmul_rn(__fsub_rn(x1, h.y), 16.f));
  return s;
}
__device__ __forceinline__ float join_q(float hi, float lo) { return __fmaf_rn(lo, 0.0625f, hi); }

// The form with one scale, for two products into one accumulator: lo = e5m2(x -
// hi), whose 3 bits hold the at most 8 units that hi leaves of a bf16 value.
__device__ __forceinline__ uint32_t e5m2x2_of(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e5m2x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ Split2 split_q_one_scale(float x0, float x1) {
  Split2 s;
  s.hi = e4m3x2_of(x0, x1);
  const float2 h = __half22float2(half2_of_e4m3x2(s.hi));
  s.lo = e5m2x2_of(__fsub_rn(x0, h.x), __fsub_rn(x1, h.y));
  return s;
}

// A probability in [0, 2^15], rounded to fp16 (11 bits: off by at most 2^-11
// relative, 2^-25 where fp16 is subnormal), enters P V as three e5m2 operands
// whose products are accumulated apart and joined in fp32 as hi + (mid + lo /
// 16) / 16:
//   hi = e5m2(p),  mid = e5m2(16 (p - hi)),  lo = e5m2(16 (16 (p - hi) - mid)).
// The differences are exact in fp16.  e5m2 rounds to 3 bits, so of p's 11 bits
// hi leaves at most 2^7 units of the last and mid at most 2^3, which lo holds:
// the three are the fp16 value, the subnormal ones included (hi's smallest step
// is 2^-16, lo's 2^-16 / 2^8 is fp16's).  (e4m3 pieces, with a bit more each but
// 2^7 less range, lost every p below 2^-18 against a largest of 2^2 to 2^8:
// with one token 12 to 15 nats above thousands of others, all of theirs.)
struct SplitP {
  uint32_t hi, mid, lo;
};
__device__ __forceinline__ SplitP split_p(float p0, float p1) {
  SplitP s;
  const __half2 k16 = __floats2half2_rn(16.f, 16.f);
  __half2 r = __floats2half2_rn(p0, p1);
  s.hi = e5m2x2_of(r);
  r = __hmul2(__hsub2(r, half2_of_e5m2x2(s.hi)), k16);
  s.mid = e5m2x2_of(r);
  r = __hmul2(__hsub2(r, half2_of_e5m2x2(s.mid)), k16);
  s.lo = e5m2x2_of(r);
  return s;
}
__device__ __forceinline__ float join_p(float hi, float mid, float lo) {
  return __fmaf_rn(__fmaf_rn(lo, 0.0625f, mid), 0.0625f, hi);
}

}  // namespace pkv
