// q8.cuh -- device helpers of the 8-bit cache kernels: codes, scales, pages.
#pragma once

#include <cuda_fp16.h>

#include "common.cuh"
#include "q8.h"

namespace lychee {

enum { kCodeE4M3 = 0, kCodeInt8 = 1 };

// The scale of a block is 2^e, e in [kScaleExpMin, kScaleExpMax]: the smallest
// that brings the block's largest magnitude within the codes' range.  A power of
// two makes dividing by it exact, so a value is rounded once, and lets e4m3
// codes move to a larger scale without loss but for those that leave the normal
// range.
constexpr int kScaleExpMin = -60, kScaleExpMax = 60;

__device__ __forceinline__ float exp2_int(int e) { return __int_as_float((e + 127) << 23); }

// ceil(log2(amax / M)) for finite amax > 0, clamped: with amax = f 2^x (1 <= f <
// 2) and M = m 2^y it is x - y, one more when f > m.  M = 448 = 1.75 * 2^8 for
// e4m3, 127 = 1.984375 * 2^6 for int8.  Subnormal amax lands at the lower clamp.
template <int CODE>
__device__ __forceinline__ int scale_exp(float amax) {
  const uint32_t u = __float_as_uint(amax);
  const int y = CODE == kCodeE4M3 ? 8 : 6;
  const uint32_t m = CODE == kCodeE4M3 ? 0x600000u : 0x7e0000u;   // fraction bits of m
  const int e = (int)(u >> 23) - 127 - y + ((u & 0x7fffffu) > m ? 1 : 0);
  return max(kScaleExpMin, min(kScaleExpMax, e));
}

// Four values (already divided by the scale) -> four codes, to nearest, ties to
// even, saturated; NaN -> 0.
template <int CODE>
__device__ __forceinline__ uint32_t quantise4(float a, float b, float c, float d) {
  a = a == a ? a : 0.f;
  b = b == b ? b : 0.f;
  c = c == c ? c : 0.f;
  d = d == d ? d : 0.f;
  if constexpr (CODE == kCodeE4M3) {
    uint16_t lo, hi;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(b), "f"(a));
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(d), "f"(c));
    return (uint32_t)lo | ((uint32_t)hi << 16);
  } else {
    auto one = [](float x) {
      return (uint32_t)__float2int_rn(fminf(fmaxf(x, -127.f), 127.f)) & 0xffu;
    };
    return one(a) | (one(b) << 8) | (one(c) << 16) | (one(d) << 24);
  }
}

// Four codes -> their values as two half pairs (exact: both code types fit 11
// bits).
template <int CODE>
__device__ __forceinline__ void codes_to_half(uint32_t w, uint32_t& lo, uint32_t& hi) {
  if constexpr (CODE == kCodeE4M3) {
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\t"
        "cvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
        : "=r"(lo), "=r"(hi)
        : "r"(w));
  } else {
    // 0x6400 | u is the half 1024 + u: u = code + 128, then subtract 1152
    w ^= 0x80808080u;
    const __half2 off = __half2(__ushort_as_half(0x6480), __ushort_as_half(0x6480));
    uint32_t a = __byte_perm(w, 0x64646464u, 0x4140), b = __byte_perm(w, 0x64646464u, 0x4342);
    __half2 ha = __hsub2(*reinterpret_cast<__half2*>(&a), off);
    __half2 hb = __hsub2(*reinterpret_cast<__half2*>(&b), off);
    lo = *reinterpret_cast<uint32_t*>(&ha);
    hi = *reinterpret_cast<uint32_t*>(&hb);
  }
}

template <int CODE>
__device__ __forceinline__ float4 codes_to_float(uint32_t w) {
  uint32_t lo, hi;
  codes_to_half<CODE>(w, lo, hi);
  const float2 a = __half22float2(*reinterpret_cast<__half2*>(&lo));
  const float2 b = __half22float2(*reinterpret_cast<__half2*>(&hi));
  return make_float4(a.x, a.y, b.x, b.y);
}

}  // namespace lychee
