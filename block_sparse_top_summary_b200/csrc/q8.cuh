// The 8-bit cache formats: codes with one power-of-two fp32 scale per (page, KV
// head), a row element standing for code * scale.
//   e4m3: |code| <= 448, 3 fraction bits, subnormal step 2^-9;
//   i8:   |code| <= 127.
// A power of two keeps every step but the one rounding exact: x / scale, the held
// value (at most 8 significant bits, so also exact in bf16) and, except where
// bits fall off, old codes under a larger scale.
#pragma once

#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <stdint.h>

#include "ssa.h"

namespace ssa {

// The least 2^e, e >= -126, with amax <= QMAX 2^e, from the bits of amax (finite,
// not negative).  QMAX = 1.75 * 2^8 (e4m3) or 1.984375 * 2^6 (i8).
template <int F>
__device__ __forceinline__ float q8_scale(uint32_t amax_bits) {
  constexpr uint32_t kMant = F == SSA_E4M3 ? 0x600000u : 0x7e0000u;
  constexpr int kBits = F == SSA_E4M3 ? 8 : 6;
  // biased exponent of the scale; a subnormal amax has field 0 and ends at 1
  int e = (int)(amax_bits >> 23) - kBits + ((amax_bits & 0x7fffffu) > kMant ? 1 : 0);
  e = e < 1 ? 1 : e;
  return __uint_as_float((uint32_t)e << 23);
}

// Code of y = x / scale, |y| <= QMAX: nearest, ties to even.
template <int F>
__device__ __forceinline__ uint32_t q8_code(float y) {
  if constexpr (F == SSA_E4M3) {
    return (uint32_t)__nv_cvt_float_to_fp8(y, __NV_SATFINITE, __NV_E4M3);
  } else {
    return (uint32_t)__float2int_rn(y) & 255u;
  }
}

// Two codes, a in the low byte.
template <int F>
__device__ __forceinline__ uint32_t q8_code2(float a, float b) {
  if constexpr (F == SSA_E4M3) {
    return (uint32_t)__nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
  } else {
    return q8_code<F>(a) | (q8_code<F>(b) << 8);
  }
}

// Four codes of a word as two f16 pairs (exact: both formats fit f16): lo holds
// bytes 0 and 1, hi bytes 2 and 3.
template <int F>
__device__ __forceinline__ void q8_to_half4(uint32_t w, uint32_t& lo, uint32_t& hi) {
  if constexpr (F == SSA_E4M3) {
    asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\t"
        "cvt.rn.f16x2.e4m3x2 %0, l;\n\tcvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
        : "=r"(lo), "=r"(hi)
        : "r"(w));
  } else {
    // byte + 128 as the low bits of 1024 + byte + 128, then minus 1152
    const uint32_t u = w ^ 0x80808080u;
    const __half2 off = __half2half2(__ushort_as_half(0x6480));  // 1152
    uint32_t a = __byte_perm(u, 0x64646464u, 0x4140);
    uint32_t b = __byte_perm(u, 0x64646464u, 0x4342);
    const __half2 ha = __hsub2(*reinterpret_cast<__half2*>(&a), off);
    const __half2 hb = __hsub2(*reinterpret_cast<__half2*>(&b), off);
    lo = *reinterpret_cast<const uint32_t*>(&ha);
    hi = *reinterpret_cast<const uint32_t*>(&hb);
  }
}

// Eight codes as floats.
template <int F>
__device__ __forceinline__ void q8_unpack8(uint2 c, float* out) {
  uint32_t h[4];
  q8_to_half4<F>(c.x, h[0], h[1]);
  q8_to_half4<F>(c.y, h[2], h[3]);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h[i]));
    out[2 * i] = f.x;
    out[2 * i + 1] = f.y;
  }
}

template <int F>
__device__ __forceinline__ uint2 q8_pack8(const float* y) {
  return make_uint2(q8_code2<F>(y[0], y[1]) | (q8_code2<F>(y[2], y[3]) << 16),
                    q8_code2<F>(y[4], y[5]) | (q8_code2<F>(y[6], y[7]) << 16));
}

}  // namespace ssa
