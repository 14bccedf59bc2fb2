// Activations and their derivatives in fp32, and the 8-bit block format
// (e4m3 codes, a power of two for each 32 elements of a row).
//
// Logistic functions go through 2^x and a reciprocal of the special function
// unit (a few units of 2^-23, relative, over the range where the result is not 0
// or 1 in fp32), without the scaling that subnormal arguments would need: they
// give 1 and infinity here. gelu_tanh uses 0.5 (1 + tanh(u)) = 1 / (1 + e^(-2u)),
// which loses nothing where tanh is near -1. gelu's normal distribution function
// is erfcf's.
#pragma once

#include <cuda_fp16.h>

#include "device_common.cuh"

namespace mo {

constexpr float kGeluA = 1.5957691216057308f;   // 2 sqrt(2 / pi)
constexpr float kGeluB = 0.044715f;

__device__ __forceinline__ float exp2_fast(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ float reciprocal_fast(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
constexpr float kLog2E = 1.4426950408889634f;

// 1 / (1 + 2^-x): 0 where 2^-x is infinite
__device__ __forceinline__ float logistic2(float x) { return reciprocal_fast(1.0f + exp2_fast(-x)); }

// max(x, -3.4e38), NaN if x is: times 0, where it was -infinity, it gives -0
__device__ __forceinline__ float bounded(float x) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(x), "f"(-3.402823466e38f));
  return r;
}

__device__ __forceinline__ float normal_cdf(float x) { return 0.5f * erfcf(x * -0.70710678118654752f); }

// act(x)
template <int ACT>
__device__ __forceinline__ float act_value(float x) {
  if constexpr (ACT == MO_ACT_RELU) return x > 0.0f ? x : (x != x ? x : 0.0f);
  if constexpr (ACT == MO_ACT_GELU) return bounded(x) * normal_cdf(x);
  // the exponent is x (A + A B x^2) log2(e)
  if constexpr (ACT == MO_ACT_GELU_TANH)
    return bounded(x) * logistic2(x * fmaf(kGeluA * kGeluB * kLog2E, x * x, kGeluA * kLog2E));
  if constexpr (ACT == MO_ACT_SILU) return bounded(x) * logistic2(x * kLog2E);
  return x;
}

// x between -96 and 96, where what the slopes are made of is 0 or 1 to fp32 (or
// below 2^-126); NaN if x is
__device__ __forceinline__ float clamped(float x) {
  float r;
  asm("{\n\t.reg .f32 t;\n\tmax.NaN.f32 t, %1, %2;\n\tmin.NaN.f32 %0, t, %3;\n\t}" : "=f"(r) : "f"(x), "f"(-96.0f), "f"(96.0f));
  return r;
}

// act'(x), and act(x) in *value
template <int ACT>
__device__ __forceinline__ float act_slope(float x, float* value) {
  if constexpr (ACT == MO_ACT_RELU) {
    *value = x > 0.0f ? x : (x != x ? x : 0.0f);
    return x > 0.0f ? 1.0f : (x != x ? x : 0.0f);
  }
  if constexpr (ACT == MO_ACT_GELU) {
    const float c = normal_cdf(x);
    *value = bounded(x) * c;
    // x e^(-x^2 / 2) is 0 in fp32 from |x| = 15 on (and infinity times 0 is not a number)
    const float t = fabsf(x) < 16.0f ? x * exp2_fast(-0.5f * kLog2E * x * x) : (x != x ? x : 0.0f);
    return fmaf(0.3989422804014327f, t, c);
  }
  if constexpr (ACT == MO_ACT_GELU_TANH) {
    const float y = clamped(x), y2 = y * y;   // all 0 or 1 beyond
    const float s = logistic2(y * fmaf(kGeluA * kGeluB * kLog2E, y2, kGeluA * kLog2E));
    *value = bounded(x) * s;
    return fmaf(fmaf(-s, s, s) * y, fmaf(3.0f * kGeluA * kGeluB, y2, kGeluA), s);
  }
  if constexpr (ACT == MO_ACT_SILU) {
    const float y = clamped(x);
    const float s = logistic2(y * kLog2E);
    *value = bounded(x) * s;
    return fmaf(fmaf(-s, s, s), y, s);
  }
  *value = x;
  return 1.0f;
}

// Calls f(Act<ACT>()) for a run-time activation.
template <int ACT>
struct Act {
  static constexpr int value = ACT;
};
template <typename F>
__device__ __forceinline__ void with_act(int act, F&& f) {
  switch (act) {
    case MO_ACT_RELU: f(Act<MO_ACT_RELU>()); break;
    case MO_ACT_GELU: f(Act<MO_ACT_GELU>()); break;
    case MO_ACT_GELU_TANH: f(Act<MO_ACT_GELU_TANH>()); break;
    case MO_ACT_SILU: f(Act<MO_ACT_SILU>()); break;
    default: f(Act<MO_ACT_NONE>()); break;
  }
}

// ---------------------------------------------------------------- 8-bit blocks
// max(a, |b|, |c|), NaN if any is.
__device__ __forceinline__ float top3(float a, float b, float c) {
  float r;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(fabsf(b)), "f"(fabsf(c)));
  return r;
}
__device__ __forceinline__ float top2(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// Scale of a block with largest magnitude `top`: the least e + 127 >= 0 with
// top <= 448 2^e. 448 = 1.75 2^8: the exponent of the maximum less eight, one
// more where its mantissa exceeds 1.75. Infinity and NaN: 255, not a number.
__device__ __forceinline__ uint32_t mx8_scale(float top) {
  const uint32_t b = __float_as_uint(top) & 0x7FFFFFFFu;
  const int e = int(b >> 23) - 8 + ((b & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  return b >= 0x7F800000u ? 0xFFu : uint32_t(max(e, 0));
}
// 2^-e, by which the elements are multiplied before they are rounded
__device__ __forceinline__ float mx8_down(uint32_t scale) { return __uint_as_float((254u - min(scale, 253u)) << 23); }
// 2^e (2^-127 is subnormal; 255 is NaN)
__device__ __forceinline__ float mx8_up(uint32_t scale) {
  return __uint_as_float(scale == 0u ? 1u << 22 : scale == 255u ? 0x7FC00000u : scale << 23);
}

// Two values to e4m3 (to nearest, ties to even), the first in the low byte.
__device__ __forceinline__ uint32_t cvt_e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint32_t cvt_e4m3x4(float a, float b, float c, float d) {
  return cvt_e4m3x2(a, b) | (cvt_e4m3x2(c, d) << 16);
}
// Four codes of a word
__device__ __forceinline__ void e4m3x4_values(uint32_t w, float (&v)[4]) {
  uint32_t lo, hi;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(lo) : "h"(uint16_t(w)));
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(hi) : "h"(uint16_t(w >> 16)));
  const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&lo));
  const float2 b = __half22float2(*reinterpret_cast<const __half2*>(&hi));
  v[0] = a.x;
  v[1] = a.y;
  v[2] = b.x;
  v[3] = b.y;
}
__device__ __forceinline__ float e4m3_value(uint8_t c) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(uint16_t(c)));
  return __half2float(__ushort_as_half(uint16_t(h)));
}

// Eight consecutive elements of 16-byte aligned rows, as fp32.
__device__ __forceinline__ void load8(const uint16_t* p, float (&v)[8]) {
  const uint4 w = *reinterpret_cast<const uint4*>(p);
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(u[i] << 16);
    v[2 * i + 1] = __uint_as_float(u[i] & 0xFFFF0000u);
  }
}
__device__ __forceinline__ void load8(const float* p, float (&v)[8]) {
  const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
  v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
  v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
}
__device__ __forceinline__ void store8(uint16_t* p, const float (&v)[8]) {
  *reinterpret_cast<uint4*>(p) =
      make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
}
__device__ __forceinline__ void store8(float* p, const float (&v)[8]) {
  reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
  reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
}
__device__ __forceinline__ float load1(const uint16_t* p) { return bf16_bits_to_float(*p); }
__device__ __forceinline__ float load1(const float* p) { return *p; }
__device__ __forceinline__ void store1(uint16_t* p, float v) { *p = float_to_bf16_bits(v); }
__device__ __forceinline__ void store1(float* p, float v) { *p = v; }

}  // namespace mo
