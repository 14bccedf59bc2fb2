// Activations and their derivatives in fp32, and the 8-bit block format
// (e4m3 codes, a power of two for each 32 elements of a row).
//
// Functions take one number or a pair (ptx::F2), which costs one instruction for
// both wherever it is a product or a sum: an epilogue of 32768 elements a tile has
// to end within the products of the next tile.
//
// Logistic functions go through 2^x and a reciprocal of the special function
// unit (a few units of 2^-23, relative, over the range where the result is not 0
// or 1 in fp32), without the scaling that subnormal arguments would need: they
// give 1 and infinity here. gelu_tanh uses 0.5 (1 + tanh(u)) = 1 / (1 + e^(-2u)),
// which loses nothing where tanh is near -1.
//
// gelu's normal distribution function: Phi(-x) = e^(-x^2 / 2) R(x), x >= 0, where
// R(x) = Phi(-x) e^(x^2 / 2) falls from 1/2 as 1 / x does. R is t times a polynomial of
// degree 7 in t = 1 / (1 + 0.3 x), fitted here to R in double precision for the least
// relative error on [0, 14] (weighted least squares, the weights raised where the error
// is largest): 1.6e-7 with the coefficients below. So gelu keeps its relative accuracy in
// the left tail, down to where e^(-x^2 / 2) is 0 in fp32. (Abramowitz and Stegun 7.1.26,
// which is as exact beside 1, is 5e-5 of the value off at -3 and 1e-2 at -8.)
#pragma once

#include <cuda_fp16.h>

#include "device_common.cuh"
#include "ptx_train.cuh"

namespace mo {

using ptx::F2;

__device__ __forceinline__ float mul2(float a, float b) { return a * b; }
__device__ __forceinline__ float add2(float a, float b) { return a + b; }
__device__ __forceinline__ float fma2(float a, float b, float c) { return fmaf(a, b, c); }
using ptx::add2;
using ptx::fma2;
using ptx::mul2;

// A number in both places
template <typename N>
__device__ __forceinline__ N both(float x) {
  if constexpr (sizeof(N) == 8)
    return ptx::f2(x);
  else
    return x;
}
// f of each
template <typename F>
__device__ __forceinline__ float each(float x, F&& f) { return f(x); }
template <typename F>
__device__ __forceinline__ F2 each(F2 x, F&& f) {
  const float2 p = ptx::parts(x);
  return ptx::f2(f(p.x), f(p.y));
}
template <typename F>
__device__ __forceinline__ float each(float x, float y, F&& f) { return f(x, y); }
template <typename F>
__device__ __forceinline__ F2 each(F2 x, F2 y, F&& f) {
  const float2 p = ptx::parts(x), q = ptx::parts(y);
  return ptx::f2(f(p.x, q.x), f(p.y, q.y));
}

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
// max(x, -3.4e38), NaN if x is: times 0, where it was -infinity, it gives -0
__device__ __forceinline__ float bounded(float x) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(x), "f"(-3.402823466e38f));
  return r;
}
// x between -96 and 96, where what the slopes are made of is 0 or 1 to fp32 (or
// below 2^-126); NaN if x is
__device__ __forceinline__ float clamped(float x) {
  float r;
  asm("{\n\t.reg .f32 t;\n\tmax.NaN.f32 t, %1, %2;\n\tmin.NaN.f32 %0, t, %3;\n\t}" : "=f"(r) : "f"(x), "f"(-96.0f), "f"(96.0f));
  return r;
}

constexpr float kLog2E = 1.4426950408889634f;
constexpr float kGeluA = 1.5957691216057308f;   // 2 sqrt(2 / pi)
constexpr float kGeluB = 0.044715f;

// 1 / (1 + 2^x): 0 where 2^x is infinite
template <typename N>
__device__ __forceinline__ N logistic_of(N x) {
  return each(add2(each(x, exp2_fast), both<N>(1.0f)), reciprocal_fast);
}

// Phi(x), and e^(-x^2 / 2) in *bell
template <typename N>
__device__ __forceinline__ N normal_cdf(N x, N* bell) {
  const N e = each(mul2(mul2(x, x), both<N>(-0.5f * kLog2E)), exp2_fast);
  const N t = each(each(x, [](float v) { return fmaf(0.3f, fabsf(v), 1.0f); }), reciprocal_fast);
  N q = fma2(t, both<N>(0.035674572f), both<N>(-0.15720221f));
  q = fma2(t, q, both<N>(0.206352f));
  q = fma2(t, q, both<N>(-0.053682234f));
  q = fma2(t, q, both<N>(0.12856087f));
  q = fma2(t, q, both<N>(0.099913724f));
  q = fma2(t, q, both<N>(0.12075392f));
  q = fma2(t, q, both<N>(0.1196293f));
  const N tail = mul2(mul2(t, q), e);   // Phi(-|x|)
  *bell = e;
  return each(x, tail, [](float v, float h) { return v >= 0.0f ? 1.0f - h : h; });
}

// act(x)
template <int ACT, typename N>
__device__ __forceinline__ N act_value(N x) {
  if constexpr (ACT == MO_ACT_NONE) {
    return x;
  } else if constexpr (ACT == MO_ACT_RELU) {
    return each(x, [](float v) {
      float r;
      asm("max.NaN.f32 %0, %1, 0f00000000;" : "=f"(r) : "f"(v));
      return r;
    });
  } else {
    const N y = each(x, bounded);
    if constexpr (ACT == MO_ACT_GELU) {
      N bell;
      return mul2(y, normal_cdf(x, &bell));
    } else if constexpr (ACT == MO_ACT_GELU_TANH) {
      // the exponent is -x (A + A B x^2) log2(e)
      const N u = mul2(x, fma2(mul2(x, x), both<N>(-kGeluA * kGeluB * kLog2E), both<N>(-kGeluA * kLog2E)));
      return mul2(y, logistic_of(u));
    } else {
      return mul2(y, logistic_of(mul2(x, both<N>(-kLog2E))));
    }
  }
}

// act'(x), and act(x) in *value
template <int ACT, typename N>
__device__ __forceinline__ N act_slope(N x, N* value) {
  if constexpr (ACT == MO_ACT_NONE) {
    *value = x;
    return both<N>(1.0f);
  } else if constexpr (ACT == MO_ACT_RELU) {
    *value = act_value<ACT>(x);
    return each(x, [](float v) { return v > 0.0f ? 1.0f : (v != v ? v : 0.0f); });
  } else {
    const N z = each(x, bounded), y = each(x, clamped);
    if constexpr (ACT == MO_ACT_GELU) {
      N bell;
      const N c = normal_cdf(y, &bell);
      *value = mul2(z, c);
      return fma2(mul2(y, both<N>(0.3989422804f)), bell, c);   // (e^(-y^2 / 2) is 0 long before y is clamped)
    } else if constexpr (ACT == MO_ACT_GELU_TANH) {
      const N q = mul2(y, y);
      const N s = logistic_of(mul2(y, fma2(q, both<N>(-kGeluA * kGeluB * kLog2E), both<N>(-kGeluA * kLog2E))));
      *value = mul2(z, s);
      const N d = mul2(s, fma2(s, both<N>(-1.0f), both<N>(1.0f)));   // s (1 - s)
      return fma2(mul2(d, y), fma2(q, both<N>(3.0f * kGeluA * kGeluB), both<N>(kGeluA)), s);
    } else {
      const N s = logistic_of(mul2(y, both<N>(-kLog2E)));
      *value = mul2(z, s);
      return fma2(mul2(s, fma2(s, both<N>(-1.0f), both<N>(1.0f))), y, s);
    }
  }
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
