// Element types of the feed-forward operators' inputs and outputs (fp32,
// fp16, bf16; arithmetic is fp32 everywhere) and the activation functions.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/sherry.h"

namespace sherry {

typedef _Float16 h4 __attribute__((ext_vector_type(4)));
typedef __bf16 b4 __attribute__((ext_vector_type(4)));
typedef float f4 __attribute__((ext_vector_type(4)));

__host__ __device__ constexpr int dtype_bytes(int dtype) { return dtype == SHERRY_F32 ? 4 : 2; }

// Four consecutive elements as fp32, and back with one rounding to nearest
// even.  p is aligned to four elements.
template <typename T>
__device__ __forceinline__ f4 load4(const T* p) {
  if constexpr (sizeof(T) == 4) {
    return *reinterpret_cast<const f4*>(p);
  } else {
    typedef T v4 __attribute__((ext_vector_type(4)));
    return __builtin_convertvector(*reinterpret_cast<const v4*>(p), f4);
  }
}

template <typename T>
__device__ __forceinline__ void store4(T* p, f4 v) {
  if constexpr (sizeof(T) == 4) {
    *reinterpret_cast<f4*>(p) = v;
  } else {
    typedef T v4 __attribute__((ext_vector_type(4)));
    *reinterpret_cast<v4*>(p) = __builtin_convertvector(v, v4);
  }
}

// The same with the type known at run time (the branches are wave-uniform).
// Loading and converting are apart, so that several loads can be issued
// before the first conversion waits for one.
typedef unsigned int u4 __attribute__((ext_vector_type(4)));

__device__ __forceinline__ u4 load4_raw(const void* p, size_t i, int dtype) {
  if (dtype == SHERRY_F32) return *reinterpret_cast<const u4*>(static_cast<const float*>(p) + i);
  const uint2 v = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(p) + i);
  return u4{v.x, v.y, 0u, 0u};
}

__device__ __forceinline__ f4 as_f4(u4 v, int dtype) {
  if (dtype == SHERRY_F32) return __builtin_bit_cast(f4, v);
  const uint2 h = make_uint2(v.x, v.y);
  if (dtype == SHERRY_F16) return __builtin_convertvector(__builtin_bit_cast(h4, h), f4);
  return f4{__builtin_bit_cast(float, h.x << 16), __builtin_bit_cast(float, h.x & 0xFFFF0000u),
            __builtin_bit_cast(float, h.y << 16), __builtin_bit_cast(float, h.y & 0xFFFF0000u)};
}

__device__ __forceinline__ f4 load4_as(const void* p, size_t i, int dtype) {
  return as_f4(load4_raw(p, i, dtype), dtype);
}

__device__ __forceinline__ void store4_as(void* p, size_t i, int dtype, f4 v) {
  if (dtype == SHERRY_F32) store4(static_cast<float*>(p) + i, v);
  else if (dtype == SHERRY_F16) store4(static_cast<_Float16*>(p) + i, v);
  else store4(static_cast<__bf16*>(p) + i, v);
}

__device__ __forceinline__ uint32_t load1_raw(const void* p, size_t i, int dtype) {
  if (dtype == SHERRY_F32) return static_cast<const uint32_t*>(p)[i];
  return static_cast<const uint16_t*>(p)[i];
}

__device__ __forceinline__ float as_f1(uint32_t v, int dtype) {
  if (dtype == SHERRY_F32) return __builtin_bit_cast(float, v);
  if (dtype == SHERRY_F16) return (float)__builtin_bit_cast(_Float16, (uint16_t)v);
  return __builtin_bit_cast(float, v << 16);
}

__device__ __forceinline__ void store1_as(void* p, size_t i, int dtype, float v) {
  if (dtype == SHERRY_F32) static_cast<float*>(p)[i] = v;
  else if (dtype == SHERRY_F16) static_cast<_Float16*>(p)[i] = (_Float16)v;
  else static_cast<__bf16*>(p)[i] = (__bf16)v;
}

// Activation functions and their slopes in fp32 (SHERRY_ACT_*; the switch is
// wave-uniform).  With the logistic function S(t) = 1 / (1 + e^-t):
// silu(z) = z S(z); gelu(z) = z Phi(z), Phi the normal distribution function;
// gelu_tanh replaces Phi by (1 + tanh u) / 2 = S(2 u), u = sqrt(2 / pi) (z +
// 0.044715 z^3); relu2 is relu squared.
constexpr float kSqrtHalf = 0.70710678118654752f;
constexpr float kInvSqrt2Pi = 0.39894228040143268f;
constexpr float k2Sqrt2OverPi = 1.5957691216057308f;
constexpr float kGeluCubic = 0.044715f;
constexpr float kLog2E = 1.4426950408889634f;

// S(t) from the hardware's 2^x and reciprocal (each within an ulp).  The
// rounding of t log2(e) costs |t| / 2 ulp of e^-t, which matters only where
// S(t) ~ e^t is small: there t S(t), which is what multiplies it, is too.
// (The library's expf and a division took twice the instructions of the
// rest of the backward's epilogue.)
__device__ __forceinline__ float logistic(float t) {
  return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-kLog2E * t));
}

// Phi(z) from e = exp(-z^2 / 2): erfc(x) = P(t) exp(-x^2), t = 1 / (1 + p x), for
// x = |z| / sqrt(2) >= 0, the five-term form of Abramowitz and Stegun 7.1.26
// (|error| <= 1.5e-7, 7.5e-8 in Phi), with 1/2 and 1/sqrt(2) taken into the
// constants.  e is what the slope needs too; the library's erff took several
// times the instructions.
__device__ __forceinline__ float normal_cdf(float z, float e) {
  const float t = __builtin_amdgcn_rcpf(fmaf(0.3275911f * kSqrtHalf, fabsf(z), 1.0f));
  float p = fmaf(t, 0.5f * 1.061405429f, 0.5f * -1.453152027f);
  p = fmaf(t, p, 0.5f * 1.421413741f);
  p = fmaf(t, p, 0.5f * -0.284496736f);
  p = fmaf(t, p, 0.5f * 0.254829592f);
  const float tail = t * p * e;   // Phi(-|z|)
  return z < 0.0f ? tail : 1.0f - tail;
}

// The activation of z and, with kSlope, its slope there.
template <bool kSlope>
__device__ __forceinline__ float activate(float z, int act, float& slope) {
  switch (act) {
    case SHERRY_ACT_RELU:
      if constexpr (kSlope) slope = z > 0.0f ? 1.0f : 0.0f;
      return z > 0.0f || z != z ? z : 0.0f;
    case SHERRY_ACT_RELU2:
      if constexpr (kSlope) slope = z > 0.0f ? 2.0f * z : 0.0f;
      return z > 0.0f || z != z ? z * z : 0.0f;
    case SHERRY_ACT_SILU: {
      const float s = logistic(z);
      if constexpr (kSlope) slope = s + z * s * (1.0f - s);
      return z * s;
    }
    case SHERRY_ACT_GELU: {
      const float e = __builtin_amdgcn_exp2f(-0.5f * kLog2E * z * z);
      const float phi = normal_cdf(z, e);
      if constexpr (kSlope) slope = phi + z * (kInvSqrt2Pi * e);
      return z * phi;
    }
    case SHERRY_ACT_GELU_TANH: {
      // (beyond 11 S is 0, or 1 and 1 - S 0, in fp32, whatever z^2 is, so long as
      // it stays finite: 0 times an infinite z^2 is none)
      const float z2 = fminf(z * z, 1e6f);
      const float s = logistic(k2Sqrt2OverPi * (z + kGeluCubic * z2 * z));
      if constexpr (kSlope) slope = s + z * s * (1.0f - s) * k2Sqrt2OverPi * (1.0f + 3.0f * kGeluCubic * z2);
      return z * s;
    }
    default:
      if constexpr (kSlope) slope = 1.0f;
      return z;
  }
}

__device__ __forceinline__ float act_value(float z, int act) {
  float slope;
  return activate<false>(z, act, slope);
}

// Sum over the 64 lanes of a wave, the same value in every lane (all lanes
// active), by the DPP steps of wave_max.
template <int CTRL>
__device__ __forceinline__ float dpp_shift(float x) {
  return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(__builtin_bit_cast(int, x),
                                                               __builtin_bit_cast(int, x), CTRL, 0xF,
                                                               0xF, false));
}

// Maximum over the 16 lanes of a row, in every lane.
__device__ __forceinline__ float row16_max(float v) {
  v = fmaxf(v, dpp_shift<0xB1>(v));
  v = fmaxf(v, dpp_shift<0x4E>(v));
  v = fmaxf(v, dpp_shift<0x124>(v));
  return fmaxf(v, dpp_shift<0x128>(v));
}

__device__ __forceinline__ float wave_sum(float v) {
  v += dpp_shift<0xB1>(v);     // quad_perm [1,0,3,2]
  v += dpp_shift<0x4E>(v);     // quad_perm [2,3,0,1]
  v += dpp_shift<0x124>(v);    // row_ror:4
  v += dpp_shift<0x128>(v);    // row_ror:8
  const int u = __builtin_bit_cast(int, v);
  const float r0 = __builtin_bit_cast(float, __builtin_amdgcn_readlane(u, 0));
  const float r1 = __builtin_bit_cast(float, __builtin_amdgcn_readlane(u, 16));
  const float r2 = __builtin_bit_cast(float, __builtin_amdgcn_readlane(u, 32));
  const float r3 = __builtin_bit_cast(float, __builtin_amdgcn_readlane(u, 48));
  return (r0 + r1) + (r2 + r3);
}

}  // namespace sherry
