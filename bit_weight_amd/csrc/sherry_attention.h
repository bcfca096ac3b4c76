// What the two attention kernels over the 8-bit cache share: steps of 64 tokens,
// what a tile of queries sees of them, and 8-bit values as fp16.
#pragma once

#include "sherry_cache.h"

namespace sherry {

typedef _Float16 h8 __attribute__((ext_vector_type(8)));
typedef _Float16 h2 __attribute__((ext_vector_type(2)));

constexpr int kStep = 64;                // tokens
constexpr float kSlack = 8.0f;           // a running maximum is kept until it is passed by this (of base 2)
constexpr float kWeightExponent = 7.0f;  // weights e^(s - m) as operands are 2^7 as large: with the slack below 2^15
constexpr float kLn2 = 0.69314718055994531f;

// A value that every lane has alike, as one the compiler knows to be.
__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }
__device__ __forceinline__ int64_t uniform64(int64_t v) {
  return ((int64_t)uniform((int)(v >> 32)) << 32) | (uint32_t)uniform((int)(uint32_t)v);
}
__device__ __forceinline__ Rows uniform(Rows r) { return {uniform(r.row0), uniform(r.n), uniform(r.len)}; }

__device__ __forceinline__ int room_of(const AttentionArgs& a) { return a.c.table_width << (a.c.block_shift + 4); }

// Steps that queries at positions low .. high of a sequence look at: those of its
// first tokens, then those from the window's on.
struct Steps {
  int head, from, to;
  __device__ __forceinline__ Steps(const AttentionArgs& a, int low, int high) {
    head = from = 0;
    to = min(max(high, 0), room_of(a) - 1) / kStep + 1;     // (a sequence longer than its table gives NaN whatever it looks at)
    if (a.window > 0) {
      from = min(max(low - a.window + 1, 0) / kStep, to - 1);
      head = min((a.sinks + kStep - 1) / kStep, from);
    }
  }
  __device__ __forceinline__ int count() const { return head + to - from; }
  __device__ __forceinline__ int at(int s) const { return s < head ? s : from + s - head; }
};

// Quotients of numbers that are as a rule small: a division in 64 bits is 130 instructions.
__device__ __forceinline__ int64_t quotient(int64_t x, int y) {
  return (uint64_t)x >> 32 ? x / y : (int64_t)((uint32_t)x / (uint32_t)y);
}

// Whether every query at low .. high sees every token of a step, and whether the
// one at p sees token t.
__device__ __forceinline__ bool sees_all(const AttentionArgs& a, int t0, int low, int high) {
  return t0 + kStep - 1 <= low && (a.window == 0 || high - t0 < a.window || t0 + kStep <= a.sinks);
}

__device__ __forceinline__ bool sees(const AttentionArgs& a, int t, int p) {
  return t <= p && (a.window == 0 || p - t < a.window || t < a.sinks);
}

__device__ __forceinline__ float above(float m) { return m == -__builtin_inff() ? 0.0f : m; }

// Four 8-bit values as fp16: 1024 + (q + 128) is 0x6400 with the byte in its low half.
__device__ __forceinline__ void halves4(uint32_t w, h2& a, h2& b) {
  const h2 off = {(_Float16)-1152.0f, (_Float16)-1152.0f};
  w ^= 0x80808080u;
  a = __builtin_bit_cast(h2, __builtin_amdgcn_perm(0x64646464u, w, 0x04010400u)) + off;
  b = __builtin_bit_cast(h2, __builtin_amdgcn_perm(0x64646464u, w, 0x04030402u)) + off;
}

__device__ __forceinline__ h8 halves8(uint32_t x, uint32_t y) {
  h2 a, b, c, d;
  halves4(x, a, b);
  halves4(y, c, d);
  return h8{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}

// The power of two under which a row whose largest |q| is `top` becomes fp16: the largest near 2^13.
__device__ __forceinline__ float row_scale(float top) {
  const int e = (int)(__builtin_bit_cast(uint32_t, top) >> 23) - 127;      // 2^e <= top < 2^(e + 1)
  const int up = top > 0.0f && top < __builtin_inff() ? min(13 - e, 126) : 0;
  return __builtin_bit_cast(float, (uint32_t)(max(up, -126) + 127) << 23);
}

// 4 n consecutive values, all asked for before one is looked at (a branch on the type
// for each four would wait for each).
template <int n>
struct RawValues {
  u4 raw[n];
  __device__ __forceinline__ void load(const void* p, size_t at, int dtype) {
    if (dtype == SHERRY_F32) {
#pragma unroll
      for (int j = 0; j < n; ++j) raw[j] = reinterpret_cast<const u4*>(static_cast<const float*>(p) + at)[j];
    } else {
#pragma unroll
      for (int j = 0; j < n / 2; ++j) raw[j] = reinterpret_cast<const u4*>(static_cast<const uint16_t*>(p) + at)[j];
    }
  }
  __device__ __forceinline__ f4 get(int j, int dtype) const {
    if (dtype == SHERRY_F32) return __builtin_bit_cast(f4, raw[j]);
    const u4 w = raw[j / 2];
    return as_f4(j % 2 ? u4{w.z, w.w, 0u, 0u} : u4{w.x, w.y, 0u, 0u}, dtype);
  }
};

// Long sequences' numbers across lanes.
__device__ __forceinline__ int64_t shfl_up64(int64_t v, int d) {
  const int lo = __shfl_up((int)(uint32_t)v, d), hi = __shfl_up((int)(v >> 32), d);
  return ((int64_t)hi << 32) | (uint32_t)lo;
}

// Sum over a workgroup of kWaves waves of v, with the sum over the threads before this one.
template <int kWaves>
__device__ __forceinline__ int64_t block_scan(int64_t v, int64_t& before, int64_t* parts) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  int64_t sum = v;
#pragma unroll
  for (int d = 1; d < 64; d *= 2) {
    const int64_t u = shfl_up64(sum, d);
    if (lane >= d) sum += u;
  }
  __syncthreads();
  if (lane == 63) parts[wave] = sum;
  __syncthreads();
  int64_t total = 0;
  before = sum - v;
#pragma unroll
  for (int w = 0; w < kWaves; ++w) {
    if (w < wave) before += parts[w];
    total += parts[w];
  }
  return total;
}

}  // namespace sherry
