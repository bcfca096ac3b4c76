// Layer norm over the K features of each token:
//   mean = sum x / K, var = sum (x - mean)^2 / K, rstd = 1 / sqrt(var + eps),
//   y = (x - mean) rstd w + b,
// its form that writes the int8 tokens the products take, and its gradients
//   g = dy w, xh = (x - mean) rstd,
//   dx = rstd (g - sum g / K - xh sum(g xh) / K),
//   dw = sum over tokens of dy xh, db = sum over tokens of dy.
// All of them stream their inputs once; memory bandwidth bounds them at many
// tokens (bf16, K = 4096: forward of 2048 tokens 33.6 MB in 8.1 us, 4.1 TB/s
// with its launch, 8192 tokens 4.9 TB/s; backward of 8192 tokens 201 MB in 42.6
// us, 4.7 TB/s with its second launch), the chain of load, reductions and
// launch at few (16 tokens of 8192 into int8: 5.6 us).
//
// A group of W waves holds one token in registers, so the mean and the sum of
// squared differences from it are taken in two passes without reading x
// again: the variance has no cancellation.  Lane l of the group takes
// features V (l + 64 W j) .. + V - 1: 16 bytes a load (8 where K is no
// multiple of 8 in a 16-bit type).  Groups go on to further tokens, the next
// one's loads in flight, and keep w (and b) in registers: read again for
// every token they are as many bytes as x and dy together.
#include "sherry_device.h"
#include "sherry_launch.h"
#include "sherry_types.h"

namespace sherry {
namespace {

constexpr int kLoopThreads = 1024;        // above kNormMaxK: one token per workgroup, in loops
// backward: 16 waves that share one token or more, or 8 with one each
constexpr int back_threads(int W) { return W == 1 ? 512 : 1024; }
constexpr int kNormMaxK = 16384;          // features held in registers
constexpr int kBackBlocks = kCUs;         // most workgroups (rows of partial weight gradients)

// Sum (or maximum) over the W waves that share a token; `slot` is this
// wave's place in `red`, whose W entries from the token's first on hold the
// waves' values.  Every wave of the workgroup calls it; two buffers used in
// turn need one barrier per call.
template <int W, typename T, typename F>
__device__ __forceinline__ T group_join(T v, T* red, int wave, F op) {
  if constexpr (W == 1) {
    return v;
  } else {
    if ((threadIdx.x & 63) == 0) red[wave] = v;
    __syncthreads();
    const int first = wave / W * W;
    T r = red[first];
#pragma unroll
    for (int i = 1; i < W; ++i) r = op(r, red[first + i]);
    return r;
  }
}

// A double from another lane of its 16-lane row by DPP control CTRL, and
// from one lane of the wave.
template <int CTRL>
__device__ __forceinline__ double dpp_shift(double x) {
  const uint64_t u = __builtin_bit_cast(uint64_t, x);
  const int lo = (int)(uint32_t)u, hi = (int)(uint32_t)(u >> 32);
  const uint32_t l = (uint32_t)__builtin_amdgcn_update_dpp(lo, lo, CTRL, 0xF, 0xF, false);
  const uint32_t h = (uint32_t)__builtin_amdgcn_update_dpp(hi, hi, CTRL, 0xF, 0xF, false);
  return __builtin_bit_cast(double, (uint64_t)h << 32 | l);
}

__device__ __forceinline__ double from_lane(double x, int lane) {
  const uint64_t u = __builtin_bit_cast(uint64_t, x);
  const uint32_t l = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)u, lane);
  const uint32_t h = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)(u >> 32), lane);
  return __builtin_bit_cast(double, (uint64_t)h << 32 | l);
}

// As wave_sum and wave_max (shuffles, six LDS round trips each, took longer).
template <typename F>
__device__ __forceinline__ double wave_join64(double v, F op) {
  v = op(v, dpp_shift<0xB1>(v));     // quad_perm [1,0,3,2]
  v = op(v, dpp_shift<0x4E>(v));     // quad_perm [2,3,0,1]
  v = op(v, dpp_shift<0x124>(v));    // row_ror:4
  v = op(v, dpp_shift<0x128>(v));    // row_ror:8
  return op(op(from_lane(v, 0), from_lane(v, 16)), op(from_lane(v, 32), from_lane(v, 48)));
}

__device__ __forceinline__ double wave_sum64(double v) {
  return wave_join64(v, [](double a, double b) { return a + b; });
}

__device__ __forceinline__ double wave_max64(double v) {
  return wave_join64(v, [](double a, double b) { return fmax(a, b); });
}

__device__ __forceinline__ double wave_total(double v) { return wave_sum64(v); }
__device__ __forceinline__ float wave_total(float v) { return wave_sum(v); }
__device__ __forceinline__ double wave_top(double v) { return wave_max64(v); }
__device__ __forceinline__ float wave_top(float v) { return wave_max(v); }

struct NormArgs {
  const void* x;
  const float* w;     // nullptr: ones
  const float* b;     // nullptr: zeros
  void* y;            // the type of x, or
  int8_t* q;          // int8 with
  float* s;           //   one scale per token
  float* mean;        // nullptr: not wanted
  float* rstd;
  float eps;
  int M, K;
};

// V consecutive features: as loaded, and as fp32.
template <typename T, int V>
using Raw = T __attribute__((ext_vector_type(V)));
template <int V>
using Vec = float __attribute__((ext_vector_type(V)));

template <typename T, int V>
__device__ __forceinline__ Raw<T, V> load_raw(const T* p, bool in) {
  Raw<T, V> r{};
  if (in) r = *reinterpret_cast<const Raw<T, V>*>(p);
  return r;
}

// One token's row as a buffer (n bytes; 0 for a token past the last), whose
// range check stands for the bounds: loads past it give zeros, stores nothing.
// (The check does not see a scalar offset: the whole offset is the lane's.)
__device__ __forceinline__ __amdgpu_buffer_rsrc_t row_of(const void* base, size_t at, int n) {
  return __builtin_amdgcn_make_buffer_rsrc(static_cast<char*>(const_cast<void*>(base)) + at, 0, n, 0x00020000);
}

template <typename T, int V>
__device__ __forceinline__ Raw<T, V> load_row(__amdgpu_buffer_rsrc_t r, int at) {
  if constexpr (sizeof(T) * V == 16) return __builtin_bit_cast(Raw<T, V>, __builtin_amdgcn_raw_buffer_load_b128(r, at, 0, 0));
  else return __builtin_bit_cast(Raw<T, V>, __builtin_amdgcn_raw_buffer_load_b64(r, at, 0, 0));
}

template <typename T, int V>
__device__ __forceinline__ void store_row(__amdgpu_buffer_rsrc_t r, int at, Raw<T, V> v) {
  typedef unsigned int v4u __attribute__((ext_vector_type(4)));
  typedef unsigned int v2u __attribute__((ext_vector_type(2)));
  if constexpr (sizeof(T) * V == 16) __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(v4u, v), r, at, 0, 0);
  else __builtin_amdgcn_raw_buffer_store_b64(__builtin_bit_cast(v2u, v), r, at, 0, 0);
}

template <int V>
__device__ __forceinline__ Vec<V> load_vec(const float* p, bool in, float otherwise) {
  Vec<V> r;
#pragma unroll
  for (int i = 0; i < V; i += 4) {
    const f4 v = in ? load4(p + i) : f4{otherwise, otherwise, otherwise, otherwise};
#pragma unroll
    for (int c = 0; c < 4; ++c) r[i + c] = v[c];
  }
  return r;
}

// y = (d rstd) w + b of four features, in type S.
template <typename S>
__device__ __forceinline__ void normed4(const S (&d)[4], S rstd, const NormArgs& a, int k, S (&v)[4]) {
  const f4 w = a.w ? load4(a.w + k) : f4{1.0f, 1.0f, 1.0f, 1.0f};
  const f4 b = a.b ? load4(a.b + k) : f4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = d[i] * rstd * (S)w[i] + (S)b[i];
}

// A token with a value that is not finite has no scale: s = NaN, so that every
// product of it is NaN, and steps without a meaning.  Its largest |v| is made
// infinite here (a maximum passes over NaN): a feature that is not finite leaves
// no finite spread, which is looked at once a token, and a lane with a weight
// or bias that is not takes 0 and infinity for its first ones.
constexpr double kNoScale = __builtin_inf();
__device__ __forceinline__ float scale_of(double amax) {
  if (amax == kNoScale) return __builtin_nanf("");
  const float s = (float)(amax / 127.0);
  return s > 0.0f ? s : 1.0f;
}

// Four int8 step counts in a word: rounded half to even by an addition that
// leaves no bits behind the point, clamped.
__device__ __forceinline__ int quant_at(double t) {
  const int n = (int)(uint32_t)__builtin_bit_cast(uint64_t, t + 0x1.8p52);
  return n < -127 ? -127 : n > 127 ? 127 : n;
}
__device__ __forceinline__ uint32_t quant4(double t0, double t1, double t2, double t3) {
  const uint32_t lo = __builtin_amdgcn_perm((uint32_t)quant_at(t1), (uint32_t)quant_at(t0), 0x0C0C0400u);
  const uint32_t hi = __builtin_amdgcn_perm((uint32_t)quant_at(t3), (uint32_t)quant_at(t2), 0x04000C0Cu);
  return lo | hi;
}

__device__ __forceinline__ float inverse_root(float v) { return 1.0f / sqrtf(v); }
// Newton's steps y + y (1 - v y^2) / 2 from the hardware's estimate.
__device__ __forceinline__ double inverse_root(double v) {
  double y = __builtin_amdgcn_rsq(v);
  y += 0.5 * y * (1.0 - v * y * y);
  y += 0.5 * y * (1.0 - v * y * y);
  return y;
}

// The forward on tokens that fit registers.  Q: int8 output; then everything
// from the mean on is computed in 64 bits, so that a value next to a border
// between two int8 steps falls where exact arithmetic puts it (in 32 bits
// about one value in 1e5 lands on the other side); S is the sums' type.  A
// 64-bit operation issues as fast as a 32-bit one, but a division is some 12
// of them and a rounding with its clamp 6, so the steps are counted by a
// product with 1 / s, rounded by one addition, and the two divisions by K and
// the root are products and Newton steps (8192 x 4096 bf16 48.6 -> 31.9 us, 16 x
// 8192 6.5 -> 5.6; the bytes take 19 and 0.2; with v in 32 bits and only
// what is next to a border in 64: 43).
template <typename T, int V, int W, int J, bool Q>
__global__ __launch_bounds__(W == 16 ? 1024 : 256) void norm_kernel(NormArgs a) {
  using S = std::conditional_t<Q, double, float>;
  constexpr int kThreads = W == 16 ? 1024 : 256;
  constexpr int G = kThreads / 64 / W;   // tokens at a time
  // w and b beside 16 features in 64 bits do not fit 128 registers
  constexpr bool kLds = Q && W == 16 && J * V == 16;
  __shared__ Vec<V> w_lds[kLds ? 64 * W * J : 1], b_lds[kLds ? 64 * W * J : 1];
  __shared__ S red[2][3][kThreads / 64];
  const int wave = threadIdx.x >> 6;
  const int lane = threadIdx.x % (64 * W);
  const auto add = [](S p, S q) { return p + q; };
  const auto top = [](S p, S q) { return p > q ? p : q; };
  const S inv_k = (S)1 / (S)a.K;
  auto over_k = [&](S t) { return Q ? t * inv_k : t / (S)a.K; };
  // the mean to the last bit, by one step on what the product leaves of the
  // sum: equal features then have no spread (K = 196: all ones were 2^-53 off
  // their mean, and that became the scale)
  auto mean_of = [&](S t) {
    const S m = over_k(t);
    return Q ? (S)fma(fma(-m, (S)a.K, t), inv_k, m) : m;
  };
  auto feature = [&](int j) { return V * (lane + 64 * W * j); };
  auto load = [&](int m, Raw<T, V> (&r)[J]) {
#pragma unroll
    for (int j = 0; j < J; ++j)
      r[j] = load_raw<T, V>(static_cast<const T*>(a.x) + (size_t)m * a.K + feature(j), m < a.M && feature(j) < a.K);
  };
  Raw<T, V> next[J];
  load(blockIdx.x * G + wave / W, next);
  Vec<V> w[kLds ? 1 : J], b[kLds ? 1 : J];
  float odd = 0.0f;   // NaN where a weight or bias is not finite
#pragma unroll
  for (int j = 0; j < J; ++j) {
    const Vec<V> wj = load_vec<V>(a.w + feature(j), a.w && feature(j) < a.K, 1.0f);
    const Vec<V> bj = load_vec<V>(a.b + feature(j), a.b && feature(j) < a.K, 0.0f);
    if constexpr (Q) {
#pragma unroll
      for (int i = 0; i < V; ++i) odd = fmaf(bj[i], 0.0f, fmaf(wj[i], 0.0f, odd));
    }
    if constexpr (kLds) {
      w_lds[lane + 64 * W * j] = wj;   // (read by this thread only)
      b_lds[lane + 64 * W * j] = bj;
    } else {
      w[j] = wj;
      b[j] = bj;
    }
  }
  if (Q && odd != 0.0f) {
    Vec<V>& w0 = kLds ? w_lds[lane] : w[0];
    Vec<V>& b0 = kLds ? b_lds[lane] : b[0];
    w0[0] = 0.0f;
    b0[0] = __builtin_inff();
  }
  // the same number of trips for every wave of the workgroup (barriers)
  int turn = 0;
  for (int m0 = blockIdx.x * G; m0 < a.M; m0 += gridDim.x * G, turn ^= 1) {
    const int m = m0 + wave / W;
    const bool live = m < a.M;
    Vec<V> xv[J];
#pragma unroll
    for (int j = 0; j < J; ++j) xv[j] = __builtin_convertvector(next[j], Vec<V>);
    if (m0 + (int)gridDim.x * G < a.M) load(m + gridDim.x * G, next);
    S sum = 0;
#pragma unroll
    for (int j = 0; j < J; ++j) {
      S part = 0;
#pragma unroll
      for (int i = 0; i < V; ++i) part += (S)xv[j][i];
      sum += part;
    }
    const S mean = mean_of(group_join<W>((S)wave_total(sum), red[turn][0], wave, add));
    S sq = 0;
#pragma unroll
    for (int j = 0; j < J; ++j) {
      if (feature(j) < a.K) {
#pragma unroll
        for (int i = 0; i < V; ++i) {
          const S d = (S)xv[j][i] - mean;
          sq += d * d;
        }
      }
    }
    const S var = over_k(group_join<W>((S)wave_total(sq), red[turn][1], wave, add));
    const S rstd = inverse_root(var + (S)a.eps);
    if (a.mean && live && lane == 0) {
      a.mean[m] = (float)mean;
      a.rstd[m] = (float)rstd;
    }
    S v[J][V];
#pragma unroll
    for (int j = 0; j < J; ++j) {
      const Vec<V> wj = kLds ? w_lds[lane + 64 * W * j] : w[kLds ? 0 : j];
      const Vec<V> bj = kLds ? b_lds[lane + 64 * W * j] : b[kLds ? 0 : j];
#pragma unroll
      for (int i = 0; i < V; ++i) v[j][i] = ((S)xv[j][i] - mean) * rstd * (S)wj[i] + (S)bj[i];
    }
    if constexpr (!Q) {
      T* y = static_cast<T*>(a.y) + (size_t)m * a.K;
#pragma unroll
      for (int j = 0; j < J; ++j) {
        Vec<V> o;
#pragma unroll
        for (int i = 0; i < V; ++i) o[i] = v[j][i];
        if (live && feature(j) < a.K)
          *reinterpret_cast<Raw<T, V>*>(y + feature(j)) = __builtin_convertvector(o, Raw<T, V>);
      }
    } else {
      S amax = 0;
#pragma unroll
      for (int j = 0; j < J; ++j) {
        if (feature(j) < a.K) {
#pragma unroll
          for (int i = 0; i < V; ++i) amax = fmax(amax, fabs(v[j][i]));
        }
      }
      if (!(var < kNoScale)) amax = kNoScale;   // a feature that is not finite: no finite spread
      amax = group_join<W>((S)wave_top(amax), red[turn][2], wave, top);
      // the scale is the fp32 the product reads; the steps are counted in it
      const float s = scale_of(amax);
      if (live && lane == 0) a.s[m] = s;
      const S inv = (S)1 / (S)s;
#pragma unroll
      for (int j = 0; j < J; ++j) {
        uint32_t q[V / 4];
#pragma unroll
        for (int i = 0; i < V; i += 4)
          q[i / 4] = quant4(v[j][i] * inv, v[j][i + 1] * inv, v[j][i + 2] * inv, v[j][i + 3] * inv);
        if (live && feature(j) < a.K) {
          uint32_t* out = reinterpret_cast<uint32_t*>(a.q + (size_t)m * a.K + feature(j));   // 4-byte aligned
#pragma unroll
          for (int i = 0; i < V / 4; ++i) out[i] = q[i];
        }
      }
    }
  }
}

// The forward on tokens of more than kNormMaxK features: one workgroup of 16
// waves per token, which reads the token again for each pass: from L2 while the
// tokens in work fit it (an XCD's 32 tokens in 4 MB: 64K features in 16 bits).
template <typename T, bool Q>
__global__ __launch_bounds__(kLoopThreads) void norm_loop_kernel(NormArgs a) {
  using S = std::conditional_t<Q, double, float>;
  constexpr int W = kLoopThreads / 64;
  __shared__ S red[3][W];
  const int wave = threadIdx.x >> 6;
  const int m = blockIdx.x;
  const T* x = static_cast<const T*>(a.x) + (size_t)m * a.K;
  const auto add = [](S p, S q) { return p + q; };
  const auto top = [](S p, S q) { return p > q ? p : q; };
  S sum = 0;
  for (int k = 4 * threadIdx.x; k < a.K; k += 4 * kLoopThreads) {
    const f4 v = load4(x + k);
    sum += ((S)v[0] + (S)v[1]) + ((S)v[2] + (S)v[3]);
  }
  const S mean = group_join<W>((S)wave_total(sum), red[0], wave, add) / (S)a.K;
  S sq = 0;
  for (int k = 4 * threadIdx.x; k < a.K; k += 4 * kLoopThreads) {
    const f4 v = load4(x + k);
#pragma unroll
    for (int i = 0; i < 4; ++i) sq += ((S)v[i] - mean) * ((S)v[i] - mean);
  }
  const S var = group_join<W>((S)wave_total(sq), red[1], wave, add) / (S)a.K;
  const S rstd = (S)1 / sqrt(var + (S)a.eps);
  if (a.mean && threadIdx.x == 0) {
    a.mean[m] = (float)mean;
    a.rstd[m] = (float)rstd;
  }
  auto value = [&](int k, S (&v)[4]) {
    const f4 xv = load4(x + k);
    const S d[4] = {xv[0] - mean, xv[1] - mean, xv[2] - mean, xv[3] - mean};
    normed4(d, rstd, a, k, v);
  };
  S v[4];
  if constexpr (!Q) {
    T* y = static_cast<T*>(a.y) + (size_t)m * a.K;
    for (int k = 4 * threadIdx.x; k < a.K; k += 4 * kLoopThreads) {
      value(k, v);
      store4(y + k, f4{v[0], v[1], v[2], v[3]});
    }
  } else {
    S amax = 0;
    bool none = false;
    for (int k = 4 * threadIdx.x; k < a.K; k += 4 * kLoopThreads) {
      value(k, v);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        amax = fmax(amax, fabs(v[i]));
        none |= v[i] != v[i];
      }
    }
    if (none) amax = kNoScale;
    amax = group_join<W>((S)wave_top(amax), red[2], wave, top);
    const float s = scale_of(amax);
    if (threadIdx.x == 0) a.s[m] = s;
    const S inv = (S)1 / (S)s;
    uint32_t* q = reinterpret_cast<uint32_t*>(a.q + (size_t)m * a.K);
    for (int k = 4 * threadIdx.x; k < a.K; k += 4 * kLoopThreads) {
      value(k, v);
      q[k / 4] = quant4(v[0] * inv, v[1] * inv, v[2] * inv, v[3] * inv);
    }
  }
}

struct NormBackArgs {
  const void* dy;
  const void* x;
  const float* mean;
  const float* rstd;
  const float* w;     // nullptr: ones
  void* dx;
  float* part;        // [blocks][2][K] partial dw, db
  int M, K;
};

// Gradients on tokens that fit registers, 16 features a lane.  A group of W
// waves takes tokens group, group + groups, ... and keeps its sums of dw and
// db over them in registers; the workgroup adds its groups through LDS at the
// end and writes one row of partial sums, so no atomics and a fixed order.
// One workgroup per CU: with two, the partial rows double (8192 x 4096 bf16:
// 52.3 against 47.1 us).  w waits in LDS and the rows are buffers with a scalar
// base, so 16 waves fit their 128 registers; 8 waves of 32 features a lane
// with w in registers and a pointer per load spilled (8192 x 4096 bf16 47.1 ->
// 42.6 us, fp32 4096 x 4096 80.6 -> 47.8, fp16 4096 x 8192 89.9 -> 46.5, fp32
// 2048 x 16384 182 -> 88.9).  Groups of one wave (K <= 1024) have few features a
// lane and join more groups: 8 of them (8192 x 1024 fp32 23 us, 16 of them 31).
template <typename T, int V, int W, int J>
__global__ __launch_bounds__(back_threads(W)) void norm_backward_kernel(NormBackArgs a) {
  constexpr int kThreads = back_threads(W), G = kThreads / 64 / W;
  __shared__ float2 red[2][kThreads / 64];
  __shared__ Vec<V> w[64 * W * J];
  __shared__ Vec<V> col[G > 1 ? G : 1][G > 1 ? 64 * W * J : 1];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);   // (the rows' addresses: scalar)
  const int lane = threadIdx.x % (64 * W);
  const int group = wave / W;
  const float inv_k = 1.0f / (float)a.K;
  auto feature = [&](int j) { return V * (lane + 64 * W * j); };
  constexpr int kChunk = V * (int)sizeof(T);
  const int bytes = a.K * (int)sizeof(T);   // of a row
  struct Token {
    Raw<T, V> x[J], dy[J];
    float mean, rstd;
  };
  auto load = [&](int m, Token& t) {
    const bool live = m < a.M;
    const size_t row = (size_t)m * bytes;
    const __amdgpu_buffer_rsrc_t rx = row_of(a.x, row, live ? bytes : 0), rdy = row_of(a.dy, row, live ? bytes : 0);
#pragma unroll
    for (int j = 0; j < J; ++j) {
      t.x[j] = load_row<T, V>(rx, kChunk * (lane + 64 * W * j));
      t.dy[j] = load_row<T, V>(rdy, kChunk * (lane + 64 * W * j));
    }
    t.mean = live ? a.mean[m] : 0.0f;
    t.rstd = live ? a.rstd[m] : 0.0f;
  };
  Token next;
  load(blockIdx.x * G + group, next);
  Vec<V> dw[J], db[J];
#pragma unroll
  for (int j = 0; j < J; ++j) dw[j] = db[j] = Vec<V>{};
  for (int i = threadIdx.x; i < 64 * W * J; i += kThreads)
    w[i] = load_vec<V>(a.w + V * i, a.w && V * i < a.K, 1.0f);
  __syncthreads();
  // every wave of the workgroup makes the same number of trips (barriers)
  int turn = 0;
  for (int m0 = blockIdx.x * G; m0 < a.M; m0 += gridDim.x * G, turn ^= 1) {
    const int m = m0 + group;
    const float mean = next.mean, rstd = next.rstd;
    Vec<V> xh[J], g[J];
#pragma unroll
    for (int j = 0; j < J; ++j) {
      xh[j] = __builtin_convertvector(next.x[j], Vec<V>);
      g[j] = __builtin_convertvector(next.dy[j], Vec<V>);
    }
    if (m0 + (int)gridDim.x * G < a.M) load(m + gridDim.x * G, next);
    asm volatile("" ::: "memory");   // w stays in LDS
    float s1 = 0.0f, s2 = 0.0f;
#pragma unroll
    for (int j = 0; j < J; ++j) {
      const bool in = feature(j) < a.K;   // past K: dy is 0, and xh is made 0
      const Vec<V> wj = w[lane + 64 * W * j];
#pragma unroll
      for (int i = 0; i < V; ++i) {
        xh[j][i] = in ? (xh[j][i] - mean) * rstd : 0.0f;
        dw[j][i] += g[j][i] * xh[j][i];
        db[j][i] += g[j][i];
        g[j][i] *= wj[i];
        s1 += g[j][i];
        s2 += g[j][i] * xh[j][i];
      }
    }
    s1 = wave_sum(s1);
    s2 = wave_sum(s2);
    if constexpr (W > 1) {
      if ((threadIdx.x & 63) == 0) red[turn][wave] = make_float2(s1, s2);
      __syncthreads();
      s1 = s2 = 0.0f;
#pragma unroll (W < 4 ? W : 4)
      for (int i = 0; i < W; ++i) {
        const float2 r = red[turn][group * W + i];
        s1 += r.x;
        s2 += r.y;
      }
    }
    s1 *= inv_k;
    s2 *= inv_k;
    const __amdgpu_buffer_rsrc_t rdx = row_of(a.dx, (size_t)m * bytes, m < a.M ? bytes : 0);
#pragma unroll
    for (int j = 0; j < J; ++j) {
      Vec<V> v;
#pragma unroll
      for (int i = 0; i < V; ++i) v[i] = rstd * (g[j][i] - s1 - xh[j][i] * s2);
      store_row<T, V>(rdx, kChunk * (lane + 64 * W * j), __builtin_convertvector(v, Raw<T, V>));
    }
  }
  // the groups' sums of each column, joined through LDS in the groups' order
  float* part = a.part + (size_t)blockIdx.x * 2 * a.K;
  auto put = [&](int which, int k, Vec<V> t) {
#pragma unroll
    for (int i = 0; i < V; i += 4)
      store4(part + (size_t)which * a.K + k + i, f4{t[i], t[i + 1], t[i + 2], t[i + 3]});
  };
#pragma unroll
  for (int which = 0; which < 2; ++which) {
    if constexpr (G == 1) {
#pragma unroll
      for (int j = 0; j < J; ++j)
        if (feature(j) < a.K) put(which, feature(j), which ? db[j] : dw[j]);
    } else {
      __syncthreads();
#pragma unroll
      for (int j = 0; j < J; ++j) col[group][lane + 64 * W * j] = which ? db[j] : dw[j];
      __syncthreads();
      for (int i = threadIdx.x; i < 64 * W * J && V * i < a.K; i += kThreads) {
        Vec<V> t = col[0][i];
#pragma unroll 4
        for (int gg = 1; gg < G; ++gg) t += col[gg][i];
        put(which, V * i, t);
      }
    }
  }
}

// Gradients on longer tokens: dx by one workgroup per token that reads it
// twice, and before it (it may overwrite dy) ...
template <typename T>
__global__ __launch_bounds__(kLoopThreads) void norm_backward_dx_kernel(NormBackArgs a) {
  constexpr int W = kLoopThreads / 64;
  __shared__ float red[2][W];
  const int wave = threadIdx.x >> 6;
  const int m = blockIdx.x;
  const T* x = static_cast<const T*>(a.x) + (size_t)m * a.K;
  const T* dy = static_cast<const T*>(a.dy) + (size_t)m * a.K;
  T* dx = static_cast<T*>(a.dx) + (size_t)m * a.K;
  const auto add = [](float p, float q) { return p + q; };
  const float mean = a.mean[m], rstd = a.rstd[m];
  auto load = [&](int k, f4& g, f4& xh) {
    g = load4(dy + k);
    if (a.w) g *= load4(a.w + k);
    xh = (load4(x + k) - mean) * rstd;
  };
  float s1 = 0.0f, s2 = 0.0f;
  f4 g, xh;
  for (int k = 4 * threadIdx.x; k < a.K; k += 4 * kLoopThreads) {
    load(k, g, xh);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      s1 += g[i];
      s2 += g[i] * xh[i];
    }
  }
  s1 = group_join<W>(wave_sum(s1), red[0], wave, add) / (float)a.K;
  s2 = group_join<W>(wave_sum(s2), red[1], wave, add) / (float)a.K;
  for (int k = 4 * threadIdx.x; k < a.K; k += 4 * kLoopThreads) {
    load(k, g, xh);
    store4(dx + k, (g - s1 - xh * s2) * rstd);
  }
}

// ... partial dw, db by workgroups that each take 1024 columns (grid x)
// of a share of the tokens (grid y).
template <typename T>
__global__ __launch_bounds__(256) void norm_backward_columns_kernel(NormBackArgs a) {
  const int k = 4 * (blockIdx.x * 256 + threadIdx.x);
  if (k >= a.K) return;
  f4 dw{0.0f, 0.0f, 0.0f, 0.0f}, db = dw;
  for (int m = blockIdx.y; m < a.M; m += gridDim.y) {
    const f4 g = load4(static_cast<const T*>(a.dy) + (size_t)m * a.K + k);
    const f4 x = load4(static_cast<const T*>(a.x) + (size_t)m * a.K + k);
    dw += g * ((x - a.mean[m]) * a.rstd[m]);
    db += g;
  }
  float* part = a.part + (size_t)blockIdx.y * 2 * a.K;
  store4(part + k, dw);
  store4(part + a.K + k, db);
}

// Sums of the partial rows: 64 columns x 16 shares of the rows per workgroup.
__global__ __launch_bounds__(1024) void norm_columns_kernel(const float* part, int rows, int K, float* dw,
                                                            float* db) {
  __shared__ float red[16][64];
  const int lane = threadIdx.x & 63, share = threadIdx.x >> 6;
  const int k = blockIdx.x * 64 + lane;      // of 2 K: dw's columns, then db's
  float t = 0.0f;
  if (k < 2 * K) {
#pragma unroll 8
    for (int r = share; r < rows; r += 16) t += part[(size_t)r * 2 * K + k];
  }
  red[share][lane] = t;
  __syncthreads();
  if (share == 0 && k < 2 * K) {
    for (int i = 1; i < 16; ++i) t += red[i][lane];
    if (k < K) {
      if (dw) dw[k] = t;
    } else if (db) {
      db[k - K] = t;
    }
  }
}

// As many workgroups as the registers hold at once, which then take further
// tokens in turns with w and b at hand (bf16, us, against 4 per CU: 2048 x 4096
// 8.6 -> 8.1, into int8 11.1 -> 10.0; 4096 x 8192 29.6 -> 26.5, 2048 x 12288 27.4
// -> 24.8).  With up to 8 features a lane that is 4 (16384 x 2048 29.9 -> 27.6
// against 3, 4096 x 2048 9.40 -> 9.33), but 3 into int8 (2048 x 2048 8.1 -> 7.8
// against 4, though 16384 x 2048 42.1 -> 44.3).
template <typename T, int V, int W, int J, bool Q>
void launch_norm_tokens(const NormArgs& a, hipStream_t stream) {
  constexpr int kThreads = W == 16 ? 1024 : 256, G = kThreads / 64 / W;
  const int need = (a.M + G - 1) / G, most = (W == 16 ? 1 : J * V > 16 ? 2 : J * V > 8 || Q ? 3 : 4) * kCUs;
  hipLaunchKernelGGL((norm_kernel<T, V, W, J, Q>), dim3(need < most ? need : most), dim3(kThreads), 0, stream, a);
}

// W: 1 wave up to 1024 features (no barrier); above, 4, or 16 where the tokens
// are too few to fill the GPU with 4 each (at most kCUs of them; measured at
// 16 tokens of 8192 bf16 features into int8: 4 waves 9.0 us, 16 waves 7.0), and
// for int8 above 8192 features, where 4 waves' registers spill (4096 x 16384
// fp32 259 us, 16 waves 93.7; 2048 x 12288 bf16 35.3 and 37.6; at 8192 features
// and below 16 waves are slower, 4096 x 8192 bf16 57.8 against 30.5).
template <typename T, int V, bool Q>
hipError_t launch_norm_as(const NormArgs& a, hipStream_t stream) {
  const int chunks = (a.K + V - 1) / V;   // of V features
  const bool wide = a.M <= kCUs || (Q && a.K > 8192);
  if (a.K <= 1024) {
    if (chunks <= 64) launch_norm_tokens<T, V, 1, 1, Q>(a, stream);
    else if (chunks <= 128) launch_norm_tokens<T, V, 1, 2, Q>(a, stream);
    else if constexpr (V == 4) launch_norm_tokens<T, V, 1, 4, Q>(a, stream);
  } else if (wide && a.K <= kNormMaxK) {
    if (chunks <= 1024) launch_norm_tokens<T, V, 16, 1, Q>(a, stream);
    else if (chunks <= 2048) launch_norm_tokens<T, V, 16, 2, Q>(a, stream);
    else if constexpr (V == 4) launch_norm_tokens<T, V, 16, 4, Q>(a, stream);
  } else if (a.K <= kNormMaxK) {
    if (chunks <= 256) launch_norm_tokens<T, V, 4, 1, Q>(a, stream);
    else if (chunks <= 512) launch_norm_tokens<T, V, 4, 2, Q>(a, stream);
    else if (chunks <= 1024) launch_norm_tokens<T, V, 4, 4, Q>(a, stream);
    else if constexpr (V == 4 || !Q) {
      if (chunks <= 2048) launch_norm_tokens<T, V, 4, 8, Q>(a, stream);
      else if constexpr (!Q) launch_norm_tokens<T, V, 4, 16, Q>(a, stream);
    }
  } else {
    hipLaunchKernelGGL((norm_loop_kernel<T, Q>), dim3(a.M), dim3(kLoopThreads), 0, stream, a);
  }
  return hipGetLastError();
}

// 16 bytes a load where the rows allow it.
template <typename T, bool Q>
hipError_t launch_norm_type(const NormArgs& a, hipStream_t stream) {
  if constexpr (sizeof(T) == 2) {
    if (a.K % 8 == 0) return launch_norm_as<T, 8, Q>(a, stream);
  }
  return launch_norm_as<T, 4, Q>(a, stream);
}

// Waves per token of the backward.
int back_waves(int K) { return K <= 1024 ? 1 : K <= 2048 ? 2 : K <= 4096 ? 4 : K <= 8192 ? 8 : 16; }

template <typename T, int V>
hipError_t launch_norm_backward_as(const NormBackArgs& a, int blocks, hipStream_t stream) {
#define SHERRY_NORM_BACK(W_, J_) \
  hipLaunchKernelGGL((norm_backward_kernel<T, V, W_, J_ * 4 / V>), dim3(blocks), dim3(back_threads(W_)), 0, stream, a)
  if (a.K <= 512) SHERRY_NORM_BACK(1, 2);
  else if (a.K <= 1024) SHERRY_NORM_BACK(1, 4);
  else if (a.K <= 2048) SHERRY_NORM_BACK(2, 4);
  else if (a.K <= 4096) SHERRY_NORM_BACK(4, 4);
  else if (a.K <= 8192) SHERRY_NORM_BACK(8, 4);
  else SHERRY_NORM_BACK(16, 4);
#undef SHERRY_NORM_BACK
  return hipGetLastError();
}

template <typename T>
hipError_t launch_norm_backward_type(const NormBackArgs& a, int blocks, hipStream_t stream) {
  if (a.K > kNormMaxK) {
    // (the columns first: dx may be dy)
    hipLaunchKernelGGL(norm_backward_columns_kernel<T>, dim3((a.K + 1023) / 1024, blocks), dim3(256), 0, stream, a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(norm_backward_dx_kernel<T>, dim3(a.M), dim3(kLoopThreads), 0, stream, a);
    return hipGetLastError();
  }
  if constexpr (sizeof(T) == 2) {
    if (a.K % 8 == 0) return launch_norm_backward_as<T, 8>(a, blocks, stream);
  }
  return launch_norm_backward_as<T, 4>(a, blocks, stream);
}

}  // namespace

hipError_t launch_layernorm(const void* x, const float* w, const float* b, float eps, void* y, int8_t* q,
                            float* s, float* mean, float* rstd, int dtype, int M, int K, hipStream_t stream) {
  const NormArgs a{x, w, b, y, q, s, mean, rstd, eps, M, K};
  if (dtype == SHERRY_F32) return q ? launch_norm_type<float, true>(a, stream) : launch_norm_type<float, false>(a, stream);
  if (dtype == SHERRY_F16)
    return q ? launch_norm_type<_Float16, true>(a, stream) : launch_norm_type<_Float16, false>(a, stream);
  return q ? launch_norm_type<__bf16, true>(a, stream) : launch_norm_type<__bf16, false>(a, stream);
}

// Workgroups of the backward = rows of partial dw, db.
int layernorm_backward_rows(int M, int K) {
  if (K > kNormMaxK) return M < 64 ? M : 64;
  const int per = back_threads(back_waves(K)) / 64 / back_waves(K);   // tokens per workgroup and trip
  const int need = (M + per - 1) / per;
  return need < kBackBlocks ? need : kBackBlocks;
}

hipError_t launch_layernorm_backward(const void* dy, const void* x, const float* mean, const float* rstd,
                                     const float* w, void* dx, float* dw, float* db, int dtype, int M, int K,
                                     float* part, hipStream_t stream, bool* partial) {
  const NormBackArgs a{dy, x, mean, rstd, w, dx, part, M, K};
  const int blocks = layernorm_backward_rows(M, K);
  *partial = false;
  hipError_t e = dtype == SHERRY_F32   ? launch_norm_backward_type<float>(a, blocks, stream)
                 : dtype == SHERRY_F16 ? launch_norm_backward_type<_Float16>(a, blocks, stream)
                                       : launch_norm_backward_type<__bf16>(a, blocks, stream);
  if (e != hipSuccess) return e;
  *partial = true;
  if (dw || db) {
    hipLaunchKernelGGL(norm_columns_kernel, dim3((2 * K + 63) / 64), dim3(1024), 0, stream, part, blocks, K, dw, db);
    e = hipGetLastError();
  }
  return e;
}

}  // namespace sherry
