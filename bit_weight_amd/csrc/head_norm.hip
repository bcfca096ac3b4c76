// Queries and keys of a stacked q/k/v projection, each head normalized and
// turned by its token's position in one pass:
//   r = 1 / sqrt(sum x^2 / D + eps),  y = x r w   (or y = x without the norm),
//   z = y with the pairs (a, b) of its first R features turned by the angle
//       position * freq: (a cos - b sin, b cos + a sin),
// and its gradients, from dz:
//   dy = dz turned back,  dw = sum over tokens and heads of dy x r,  g = dy w,
//   dx = r (g - x r mean(g x r)).
//
// A lane holds 8 features of a head as four pairs (features 4 j .. and R/2 +
// 4 j .. for pairs of halves, 8 j .. for neighbours), so that nothing crosses
// lanes but the sums; D / 8 lanes, rounded up to a power of two, hold a head
// and a wave 64 / that many heads of one token.  The four angles are taken in
// 64 bits once for all heads of the token: 2^20 turns lose 20 of 24 bits in
// fp32.  The backward reads x again instead of anything saved.
//
// Bound by memory at many tokens: 8192 tokens of 32 + 8 heads of 128 in bf16 take 32.5 to
// 36.5 us forward (4.6 to 5.2 TB/s) and 55 to 58 backward with the columns' 4.6 (4.5 TB/s;
// the vector units are busy half the time); 8 tokens 5.3, a launch.
#include "sherry_device.h"
#include "sherry_launch.h"
#include "sherry_types.h"

namespace sherry {
namespace {

constexpr int kWaves = 4;
constexpr int kBackBlocks = 2 * kCUs;   // most workgroups of the backward (rows of partial weight gradients)
constexpr int kAhead = 4;               // heads a lane loads before it computes the first

__device__ __forceinline__ float shift_sum(float v, int width) {
  if (width > 1) v += dpp_shift<0xB1>(v);     // neighbours
  if (width > 2) v += dpp_shift<0x4E>(v);     // pairs
  if (width > 4) v += dpp_shift<0x141>(v);    // mirrored halves of 16 lanes: the other four
  if (width > 8) v += dpp_shift<0x140>(v);    // mirrored rows: the other eight
  if (width > 16) v += __shfl_xor(v, 16);
  return v;
}

struct Unit {      // a lane's eight features: the first and second of four pairs, or 4 + 4 that do not turn
  f4 a, b;
};

// Where they lie in the head, and the four pairs they make.
struct Place {
  int a, b;
  bool turns, next;    // next: pairs of neighbours
  __device__ __forceinline__ Unit pairs(Unit u) const {
    return next ? Unit{f4{u.a.x, u.a.z, u.b.x, u.b.z}, f4{u.a.y, u.a.w, u.b.y, u.b.w}} : u;
  }
  __device__ __forceinline__ Unit order(Unit u) const {
    return next ? Unit{f4{u.a.x, u.b.x, u.a.y, u.b.y}, f4{u.a.z, u.b.z, u.a.w, u.b.w}} : u;
  }
};

__device__ __forceinline__ Place place_of(int j, int rotary, bool interleaved) {
  const bool turns = 8 * j < rotary;
  if (turns && !interleaved) return {4 * j, rotary / 2 + 4 * j, true, false};
  return {8 * j, 8 * j + 4, turns, turns};
}

// cos and sin of the lane's four angles (1 and 0 where nothing turns).
__device__ __forceinline__ void angles(const double* freqs, int position, int j, bool turns, f4& c, f4& s) {
  c = f4{1.0f, 1.0f, 1.0f, 1.0f};
  s = f4{};
  if (!turns) return;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    // in turns, the whole ones taken off in 64 bits
    const double t = (double)position * (freqs[4 * j + i] * 0.15915494309189533577);
    const float f = (float)(t - rint(t));
    float si, co;
    sincospif(2.0f * f, &si, &co);
    c[i] = co;
    s[i] = si;
  }
}

__device__ __forceinline__ Unit turn(Unit u, f4 c, f4 s) { return {u.a * c - u.b * s, u.b * c + u.a * s}; }

__device__ __forceinline__ float dot(Unit u, Unit v) {
  const f4 p = u.a * v.a + u.b * v.b;
  return (p.x + p.y) + (p.z + p.w);
}

// 1 / sqrt(mean of squares + eps).  Where the squares pass fp32's range, u is
// made 2^-70 as large (`down`) and so is what it is the inverse of.
__device__ __forceinline__ float rms(Unit& u, float inv_d, float eps, int width, float& down) {
  const float m = shift_sum(dot(u, u), width) * inv_d;
  down = 1.0f;
  if (m < 1e37f) return rsqrtf(m + eps);
  down = 0x1p-70f;
  u.a *= down;
  u.b *= down;
  return rsqrtf(shift_sum(dot(u, u), width) * inv_d + eps * down * down);
}

template <typename T>
struct RawUnit {
  typedef T v4 __attribute__((ext_vector_type(4)));
  v4 a, b;
  __device__ __forceinline__ Unit get() const {
    return {__builtin_convertvector(a, f4), __builtin_convertvector(b, f4)};
  }
  __device__ __forceinline__ void load(const T* head, const Place& p) {
    a = *reinterpret_cast<const v4*>(head + p.a);
    b = *reinterpret_cast<const v4*>(head + p.b);
  }
};

template <typename T>
__device__ __forceinline__ void store_unit(T* head, const Place& p, Unit u) {
  store4(head + p.a, u.a);
  store4(head + p.b, u.b);
}

__device__ __forceinline__ Unit weight_of(const float* w, const Place& p, bool in) {
  if (!w || !in) return {f4{1.0f, 1.0f, 1.0f, 1.0f}, f4{1.0f, 1.0f, 1.0f, 1.0f}};
  return {load4(w + p.a), load4(w + p.b)};
}

template <typename T, int kWidth, bool kNorm>
__global__ __launch_bounds__(64 * kWaves) void head_norm_kernel(HeadNormArgs g, int per_item, int items) {
  constexpr int kHeads = 64 / kWidth;
  const int lane = threadIdx.x & 63, j = lane % kWidth, sub = lane / kWidth;
  const int item = blockIdx.x * kWaves + (threadIdx.x >> 6);
  const int chunks = items / g.T, t = item / chunks;
  if (t >= g.T) return;
  const int all = g.Hq + g.Hk, first = (item - t * chunks) * per_item, last = min(first + per_item, all);
  const bool in = 8 * j < g.D;
  const Place p = place_of(in ? j : 0, g.R, g.interleaved);
  const T* x = static_cast<const T*>(g.x) + (size_t)t * g.x_stride;
  T* q = static_cast<T*>(g.q) + (size_t)t * g.Hq * g.D;
  T* k = static_cast<T*>(g.k) + (size_t)t * g.Hk * g.D;
  const Unit wq = weight_of(kNorm ? g.wq : nullptr, p, in), wk = weight_of(kNorm ? g.wk : nullptr, p, in);
  RawUnit<T> raw[kAhead];
  f4 c, s;
  angles(g.freqs, g.positions[t], j, in && p.turns, c, s);
  const float inv_d = 1.0f / (float)g.D;
  for (int h0 = first + sub; h0 < last + sub; h0 += kAhead * kHeads) {     // (the same count for every lane)
#pragma unroll
    for (int i = 0; i < kAhead; ++i) raw[i].load(x + (size_t)min(h0 + i * kHeads, last - 1) * g.D, p);
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const int h = h0 + i * kHeads;
      const bool write = in && h < last, is_q = h < g.Hq;
      Unit u = raw[i].get();
      if constexpr (kNorm) {
        if (!in) u = Unit{f4{}, f4{}};
        float down;
        const float r = rms(u, inv_d, g.eps, kWidth, down);
        u.a = u.a * r * (is_q ? wq.a : wk.a);
        u.b = u.b * r * (is_q ? wq.b : wk.b);
      }
      u = p.order(turn(p.pairs(u), c, s));
      if (write) store_unit(is_q ? q + (size_t)h * g.D : k + (size_t)(h - g.Hq) * g.D, p, u);
    }
  }
}

// Tokens in turn; dw of a lane's features in registers, joined at the end.  kAt: query heads a
// lane loads before it computes the first.
template <typename T, int kWidth, bool kNorm, int kAt>
__global__ __launch_bounds__(64 * kWaves) void head_norm_backward_kernel(HeadNormArgs g, int per_item, int items) {
  constexpr int kHeads = 64 / kWidth;
  __shared__ float join[kWaves][2][8 * kWidth];
  const int lane = threadIdx.x & 63, j = lane % kWidth, sub = lane / kWidth, wave = threadIdx.x >> 6;
  const bool in = 8 * j < g.D;
  const Place p = place_of(in ? j : 0, g.R, g.interleaved);
  const float inv_d = 1.0f / (float)g.D;
  const int chunks = items / g.T, all = g.Hq + g.Hk;
  Unit dw[2] = {};
  const Unit weights[2] = {weight_of(kNorm ? g.wq : nullptr, p, in), weight_of(kNorm ? g.wk : nullptr, p, in)};

  // heads first .. last - 1 of one kind, x and dx at the token's head 0, dz at its first of this kind
  auto heads = [&](auto of, const T* x, const T* dz, T* dx, int first, int last, f4 c, f4 s) {
    constexpr int kind = decltype(of)::value;      // 0: queries, 1: keys
    constexpr int kIn = kind ? 2 : kAt;
    const int base = kind ? g.Hq : 0;
    for (int h0 = first + sub; h0 < last + sub; h0 += kIn * kHeads) {
      RawUnit<T> rx[kIn], rz[kIn];
#pragma unroll
      for (int i = 0; i < kIn; ++i) {
        const int h = min(h0 + i * kHeads, last - 1);
        if constexpr (kNorm) rx[i].load(x + (size_t)h * g.D, p);
        rz[i].load(dz + (size_t)(h - base) * g.D, p);
      }
#pragma unroll
      for (int i = 0; i < kIn; ++i) {
        const int h = h0 + i * kHeads;
        const bool use = in && h < last;
        Unit dy = p.order(turn(p.pairs(rz[i].get()), c, -s));
        if constexpr (kNorm) {
          Unit u = rx[i].get();
          if (!use) u = dy = Unit{f4{}, f4{}};
          float down;
          const float r = rms(u, inv_d, g.eps, kWidth, down);
          u.a *= r;
          u.b *= r;
          dw[kind].a += dy.a * u.a;
          dw[kind].b += dy.b * u.b;
          dy.a *= weights[kind].a;
          dy.b *= weights[kind].b;
          const float m = shift_sum(dot(dy, u), kWidth) * inv_d;
          dy.a = down * (r * (dy.a - u.a * m));
          dy.b = down * (r * (dy.b - u.b * m));
        }
        if (use) store_unit(dx + (size_t)h * g.D, p, dy);
      }
    }
  };

  for (int item = blockIdx.x * kWaves + wave; item < items; item += gridDim.x * kWaves) {
    const int t = item / chunks, first = (item - t * chunks) * per_item, last = min(first + per_item, all);
    const T* x = static_cast<const T*>(g.x) + (size_t)t * g.x_stride;
    T* dx = static_cast<T*>(g.dx) + (size_t)t * g.dx_stride;
    f4 c, s;
    angles(g.freqs, g.positions[t], j, in && p.turns, c, s);
    if (first < g.Hq)
      heads(std::integral_constant<int, 0>{}, x, static_cast<const T*>(g.q) + (size_t)t * g.Hq * g.D, dx, first, min(last, g.Hq), c, s);
    if (last > g.Hq)
      heads(std::integral_constant<int, 1>{}, x, static_cast<const T*>(g.k) + (size_t)t * g.Hk * g.D, dx, max(first, g.Hq), last, c, s);
  }
  if constexpr (kNorm) {
#pragma unroll
    for (int kind = 0; kind < 2; ++kind)
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        float v = i < 4 ? dw[kind].a[i] : dw[kind].b[i - 4];
#pragma unroll
        for (int d = kWidth; d < 64; d *= 2) v += __shfl_xor(v, d);
        if (sub == 0 && in) join[wave][kind][i < 4 ? p.a + i : p.b + i - 4] = v;
      }
    __syncthreads();
    for (int i = threadIdx.x; i < 2 * g.D; i += 64 * kWaves) {
      const int kind = i / g.D, f = i - kind * g.D;
      float v = 0.0f;
#pragma unroll
      for (int w = 0; w < kWaves; ++w) v += join[w][kind][f];
      g.part[(size_t)blockIdx.x * 2 * g.D + i] = v;
    }
  }
}

// Sums of the workgroups' rows of 2 D, always in the same order: 16 columns and 64
// rows at a time, 8 loads asked for together (64 columns and 16 rows: 1 us more).
__global__ __launch_bounds__(1024) void head_norm_columns_kernel(const float* part, int rows, int D, float* dwq,
                                                                 float* dwk) {
  __shared__ float join[16][16];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, col = blockIdx.x * 16 + (lane & 15);
  float v = 0.0f;
  if (col < 2 * D) {
    for (int r0 = threadIdx.x >> 4; r0 < rows; r0 += 8 * 64) {
      float x[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = part[(size_t)min(r0 + 64 * i, rows - 1) * 2 * D + col];
#pragma unroll
      for (int i = 0; i < 8; ++i) v += r0 + 64 * i < rows ? x[i] : 0.0f;
    }
  }
  v += __shfl_xor(v, 16);
  v += __shfl_xor(v, 32);
  if (lane < 16) join[wave][lane] = v;
  __syncthreads();
  if (threadIdx.x < 16 && col < 2 * D) {
    v = 0.0f;
#pragma unroll
    for (int i = 0; i < 16; ++i) v += join[i][threadIdx.x];
    if (col < D) {
      if (dwq) dwq[col] = v;
    } else if (dwk) {
      dwk[col - D] = v;
    }
  }
}

int width_of(int D) {
  int w = 2;
  while (8 * w < D) w *= 2;
  return w;
}

// Heads a wave takes of a token: all of them where the tokens alone give
// every SIMD two waves, fewer (whole loads of the wave) at few tokens.
int heads_per_item(int T, int all, int heads_in_wave) {
  const int want = 2 * 4 * kCUs, chunks = max(1, min((want + T - 1) / T, (all + heads_in_wave - 1) / heads_in_wave));
  return (((all + chunks - 1) / chunks) + heads_in_wave - 1) / heads_in_wave * heads_in_wave;
}

template <typename T, int kWidth, bool kNorm>
void launch_forward(const HeadNormArgs& g, hipStream_t stream) {
  const int all = g.Hq + g.Hk, per = heads_per_item(g.T, all, 64 / kWidth), items = g.T * ((all + per - 1) / per);
  head_norm_kernel<T, kWidth, kNorm><<<(items + kWaves - 1) / kWaves, 64 * kWaves, 0, stream>>>(g, per, items);
}

template <typename T, int kWidth, bool kNorm, int kAt>
void launch_back_at(const HeadNormArgs& g, hipStream_t stream) {
  const int all = g.Hq + g.Hk, per = heads_per_item(g.T, all, 64 / kWidth), items = g.T * ((all + per - 1) / per);
  head_norm_backward_kernel<T, kWidth, kNorm, kAt>
      <<<min((items + kWaves - 1) / kWaves, kBackBlocks), 64 * kWaves, 0, stream>>>(g, per, items);
}

// Four heads at a time where an item has so many, else two: 8192 tokens of 32 + 8 heads of
// 128 in bf16 54.7 and 58.4 us, 777 of 12 + 4 heads of 80 in fp32 12.3 and 10.2.
template <typename T, int kWidth, bool kNorm>
void launch_back(const HeadNormArgs& g, hipStream_t stream) {
  if (heads_per_item(g.T, g.Hq + g.Hk, 64 / kWidth) >= 4 * (64 / kWidth)) launch_back_at<T, kWidth, kNorm, 4>(g, stream);
  else launch_back_at<T, kWidth, kNorm, 2>(g, stream);
}

template <typename F>
void by_width(int D, F f) {
  switch (width_of(D)) {
    case 2: return f(std::integral_constant<int, 2>{});
    case 4: return f(std::integral_constant<int, 4>{});
    case 8: return f(std::integral_constant<int, 8>{});
    case 16: return f(std::integral_constant<int, 16>{});
    default: return f(std::integral_constant<int, 32>{});
  }
}

template <typename F>
void by_type(int dtype, F f) {
  if (dtype == SHERRY_F32) f(float{});
  else if (dtype == SHERRY_F16) f(_Float16{});
  else f(__bf16{});
}

}  // namespace

hipError_t launch_head_norm(const HeadNormArgs& g, hipStream_t stream) {
  by_type(g.dtype, [&](auto t) {
    by_width(g.D, [&](auto w) {
      if (g.norm) launch_forward<decltype(t), decltype(w)::value, true>(g, stream);
      else launch_forward<decltype(t), decltype(w)::value, false>(g, stream);
    });
  });
  return hipGetLastError();
}

int head_norm_backward_rows(int T, int all, int D) {
  const int per = heads_per_item(T, all, 64 / width_of(D)), items = T * ((all + per - 1) / per);
  return min((items + kWaves - 1) / kWaves, kBackBlocks);
}

hipError_t launch_head_norm_backward(const HeadNormArgs& g, float* dwq, float* dwk, hipStream_t stream,
                                     bool* partial) {
  by_type(g.dtype, [&](auto t) {
    by_width(g.D, [&](auto w) {
      if (g.norm) launch_back<decltype(t), decltype(w)::value, true>(g, stream);
      else launch_back<decltype(t), decltype(w)::value, false>(g, stream);
    });
  });
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || !g.norm || (!dwq && !dwk)) return e;
  *partial = true;
  head_norm_columns_kernel<<<(2 * g.D + 15) / 16, 1024, 0, stream>>>(
      g.part, head_norm_backward_rows(g.T, g.Hq + g.Hk, g.D), g.D, dwq, dwk);
  return hipGetLastError();
}

}  // namespace sherry
