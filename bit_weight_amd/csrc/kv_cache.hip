// Writing keys and values into the 8-bit cache and reading them back.
//
// A block (16 tokens of one head) has one scale, the least power of two 2^e with
// max|x| <= 127 2^e; q = rint(x 2^-e).  With a power of two every product here is
// exact, so q and the values read back are what the definition says to the last
// bit, and when a later token makes the scale grow, the older values take one
// more rounding of half a new step each time it doubles: one step at most in all.
// (A scale of max/127 would use the range better by half a bit on average, but
// grow, and round the older values again, with almost every new maximum.)
//
// A wave holds one block of keys or of values: 16 features of one token are a
// lane's unit, and D units a block's.  Values lie token by token in memory and
// feature by feature in the cache, so they cross lanes through LDS.
#include "sherry_cache.h"

namespace sherry {
namespace {

constexpr int kWaves = 4;

// Least scale for a largest |x|: 1.f 2^E <= 127 2^e = 1.984375 2^(e + 6).
__device__ __forceinline__ float least_scale(float top) {
  const uint32_t u = __builtin_bit_cast(uint32_t, top);
  const int e = (int)(u >> 23) - 6 + ((u & 0x7FFFFFu) > 0x7E0000u ? 1 : 0);
  return __builtin_bit_cast(float, (uint32_t)max(e, 1) << 23);
}

// Sixteen consecutive values.
struct Sixteen {
  f4 v[4];
};

__device__ __forceinline__ Sixteen load16(const void* p, size_t i, int dtype) {
  u4 raw[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) raw[j] = load4_raw(p, i + 4 * j, dtype);
  Sixteen s;
#pragma unroll
  for (int j = 0; j < 4; ++j) s.v[j] = as_f4(raw[j], dtype);
  return s;
}

__device__ __forceinline__ uint32_t pack4(f4 v, float inv) {
  uint32_t w = 0;
#pragma unroll
  for (int j = 0; j < 4; ++j)
    w |= ((uint32_t)(int)rintf(fminf(fmaxf(v[j] * inv, -127.0f), 127.0f)) & 255u) << (8 * j);
  return w;
}

__device__ __forceinline__ uint4 pack16(const Sixteen& s, float inv) {
  return make_uint4(pack4(s.v[0], inv), pack4(s.v[1], inv), pack4(s.v[2], inv), pack4(s.v[3], inv));
}

__device__ __forceinline__ f4 bytes4(uint32_t w) {
  return f4{(float)(int8_t)w, (float)(int8_t)(w >> 8), (float)(int8_t)(w >> 16), (float)(int8_t)(w >> 24)};
}

__device__ __forceinline__ uint32_t again4(uint32_t w, float ratio) { return pack4(bytes4(w), ratio); }

__device__ __forceinline__ uint4 again16(uint4 w, float ratio) {
  return make_uint4(again4(w.x, ratio), again4(w.y, ratio), again4(w.z, ratio), again4(w.w, ratio));
}

// kUnits: units of a lane, D / 64 rounded up.
template <int kUnits>
__global__ __launch_bounds__(64 * kWaves) void cache_write_kernel(CacheArgs c, int blocks) {
  __shared__ uint4 turn[kWaves][64 * kUnits];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int item = blockIdx.x * kWaves + wave, w = item / (2 * c.H);
  const bool values = item & 1;
  const int h = (item >> 1) % c.H, chunks = c.D / 16;
  int seq = 0, number = 0;
  bool work = w < blocks && find_item(c.S, w, [&](int i) { return blocks_of(rows_of(c, i)).y; }, seq, number);
  const Rows r = rows_of(c, seq);
  const int first = r.len - r.n, sb = blocks_of(r).x + number;       // position of the first new token
  const int page = work ? page_of(c, seq, sb) : -1;
  work = page >= 0;
  const size_t block = work ? block_of(c, page, h, sb) : 0;
  uint8_t* at = (values ? c.v : c.k) + block * (16 * c.D);
  float* scale = (values ? c.v_scale : c.k_scale) + block;
  const int old = min(max(first - 16 * sb, 0), 16), end = min(r.len - 16 * sb, 16);   // tokens old .. end - 1 are new

  Sixteen x[kUnits];
  float top = 0.0f;
  bool finite = true;
#pragma unroll
  for (int u = 0; u < kUnits; ++u) {
    const int unit = lane + 64 * u, i = unit / chunks, d = 16 * (unit - i * chunks);
    if (work && i >= old && i < end) {
      const size_t row = (size_t)(r.row0 + 16 * sb + i - first);
      x[u] = values ? load16(c.x_v, row * c.v_stride + (size_t)h * c.D + d, c.dtype)
                    : load16(c.x_k, row * c.k_stride + (size_t)h * c.D + d, c.dtype);
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int b = 0; b < 4; ++b) {
          const float a = fabsf(x[u].v[j][b]);
          top = fmaxf(top, a);
          finite &= a < __builtin_inff();
        }
    }
  }
  top = wave_max(top);
  float now = least_scale(top), before = 0.0f;
  if (!__all(finite)) now = __builtin_nanf("");
  if (work && old > 0) {
    before = *scale;
    now = before > now || before != before ? before : now;
  }
  const float inv = 1.0f / now, ratio = before * inv;
  if (work && !values) {
#pragma unroll
    for (int u = 0; u < kUnits; ++u) {
      const int unit = lane + 64 * u, i = unit / chunks, piece = unit - i * chunks;
      uint4* to = reinterpret_cast<uint4*>(at + 256 * piece + 16 * i);
      if (i >= old && i < end) *to = pack16(x[u], inv);
      else if (i < old && ratio != 1.0f) *to = again16(*to, ratio);
    }
  }
  uint8_t* bytes = reinterpret_cast<uint8_t*>(turn[wave]);      // [16 tokens][D]
  if (work && values) {
#pragma unroll
    for (int u = 0; u < kUnits; ++u) {
      const int unit = lane + 64 * u;
      if (unit < c.D) reinterpret_cast<uint4*>(bytes)[unit] = pack16(x[u], inv);
    }
  }
  __syncthreads();
  if (work && values) {
#pragma unroll
    for (int u = 0; u < kUnits; ++u) {
      const int f = lane + 64 * u;       // one feature of 16 tokens
      if (f >= c.D) continue;
      uint4* to = reinterpret_cast<uint4*>(at + 16 * f);
      uint32_t had[4] = {}, put[4];
      if (old > 0 || end < 16) {
        const uint4 o = *to;
        had[0] = o.x, had[1] = o.y, had[2] = o.z, had[3] = o.w;
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t rounded = ratio != 1.0f ? again4(had[j], ratio) : had[j];
        uint32_t v = 0;
#pragma unroll
        for (int b = 0; b < 4; ++b) {
          const int i = 4 * j + b;
          const uint32_t byte = i < old ? (rounded >> (8 * b)) & 255u
                              : i < end ? bytes[i * c.D + f] : (had[j] >> (8 * b)) & 255u;
          v |= byte << (8 * b);
        }
        put[j] = v;
      }
      *to = make_uint4(put[0], put[1], put[2], put[3]);
    }
  }
  if (work && lane == 0 && now != before) *scale = now;
}

// Tokens without a page are read back as NaN.
template <int kUnits>
__global__ __launch_bounds__(64 * kWaves) void cache_read_kernel(CacheArgs c, int blocks, void* k, void* v) {
  constexpr int kPitch = 272;      // of 16 features: 256 bytes and 16 between, so that lanes read different banks
  __shared__ uint4 turn[kWaves][kUnits * 4 * kPitch / 16];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int item = blockIdx.x * kWaves + wave, w = item / (2 * c.H);
  const bool values = item & 1;
  const int h = (item >> 1) % c.H, chunks = c.D / 16;
  int seq = 0, number = 0;
  const bool work = w < blocks && find_item(c.S, w, [&](int i) { return blocks_of(rows_of(c, i)).y; }, seq, number);
  const Rows r = rows_of(c, seq);
  const int first = r.len - r.n, sb = blocks_of(r).x + number;
  const int page = work ? page_of(c, seq, sb) : -1;
  const size_t block = page >= 0 ? block_of(c, page, h, sb) : 0;
  const uint8_t* at = (values ? c.v : c.k) + block * (16 * c.D);
  float scale = (values ? c.v_scale : c.k_scale)[block];
  if (page < 0) scale = __builtin_nanf("");
  uint8_t* bytes = reinterpret_cast<uint8_t*>(turn[wave]);
  uint4 q[kUnits];
#pragma unroll
  for (int u = 0; u < kUnits; ++u) {
    const int unit = lane + 64 * u;
    if (!work || unit >= c.D) continue;
    if (values) {        // unit: a feature
      *reinterpret_cast<uint4*>(bytes + (unit >> 4) * kPitch + 16 * (unit & 15)) =
          *reinterpret_cast<const uint4*>(at + 16 * unit);
    } else {             // unit: 16 features of a token
      const int i = unit / chunks, piece = unit - i * chunks;
      q[u] = *reinterpret_cast<const uint4*>(at + 256 * piece + 16 * i);
    }
  }
  __syncthreads();
#pragma unroll
  for (int u = 0; u < kUnits; ++u) {
    const int unit = lane + 64 * u;
    if (!work || unit >= c.D) continue;
    const int i = unit / chunks, piece = unit - i * chunks, position = 16 * sb + i;
    if (position < first || position >= r.len) continue;
    uint32_t word[4] = {q[u].x, q[u].y, q[u].z, q[u].w};
    if (values) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        word[j] = 0;
#pragma unroll
        for (int b = 0; b < 4; ++b)
          word[j] |= (uint32_t)bytes[piece * kPitch + 16 * (4 * j + b) + i] << (8 * b);
      }
    }
    const size_t to = ((size_t)(r.row0 + position - first) * c.H + h) * c.D + 16 * piece;
#pragma unroll
    for (int j = 0; j < 4; ++j) store4_as(values ? v : k, to + 4 * j, c.dtype, bytes4(word[j]) * scale);
  }
}

// Blocks that T rows of S sequences lie in, at most: a sequence of n has no
// more than (n + 30) / 16, and no more than n.
int64_t most_blocks(const CacheArgs& c) {
  const int64_t t = c.T;
  return std::min<int64_t>(t, t / 16 + 2 * (int64_t)c.S);
}

template <typename F>
void by_units(int D, F f) {
  switch ((D + 63) / 64) {
    case 1: return f(std::integral_constant<int, 1>{});
    case 2: return f(std::integral_constant<int, 2>{});
    case 3: return f(std::integral_constant<int, 3>{});
    default: return f(std::integral_constant<int, 4>{});
  }
}

}  // namespace

hipError_t launch_cache_write(const CacheArgs& c, hipStream_t stream) {
  const int64_t blocks = most_blocks(c), items = blocks * 2 * c.H;
  by_units(c.D, [&](auto u) {
    cache_write_kernel<decltype(u)::value>
        <<<(unsigned)((items + kWaves - 1) / kWaves), 64 * kWaves, 0, stream>>>(c, (int)blocks);
  });
  return hipGetLastError();
}

hipError_t launch_cache_read(const CacheArgs& c, void* k, void* v, hipStream_t stream) {
  const int64_t blocks = most_blocks(c), items = blocks * 2 * c.H;
  by_units(c.D, [&](auto u) {
    cache_read_kernel<decltype(u)::value>
        <<<(unsigned)((items + kWaves - 1) / kWaves), 64 * kWaves, 0, stream>>>(c, (int)blocks, k, v);
  });
  return hipGetLastError();
}

}  // namespace sherry
