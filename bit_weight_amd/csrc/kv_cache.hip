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
// A workgroup takes one block of every head it is given, a wave its keys or its values in
// turn.  Keys: a lane's unit is 8 features of one token, 16 lanes a row's 256 bytes of
// bf16.  Values lie feature by feature in the cache: a lane's unit is 4 features of 4
// tokens, turned in registers, and LDS brings the 16 tokens of a feature together
// (4 features 80 bytes apart, so that 64 lanes' words lie in different banks).
//
// All loads of an item are asked for before the first is used, and arrays of loaded bytes
// are ext_vector types (as HIP's uint4 they became stack arrays, which went through LDS:
// 102 instead of 82 us).  Reading is bound by memory.  Writing is not: its waves wait 54 %
// of their time, for a chain (lengths, table, rows, maximum, store) with nothing under it
// where a wave has one or two items.  Measured with 8 heads of 128 in bf16: 64000 tokens
// read in 82 us (4.8 TB/s), 6800 tokens of 5 sequences written in 16.6 (2.5 TB/s), one
// token of 64 sequences written in 5.3, of 1024 in 31.5, of 4096 in 198 (every wave looks
// for its block among all sequences).
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

template <typename T, int n>
using Row = T __attribute__((ext_vector_type(n)));

__device__ __forceinline__ uint32_t pack4(f4 v, float inv) {
  uint32_t w = 0;
#pragma unroll
  for (int j = 0; j < 4; ++j)
    w |= ((uint32_t)(int)rintf(fminf(fmaxf(v[j] * inv, -127.0f), 127.0f)) & 255u) << (8 * j);
  return w;
}

__device__ __forceinline__ f4 bytes4(uint32_t w) {
  return f4{(float)(int8_t)w, (float)(int8_t)(w >> 8), (float)(int8_t)(w >> 16), (float)(int8_t)(w >> 24)};
}

__device__ __forceinline__ uint32_t again4(uint32_t w, float ratio) { return pack4(bytes4(w), ratio); }

// Byte c of word r from byte r of word c.
__device__ __forceinline__ u4 turn4(u4 w) {
  const uint32_t a = __builtin_amdgcn_perm(w.y, w.x, 0x05010400u), b = __builtin_amdgcn_perm(w.w, w.z, 0x05010400u);
  const uint32_t c = __builtin_amdgcn_perm(w.y, w.x, 0x07030602u), d = __builtin_amdgcn_perm(w.w, w.z, 0x07030602u);
  return u4{__builtin_amdgcn_perm(b, a, 0x05040100u), __builtin_amdgcn_perm(b, a, 0x07060302u),
            __builtin_amdgcn_perm(d, c, 0x05040100u), __builtin_amdgcn_perm(d, c, 0x07060302u)};
}

// The block of a workgroup and where its rows are.
struct Place {
  bool work;
  int seq, sb, page;
  Rows r;
  int first;        // position of the sequence's first row
  __device__ __forceinline__ Place(const CacheArgs& c, int block) {
    int number = 0;
    seq = 0;
    work = find_item(c.S, block, [&](int i) { return blocks_of(rows_of(c, i)).y; }, seq, number);
    r = rows_of(c, seq);
    first = r.len - r.n;
    sb = blocks_of(r).x + number;
    page = work ? page_of(c, seq, sb) : -1;
  }
};

// Unit u of a lane, of keys: token (16 or more: none) and eighth of a row.
struct Unit {
  int token, eighth;
  __device__ __forceinline__ Unit(int D, int unit) {
    token = unit / (D / 8);
    eighth = unit - token * (D / 8);
  }
  __device__ __forceinline__ int at() const { return 256 * (eighth >> 1) + 16 * min(token, 15) + 8 * (eighth & 1); }
};

// LDS: the 16 tokens of feature f, and the word of tokens 4 k .. of it.
__device__ __forceinline__ int feature_at(int f) { return 16 * f + 16 * (f >> 2); }

__device__ __forceinline__ void lds_order() { asm volatile("" ::: "memory"); }      // (a wave's LDS accesses keep their order)

template <typename T, int kC>
__global__ __launch_bounds__(64 * kWaves) void cache_write_kernel(CacheArgs c) {
  __shared__ __attribute__((aligned(16))) uint8_t turn[kWaves][kC * 1280];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, D = c.D;
  const Place p(c, blockIdx.x);
  if (p.page < 0) return;
  uint8_t* bytes = turn[wave];
  const int old = min(max(p.first - 16 * p.sb, 0), 16), end = min(p.r.len - 16 * p.sb, 16);   // tokens old .. end - 1 are new
  const size_t row0 = (size_t)((int64_t)p.r.row0 + 16 * p.sb - p.first);                      // row of the block's token 0
  for (int item = blockIdx.y * kWaves + wave; item < 2 * c.H; item += gridDim.y * kWaves) {
    const bool values = item & 1;
    const int h = item >> 1;
    const size_t block = block_of(c, p.page, h, p.sb);
    uint8_t* at = (values ? c.v : c.k) + block * (16 * D);
    float* scale = (values ? c.v_scale : c.k_scale) + block;
    const T* x = static_cast<const T*>(values ? c.x_v : c.x_k) + (size_t)h * D;
    const size_t stride = values ? c.v_stride : c.k_stride;
    const float before = old > 0 ? *scale : 0.0f;

    f4 v[kC][4];        // keys: units 2 u and 2 u + 1, 8 features each; values: tokens 4 k .. of unit u
    Row<T, 4> raw[kC][4];
#pragma unroll
    for (int u = 0; u < kC; ++u)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int token = values ? 4 * (lane & 3) + j : Unit(D, lane + 64 * (2 * u + j / 2)).token;
        const int d = values ? 4 * ((lane + 64 * u) >> 2) : 8 * Unit(D, lane + 64 * (2 * u + j / 2)).eighth + 4 * (j % 2);
        raw[u][j] = Row<T, 4>{};
        if (token >= old && token < end && d < D) raw[u][j] = *reinterpret_cast<const Row<T, 4>*>(x + (row0 + token) * stride + d);
      }
    float top = 0.0f;
    bool finite = true;
#pragma unroll
    for (int u = 0; u < kC; ++u)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        v[u][j] = __builtin_convertvector(raw[u][j], f4);
#pragma unroll
        for (int b = 0; b < 4; ++b) {
          const float a = fabsf(v[u][j][b]);
          top = fmaxf(top, a);
          finite &= a < __builtin_inff();
        }
      }
    float now = least_scale(wave_max(top));
    if (!__all(finite)) now = __builtin_nanf("");
    if (old > 0) now = before > now || before != before ? before : now;
    const float inv = 1.0f / now, ratio = before * inv;
    const bool rescale = old > 0 && ratio != 1.0f;
    if (!values) {
#pragma unroll
      for (int u = 0; u < 2 * kC; ++u) {
        const Unit unit(D, lane + 64 * u);
        const int i = unit.token;
        uint2* to = reinterpret_cast<uint2*>(at + unit.at());
        if (i >= old && i < end) *to = make_uint2(pack4(v[u / 2][2 * (u % 2)], inv), pack4(v[u / 2][2 * (u % 2) + 1], inv));
        else if (i < old && rescale) *to = make_uint2(again4(to->x, ratio), again4(to->y, ratio));
      }
    } else {
      lds_order();      // (the last item's reads)
#pragma unroll
      for (int u = 0; u < kC; ++u) {
        const int unit = lane + 64 * u;
        const u4 w = turn4(u4{pack4(v[u][0], inv), pack4(v[u][1], inv), pack4(v[u][2], inv), pack4(v[u][3], inv)});
#pragma unroll
        for (int j = 0; j < 4; ++j) *reinterpret_cast<uint32_t*>(bytes + feature_at(4 * (unit >> 2) + j) + 4 * (unit & 3)) = w[j];
      }
      lds_order();
#pragma unroll
      for (int u = 0; u < kC; ++u) {
        const int f = lane + 64 * u;
        if (f >= D) continue;
        uint4* to = reinterpret_cast<uint4*>(at + 16 * f);
        uint4 put = *reinterpret_cast<const uint4*>(bytes + feature_at(f));
        if (old > 0 || end < 16) {        // the others as they were, or rounded again
          const uint4 had = *to;
          uint32_t w[4] = {put.x, put.y, put.z, put.w}, o[4] = {had.x, had.y, had.z, had.w};
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const uint32_t rounded = rescale ? again4(o[j], ratio) : o[j];
            uint32_t fresh = 0, earlier = 0;
#pragma unroll
            for (int b = 0; b < 4; ++b) {
              fresh |= 4 * j + b >= old && 4 * j + b < end ? 255u << (8 * b) : 0u;
              earlier |= 4 * j + b < old ? 255u << (8 * b) : 0u;
            }
            w[j] = (w[j] & fresh) | (rounded & earlier) | (o[j] & ~(fresh | earlier));
          }
          put = make_uint4(w[0], w[1], w[2], w[3]);
        }
        *to = put;
      }
    }
    if (lane == 0 && now != before) *scale = now;
  }
}

template <typename T>
__device__ __forceinline__ void put4(T* p, uint32_t w, float scale) { store4(p, bytes4(w) * scale); }

// Tokens without a page are read back as NaN.
template <typename T, int kC>
__global__ __launch_bounds__(64 * kWaves) void cache_read_kernel(CacheArgs c, T* k, T* v) {
  __shared__ __attribute__((aligned(16))) uint8_t turn[kWaves][kC * 1280];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, D = c.D;
  const Place p(c, blockIdx.x);
  if (!p.work) return;
  uint8_t* bytes = turn[wave];
  const int from = max(p.first - 16 * p.sb, 0), end = min(p.r.len - 16 * p.sb, 16);           // tokens asked for
  const int64_t row0 = (int64_t)p.r.row0 + 16 * p.sb - p.first, stride = (int64_t)c.H * D;    // (row of the block's token 0)
  for (int item = blockIdx.y * kWaves + wave; item < 2 * c.H; item += gridDim.y * kWaves) {
    const bool values = item & 1;
    const int h = item >> 1;
    const size_t block = p.page >= 0 ? block_of(c, p.page, h, p.sb) : 0;
    const uint8_t* at = (values ? c.v : c.k) + block * (16 * D);
    float scale = (values ? c.v_scale : c.k_scale)[block];
    if (p.page < 0) scale = __builtin_nanf("");
    T* to = (values ? v : k) + (size_t)h * D;
    if (!values) {
      uint2 q[2 * kC];
#pragma unroll
      for (int u = 0; u < 2 * kC; ++u)
        q[u] = *reinterpret_cast<const uint2*>(at + Unit(D, lane + 64 * u).at());
#pragma unroll
      for (int u = 0; u < 2 * kC; ++u) {
        const Unit unit(D, lane + 64 * u);
        const int i = unit.token;
        const f4 a = bytes4(q[u].x) * scale, b = bytes4(q[u].y) * scale;
        T* p8 = to + (row0 + i) * stride + 8 * unit.eighth;
        if (i >= from && i < end) {
          if constexpr (sizeof(T) == 2) {
            *reinterpret_cast<Row<T, 8>*>(p8) = __builtin_convertvector(__builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7), Row<T, 8>);
          } else {
            store4(p8, a);
            store4(p8 + 4, b);
          }
        }
      }
    } else {
      u4 q[kC];
#pragma unroll
      for (int u = 0; u < kC; ++u)
        q[u] = *reinterpret_cast<const u4*>(at + 16 * min(lane + 64 * u, D - 1));
      lds_order();
#pragma unroll
      for (int u = 0; u < kC; ++u)
        *reinterpret_cast<u4*>(bytes + feature_at(lane + 64 * u)) = q[u];
      lds_order();
#pragma unroll
      for (int u = 0; u < kC; ++u) {
        const int unit = lane + 64 * u, f = 4 * (unit >> 2);
        u4 w;
#pragma unroll
        for (int j = 0; j < 4; ++j) w[j] = *reinterpret_cast<const uint32_t*>(bytes + feature_at(f + j) + 4 * (unit & 3));
        w = turn4(w);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int i = 4 * (unit & 3) + j;
          if (f < D && i >= from && i < end) put4(to + (row0 + i) * stride + f, w[j], scale);
        }
      }
    }
  }
}

// Blocks that T rows of S sequences lie in, at most: a sequence of n has no
// more than (n + 30) / 16, and no more than n.
int64_t most_blocks(const CacheArgs& c) {
  const int64_t t = c.T;
  return std::min<int64_t>(t, t / 16 + 2 * (int64_t)c.S);
}

// Blocks across, and the heads of a block over as many workgroups as fill the chip, or
// two items (keys or values of a head) a wave where there are blocks enough.
dim3 grid_of(const CacheArgs& c, int64_t blocks) {
  const int64_t most = (2 * c.H + kWaves - 1) / kWaves, want = (8 * kCUs + blocks - 1) / blocks;
  return dim3((unsigned)blocks, (unsigned)std::min(most, std::max(want, (most + 1) / 2)));
}

template <typename F>
void by_shape(const CacheArgs& c, F f) {
  auto width = [&](auto t) {
    switch ((c.D + 63) / 64) {
      case 1: return f(t, std::integral_constant<int, 1>{});
      case 2: return f(t, std::integral_constant<int, 2>{});
      case 3: return f(t, std::integral_constant<int, 3>{});
      default: return f(t, std::integral_constant<int, 4>{});
    }
  };
  if (c.dtype == SHERRY_F32) width(float{});
  else if (c.dtype == SHERRY_F16) width(_Float16{});
  else width(__bf16{});
}

}  // namespace

hipError_t launch_cache_write(const CacheArgs& c, hipStream_t stream) {
  by_shape(c, [&](auto t, auto u) {
    cache_write_kernel<decltype(t), decltype(u)::value><<<grid_of(c, most_blocks(c)), 64 * kWaves, 0, stream>>>(c);
  });
  return hipGetLastError();
}

hipError_t launch_cache_read(const CacheArgs& c, void* k, void* v, hipStream_t stream) {
  by_shape(c, [&](auto t, auto u) {
    using T = decltype(t);
    cache_read_kernel<T, decltype(u)::value>
        <<<grid_of(c, most_blocks(c)), 64 * kWaves, 0, stream>>>(c, static_cast<T*>(k), static_cast<T*>(v));
  });
  return hipGetLastError();
}

}  // namespace sherry
