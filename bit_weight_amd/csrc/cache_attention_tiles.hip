// Attention over the 8-bit cache for many queries a sequence (prompts): see
// cache_attention.hip for the formula and the operands.
//
// A unit is a head's tile of 128 rows (tokens and the query heads that share the
// head), four waves of 32 rows.  The workgroup turns 64 tokens' keys and values
// to fp16 once for all rows, into one of two LDS buffers, while it computes on
// the other; the next tokens' bytes are in flight meanwhile.  Two workgroups a
// CU, not in step with each other, so one's matrix products run under the
// other's exponentials.
//
// Products are 32 x 32: lane (query i, half f) of keys times queries holds 16
// scores of one query.  Keys lie in LDS with the rows of a 16-token block dealt so
// that these are tokens 8 f .. 8 f + 7 of two blocks: the operand of the product
// with the values from the same lane.  A block's key scale is part of its scores'
// factor, its value scale (over the largest so far, a power of two) part of its
// weights' exponent, and taken out of their sum again.
#include "sherry_attention.h"

namespace sherry {
namespace {

typedef float f16v __attribute__((ext_vector_type(16)));

constexpr int kWaves = 4;
constexpr int kThreads = 64 * kWaves;
constexpr int kWaveRows = 32;
constexpr int kRows = kWaves * kWaveRows;
constexpr int kLeast = 8;                // steps that a workgroup takes at least
constexpr int kPlanThreads = 1024;

constexpr int blocks_of_kernel(int kC) { return kC <= 2 ? 2 * kCUs : kCUs; }

__host__ __device__ inline size_t part_floats(int D) { return (size_t)kRows * (D + 2); }

__device__ __forceinline__ int tiles_of(const AttentionArgs& a, const Rows& r) {
  return (r.n * (a.Hq / a.c.H) + kRows - 1) / kRows;
}

// A tile's query positions and steps.
struct Tile {
  int low, high;
  __device__ __forceinline__ Tile(const AttentionArgs& a, const Rows& r, int tile) {
    const int group = a.Hq / a.c.H, first = r.len - r.n;
    low = first + kRows * tile / group;
    high = first + min((kRows * tile + kRows - 1) / group, r.n - 1);
  }
  __device__ __forceinline__ Steps steps(const AttentionArgs& a) const { return Steps(a, low, high); }
};

// Where workgroup w begins: a step of a unit.  Units follow each other by sequence,
// head and tile; all their steps are dealt evenly to `used` workgroups.
struct Start {
  int seq, head, tile, step;
};
struct Plan {
  int64_t total;
  int used;
  int pad;
  __device__ __forceinline__ int64_t first(int w) const { return total * w / used; }
};

// In scratch: the plan, where each workgroup begins, each sequence's steps (up to
// it, times the heads), then the units' parts.
struct Scratch {
  Plan* plan;
  Start* starts;
  int64_t* before;      // [S + 1]
  float* parts;
  __host__ __device__ Scratch(float* base, int blocks, int S) {
    char* p = reinterpret_cast<char*>(base);
    plan = reinterpret_cast<Plan*>(p);
    starts = reinterpret_cast<Start*>(p + 256);
    before = reinterpret_cast<int64_t*>(p + 256 + sizeof(Start) * (blocks + 1));
    const size_t at = 256 + sizeof(Start) * (blocks + 1) + sizeof(int64_t) * ((size_t)S + 1);
    parts = reinterpret_cast<float*>(p + (at + 255) / 256 * 256);
  }
};

// One workgroup: steps of each sequence (a wave a sequence, its lanes taking the
// tiles in turn), their running sum, and each workgroup's beginning.
__global__ __launch_bounds__(kPlanThreads) void attention_plan_kernel(AttentionArgs a, int blocks) {
  __shared__ int64_t parts[kPlanThreads / 64];
  const Scratch s(a.scratch, blocks, a.c.S);
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  for (int i = wave; i < a.c.S; i += kPlanThreads / 64) {
    const Rows r = rows_of(a.c, i);
    const int tiles = tiles_of(a, r);
    int64_t sum = 0;
    for (int t = lane; t < tiles; t += 64) sum += Tile(a, r, t).steps(a).count();
#pragma unroll
    for (int d = 1; d < 64; d *= 2) sum += ((int64_t)__shfl_xor((int)(sum >> 32), d) << 32) + (uint32_t)__shfl_xor((int)(uint32_t)sum, d);
    if (lane == 0) s.before[i + 1] = sum * a.c.H;
  }
  __threadfence_block();
  __syncthreads();
  int64_t total = 0;
  for (int base = 0; base < a.c.S; base += kPlanThreads) {
    const int i = base + threadIdx.x;
    const int64_t own = i < a.c.S ? s.before[i + 1] : 0;
    int64_t before;
    const int64_t all = block_scan<kPlanThreads / 64>(own, before, parts);
    if (i < a.c.S) s.before[i + 1] = total + before + own;
    total += all;
  }
  if (threadIdx.x == 0) s.before[0] = 0;
  __threadfence_block();
  __syncthreads();
  Plan plan{total, 0, 0};
  const int64_t most = (total + kLeast - 1) / kLeast;
  plan.used = (int)(most < blocks ? most : blocks);
  if (threadIdx.x == 0) *s.plan = plan;
  for (int w = threadIdx.x; w < plan.used; w += kPlanThreads) {
    const int64_t at = plan.first(w);
    int lo = 0, hi = a.c.S - 1;      // the last sequence whose steps begin at or before `at`
    while (lo < hi) {
      const int mid = (lo + hi + 1) / 2;
      if (s.before[mid] <= at) lo = mid;
      else hi = mid - 1;
    }
    const Rows r = rows_of(a.c, lo);
    const int64_t each = (s.before[lo + 1] - s.before[lo]) / a.c.H;
    int64_t rest = at - s.before[lo];
    Start b{lo, (int)(rest / each), 0, 0};
    rest -= b.head * each;
    for (;; ++b.tile) {
      const int count = Tile(a, r, b.tile).steps(a).count();
      if (rest < count) break;
      rest -= count;
    }
    b.step = (int)rest;
    s.starts[w] = b;
  }
}

// kC: D / 64 rounded up.
template <int kC>
struct Layout {
  static constexpr int kChunks = 8 * kC;                  // of 8 features, in a key's row
  static constexpr int kKeys = kStep * 64 * kC * 2;       // bytes of 64 tokens' keys as fp16 (and of values)
  static constexpr int kBuffer = 2 * kKeys;
  // 16 bytes `chunk` of key row `row`: sixteen rows of the same chunk lie in different banks
  static __device__ __forceinline__ int key(int row, int chunk) {
    return 16 * (row * kChunks + (kChunks % 16 == 0 ? chunk ^ (row & 15) : chunk ^ ((row >> 1) & 7)));
  }
  // 8 tokens `chunk` of feature `row`
  static __device__ __forceinline__ int value(int row, int chunk) { return kKeys + 16 * (8 * row + (chunk ^ ((row >> 1) & 7))); }
};

// kTerms: fp16 terms of q and of the weights.
template <int kC, int kTerms>
__global__ __launch_bounds__(kThreads, kC <= 2 ? 2 : 1) void attention_tiles_kernel(AttentionArgs a, int blocks) {
  using L = Layout<kC>;
  constexpr int kTiles = 2 * kC;          // of 32 features
  constexpr int kLoads = kC;              // 16-byte units of a thread, of keys and of values each
  __shared__ __attribute__((aligned(1024))) char lds[2 * L::kBuffer];
  __shared__ float scales[2][8];          // of the buffers' four blocks: keys, values
  const Scratch scratch(a.scratch, blocks, a.c.S);
  // neighbours in the deal share keys: give each XCD a run of them
  const int block = (blockIdx.x & 7) * (blocks / 8) + (blockIdx.x >> 3);
  const Plan plan = *scratch.plan;
  if (block >= plan.used) return;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, i = lane & 31, f = lane >> 5;
  const int D = a.c.D, pieces = D / 16, group = a.Hq / a.c.H;
  const float sign = a.scale < 0.0f ? -1.0f : 1.0f;
  int64_t left = plan.first(block + 1) - plan.first(block);
  Start at = scratch.starts[block];
  Rows r = rows_of(a.c, at.seq);
  int tiles = tiles_of(a, r);
  bool first_part = true;

  while (left > 0) {
    const Tile tile(a, r, at.tile);
    const Steps steps = tile.steps(a);
    const int count = steps.count(), s0 = at.step, s1 = (int)min((int64_t)count, s0 + left), h = at.head;

    // queries: features 16 c + 8 f .. of row i
    const int row = kRows * at.tile + kWaveRows * wave + i, token = row / group;
    const bool in = token < r.n;
    const int pos = in ? r.len - r.n + token : -1;
    h8 q[kTerms][4 * kC];
    float factor;
    {
      const size_t from = (size_t)(r.row0 + (in ? token : 0)) * a.q_stride +
                          (size_t)(h * group + (in ? row - token * group : 0)) * D + 8 * f;
      float top = 0.0f;
      f4 raw[4 * kC][2];
#pragma unroll
      for (int c = 0; c < 4 * kC; ++c)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          raw[c][j] = f4{};
          if (in && c < pieces) raw[c][j] = load4_as(a.q, from + 16 * c + 4 * j, a.c.dtype);
#pragma unroll
          for (int b = 0; b < 4; ++b) top = fmaxf(top, fabsf(raw[c][j][b]));
        }
      top = fmaxf(top, __shfl_xor(top, 32));
      const float times = row_scale(top) * sign;
      factor = a.scale * kLog2E / times;        // (positive: the sign is in q)
      if (r.len > room_of(a)) factor = __builtin_nanf("");
#pragma unroll
      for (int c = 0; c < 4 * kC; ++c)
#pragma unroll
        for (int b = 0; b < 8; ++b) {
          const float v = raw[c][b / 4][b % 4] * times;
          const _Float16 hi = (_Float16)v;
          q[0][c][b] = hi;
          if constexpr (kTerms == 2) q[kTerms - 1][c][b] = (_Float16)(v - (float)hi);
        }
    }

    // bytes of a step: unit x of block u is 16 features of a token, or 16 tokens of a feature
    uint4 kw[kLoads], vw[kLoads];
    float ks[kLoads], vs[kLoads];
    auto load = [&](int s) {
      const int ts = steps.at(s);
#pragma unroll
      for (int n = 0; n < kLoads; ++n) {
        const int x = tid + kThreads * n, u = x / D, y = x - u * D;
        if (u >= 4) continue;
        const int page = page_of(a.c, at.seq, 4 * ts + u);
        const size_t b = block_of(a.c, max(page, 0), h, 4 * ts + u);
        kw[n] = *reinterpret_cast<const uint4*>(a.c.k + b * (16 * D) + 16 * y);
        vw[n] = *reinterpret_cast<const uint4*>(a.c.v + b * (16 * D) + 16 * y);
        ks[n] = page < 0 ? __builtin_nanf("") : a.c.k_scale[b];
        vs[n] = a.c.v_scale[b];
      }
    };
    auto convert = [&](int s) {
      char* to = lds + (s & 1) * L::kBuffer;
#pragma unroll
      for (int n = 0; n < kLoads; ++n) {
        const int x = tid + kThreads * n, u = x / D, y = x - u * D;
        if (u >= 4) continue;
        const int piece = y >> 4, t = y & 15;
        // token 8 f + 4 s + r of the block is row 8 s + 4 f + r
        const int key = 16 * u + ((t & 3) | ((t & 4) << 1) | ((t & 8) >> 1));
        *reinterpret_cast<h8*>(to + L::key(key, 2 * piece)) = halves8(kw[n].x, kw[n].y);
        *reinterpret_cast<h8*>(to + L::key(key, 2 * piece + 1)) = halves8(kw[n].z, kw[n].w);
        *reinterpret_cast<h8*>(to + L::value(y, 2 * u)) = halves8(vw[n].x, vw[n].y);
        *reinterpret_cast<h8*>(to + L::value(y, 2 * u + 1)) = halves8(vw[n].z, vw[n].w);
        if (y == 0) {
          scales[s & 1][u] = vs[n] == vs[n] ? ks[n] : __builtin_nanf("");
          scales[s & 1][4 + u] = vs[n];
        }
      }
    };

    float m = -__builtin_inff(), l = 0.0f, unit = 0x1p-126f;
    f16v o[kTiles];
#pragma unroll
    for (int t = 0; t < kTiles; ++t) o[t] = f16v{};

    load(s0);
    convert(s0);
    if (s0 + 1 < s1) load(s0 + 1);
    lds_barrier();
    for (int s = s0; s < s1; ++s) {
      if (s + 1 < s1) convert(s + 1);
      if (s + 2 < s1) load(s + 2);
      const char* from = lds + (s & 1) * L::kBuffer;
      const int t0 = kStep * steps.at(s);
      f16v sc[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        sc[e] = f16v{};
#pragma unroll
        for (int c = 0; c < 4 * kC; ++c)
          if (c < pieces) {
            const h8 k = *reinterpret_cast<const h8*>(from + L::key(32 * e + i, 2 * c + f));
#pragma unroll
            for (int n = 0; n < kTerms; ++n) sc[e] = __builtin_amdgcn_mfma_f32_32x32x16_f16(k, q[n][c], sc[e], 0, 0, 0);
          }
      }
      const bool all = sees_all(a, t0, tile.low, tile.high);
      if (!all) {
#pragma unroll
        for (int e = 0; e < 2; ++e)
#pragma unroll
          for (int b = 0; b < 16; ++b)
            if (!sees(a, t0 + 32 * e + 16 * (b / 8) + 8 * f + b % 8, pos)) sc[e][b] = -__builtin_inff();
      }
      // blocks: factor of the scores, largest score, value scale
      float by[4], vscale[4], top = -__builtin_inff(), unit_now = unit;
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        by[u] = factor * scales[s & 1][u];
        vscale[u] = scales[s & 1][4 + u];
        float best = sc[u / 2][8 * (u % 2)];
#pragma unroll
        for (int b = 1; b < 8; ++b) best = fmaxf(best, sc[u / 2][8 * (u % 2) + b]);
        top = fmaxf(top, best == -__builtin_inff() ? best : best * by[u]);
        if (t0 + 16 * u <= tile.high && vscale[u] < __builtin_inff()) unit_now = fmaxf(unit_now, vscale[u]);
      }
      top = fmaxf(top, __shfl_xor(top, 32));
      if (__any(top > m + kSlack) || unit_now > unit) {
        const float now = fmaxf(m, top);
        const float keep = __builtin_amdgcn_exp2f(m - above(now)), scaled = keep * unit * __builtin_amdgcn_rcpf(unit_now);
        l *= keep;
#pragma unroll
        for (int t = 0; t < kTiles; ++t) o[t] *= scaled;
        m = now;
        unit = unit_now;
      }
      const float base = above(m) - kWeightExponent, inverse = __builtin_amdgcn_rcpf(unit);
      h8 p[kTerms][4];
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        // the weights times the value scale over `unit`; below 2^-40 of it they count in the sum alone
        const float ratio = vscale[u] * inverse;
        const bool counts = ratio >= 0x1p-40f;
        const float from_base = counts ? base - __builtin_amdgcn_logf(ratio) : base;
        float sum = 0.0f;
#pragma unroll
        for (int b = 0; b < 8; ++b) {
          const float raw = sc[u / 2][8 * (u % 2) + b];
          float e = __builtin_amdgcn_exp2f(fmaf(raw, by[u], -from_base));
          if (!all) e = raw == -__builtin_inff() ? 0.0f : e;
          sum += e;
          const float v = counts ? e : 0.0f;
          const _Float16 hi = (_Float16)v;
          p[0][u][b] = hi;
          if constexpr (kTerms == 2) p[kTerms - 1][u][b] = (_Float16)(v - (float)hi);
        }
        l += counts ? sum * __builtin_amdgcn_rcpf(ratio) : sum;
      }
#pragma unroll
      for (int t = 0; t < kTiles; ++t)
        if (2 * t < pieces) {
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            const h8 v = *reinterpret_cast<const h8*>(from + L::value(32 * t + i, 2 * u + f));
#pragma unroll
            for (int n = 0; n < kTerms; ++n) o[t] = __builtin_amdgcn_mfma_f32_32x32x16_f16(v, p[n][u], o[t], 0, 0, 0);
          }
        }
      lds_barrier();
    }

    l += __shfl_xor(l, 32);
    const float times = l == 0.0f ? 0.0f : unit / l;
    const bool whole = s0 == 0 && s1 == count;
    const float lse2 = m - kWeightExponent + __builtin_amdgcn_logf(l);
    if (whole) {
      if (in) {
        const size_t to = (size_t)(r.row0 + token) * a.Hq + h * group + row - token * group;
#pragma unroll
        for (int t = 0; t < kTiles; ++t)
#pragma unroll
          for (int b = 0; b < 4; ++b) {
            const int d = 32 * t + 8 * b + 4 * f;
            if (d < D)
              store4_as(a.y, to * D + d, a.c.dtype, f4{o[t][4 * b], o[t][4 * b + 1], o[t][4 * b + 2], o[t][4 * b + 3]} * times);
          }
        if (a.lse && f == 0) a.lse[to] = lse2 * kLn2;
      }
    } else {
      float* part = scratch.parts + (size_t)(2 * block + (first_part ? 0 : 1)) * part_floats(D);
      const int line = kWaveRows * wave + i;
#pragma unroll
      for (int t = 0; t < kTiles; ++t)
#pragma unroll
        for (int b = 0; b < 4; ++b) {
          const int d = 32 * t + 8 * b + 4 * f;
          if (d < D)
            *reinterpret_cast<f4*>(part + (size_t)line * D + d) =
                f4{o[t][4 * b], o[t][4 * b + 1], o[t][4 * b + 2], o[t][4 * b + 3]} * times;
        }
      if (f == 0) part[kRows * D + line] = lse2;
    }
    left -= s1 - s0;
    first_part = false;
    at.step = 0;
    if (++at.tile == tiles) {
      at.tile = 0;
      if (++at.head == a.c.H) {
        at.head = 0;
        do {
          ++at.seq;
          if (at.seq >= a.c.S) break;
          r = rows_of(a.c, at.seq);
          tiles = tiles_of(a, r);
        } while (tiles == 0);
      }
    }
  }
}

// Joins the units that several workgroups had.  Block w looks after the unit that
// begins in workgroup w and does not end there, if there is one; blocks y of it
// share the rows.
__global__ __launch_bounds__(kThreads) void attention_tiles_join_kernel(AttentionArgs a, int blocks) {
  const Scratch scratch(a.scratch, blocks, a.c.S);
  const int w = blockIdx.x, D = a.c.D, group = a.Hq / a.c.H;
  const Plan plan = *scratch.plan;
  if (w + 1 >= plan.used) return;
  const Start next = scratch.starts[w + 1], own = scratch.starts[w];
  if (next.step == 0) return;                                  // the workgroup ends with its unit
  const bool same = own.seq == next.seq && own.head == next.head && own.tile == next.tile;
  if (same && own.step > 0) return;                            // the unit began before
  const Rows r = rows_of(a.c, next.seq);
  const Tile tile(a, r, next.tile);
  const int count = tile.steps(a).count();
  int parts = 1;                                               // of workgroups w .. w + parts - 1
  for (int64_t done = next.step; done < count; ++parts) done += plan.first(w + parts + 1) - plan.first(w + parts);
  auto part = [&](int n) {
    return scratch.parts + (size_t)(n == 0 ? 2 * w + (same ? 0 : 1) : 2 * (w + n)) * part_floats(D);
  };
  const int quads = D / 4, per = (kRows + gridDim.y - 1) / gridDim.y, line0 = per * blockIdx.y;
  for (int x = threadIdx.x; x < per * quads; x += kThreads) {
    const int line = line0 + x / quads, d = 4 * (x % quads), row = kRows * next.tile + line, token = row / group;
    if (line >= kRows || token >= r.n) continue;
    float m = -__builtin_inff(), l = 0.0f;
    for (int n = 0; n < parts; ++n) m = fmaxf(m, part(n)[kRows * D + line]);
    f4 y{};
    for (int n = 0; n < parts; ++n) {
      const float e = __builtin_amdgcn_exp2f(part(n)[kRows * D + line] - above(m));
      l += e;
      y += e * *reinterpret_cast<const f4*>(part(n) + (size_t)line * D + d);
    }
    y = l == 0.0f ? f4{} : y / l;
    const size_t to = (size_t)(r.row0 + token) * a.Hq + next.head * group + row - token * group;
    store4_as(a.y, to * D + d, a.c.dtype, y);
    if (a.lse && d == 0) a.lse[to] = (m + __builtin_amdgcn_logf(l)) * kLn2;
  }
}

template <int kC, int kTerms>
hipError_t launch_tiles(const AttentionArgs& a, hipStream_t stream) {
  constexpr int blocks = blocks_of_kernel(kC);
  attention_tiles_kernel<kC, kTerms><<<blocks, kThreads, 0, stream>>>(a, blocks);
  return hipGetLastError();
}

template <int kTerms>
hipError_t launch_terms(const AttentionArgs& a, hipStream_t stream) {
  switch ((a.c.D + 63) / 64) {
    case 1: return launch_tiles<1, kTerms>(a, stream);
    case 2: return launch_tiles<2, kTerms>(a, stream);
    case 3: return launch_tiles<3, kTerms>(a, stream);
    default: return launch_tiles<4, kTerms>(a, stream);
  }
}

}  // namespace

size_t attention_tiles_scratch_bytes(int S, int D) {
  const int blocks = blocks_of_kernel((D + 63) / 64);
  const Scratch s(nullptr, blocks, S);
  return reinterpret_cast<size_t>(s.parts) + 2 * blocks * part_floats(D) * sizeof(float);
}

hipError_t launch_attention_tiles(const AttentionArgs& a, hipStream_t stream, bool* partial) {
  const int blocks = blocks_of_kernel((a.c.D + 63) / 64);
  attention_plan_kernel<<<1, kPlanThreads, 0, stream>>>(a, blocks);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  *partial = true;
  e = a.c.dtype == SHERRY_F32 ? launch_terms<2>(a, stream) : launch_terms<1>(a, stream);
  if (e != hipSuccess) return e;
  attention_tiles_join_kernel<<<dim3(blocks, 4), kThreads, 0, stream>>>(a, blocks);
  return hipGetLastError();
}

}  // namespace sherry
