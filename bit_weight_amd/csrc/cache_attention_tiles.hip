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
// factor.  Its value scale, over the largest that the query has seen so far (a power of
// two), goes into the query's weights and not into the values, which all queries share:
// no result depends on the scale of tokens that its query does not see.
//
// Measured: pieces of up to 1024 tokens of 4 prompts over up to 6000, 32 heads over 8 of
// 128 in bf16, 2.2e11 operations, in 308 us of which the deal is 9 and the join of parts
// 19 (0.70 PFLOP/s; the library's fp16 product reaches 1.52).  The main kernel's matrix
// units are busy 34 % of the time, the vector units 52 % (8-bit values to fp16,
// exponentials, masks), LDS 36 %: no unit is full, waits and the phases' unevenness are
// the rest.  Value scales in the weights instead of the values cost 8 us of it.  Two terms
// of the weights (fp16): 397 us, of q too (fp32, where 72 registers spill): 570.  Tiles of
// 64 rows: 448 us.
#include "sherry_attention.h"

namespace sherry {
namespace {

typedef float f16v __attribute__((ext_vector_type(16)));

constexpr int kWaves = 4;
constexpr int kThreads = 64 * kWaves;
constexpr int kWaveRows = 32;
constexpr int kRows = kWaves * kWaveRows;
constexpr int kLeast = 4;                // steps that a workgroup takes at least
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
  __device__ __forceinline__ int64_t first(int w) const { return quotient(total * w, used); }
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
  __shared__ int64_t parts[kPlanThreads / 64], near[kPlanThreads + 1];
  const Scratch s(a.scratch, blocks, a.c.S);
  int64_t* before = a.c.S <= kPlanThreads ? near : s.before;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  for (int i = wave; i < a.c.S; i += kPlanThreads / 64) {
    const Rows r = rows_of(a.c, i);
    const int tiles = tiles_of(a, r);
    int64_t sum = 0;
    for (int t = lane; t < tiles; t += 64) sum += Tile(a, r, t).steps(a).count();
#pragma unroll
    for (int d = 1; d < 64; d *= 2) sum += ((int64_t)__shfl_xor((int)(sum >> 32), d) << 32) + (uint32_t)__shfl_xor((int)(uint32_t)sum, d);
    if (lane == 0) before[i + 1] = sum * a.c.H;
  }
  __threadfence_block();
  __syncthreads();
  int64_t total = 0;
  for (int base = 0; base < a.c.S; base += kPlanThreads) {
    const int i = base + threadIdx.x;
    const int64_t own = i < a.c.S ? before[i + 1] : 0;
    int64_t earlier;
    const int64_t all = block_scan<kPlanThreads / 64>(own, earlier, parts);
    if (i < a.c.S) before[i + 1] = total + earlier + own;
    total += all;
  }
  if (threadIdx.x == 0) before[0] = 0;
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
      if (before[mid] <= at) lo = mid;
      else hi = mid - 1;
    }
    const Rows r = rows_of(a.c, lo);
    const int64_t each = (before[lo + 1] - before[lo]) / a.c.H;
    int64_t rest = at - before[lo];
    Start b{lo, (int)(rest / each), 0, 0};
    rest -= b.head * each;
    // tiles one after another, their first and last queries as Tile has them, with no division
    const int group = a.Hq / a.c.H, first = r.len - r.n, whole = kRows / group, over = kRows % group;
    int low = 0, low_over = 0, high = (kRows - 1) / group, high_over = (kRows - 1) % group;
    for (;; ++b.tile) {
      const int count = Steps(a, first + low, first + min(high, r.n - 1)).count();
      if (rest < count) break;
      rest -= count;
      low += whole;
      high += whole;
      if ((low_over += over) >= group) low_over -= group, ++low;
      if ((high_over += over) >= group) high_over -= group, ++high;
    }
    b.step = (int)rest;
    s.starts[w] = b;
  }
}

// kC: D / 64 rounded up.
template <int kC>
struct Layout {
  // of 8 features, in a key's row: a power of two, so that chunks differ in an exclusive or
  static constexpr int kChunks = kC == 3 ? 32 : 8 * kC;
  static constexpr int kKeys = kStep * kChunks * 16;      // bytes of 64 tokens' keys as fp16
  static constexpr int kBuffer = kKeys + kStep * 64 * kC * 2;
  // 16 bytes `chunk` of key row `row`: sixteen rows of the same chunk lie in different banks
  static __device__ __forceinline__ int key(int row, int chunk) {
    return 16 * (row * kChunks + (kChunks % 16 == 0 ? chunk ^ (row & 15) : chunk ^ ((row >> 1) & 7)));
  }
  // 8 tokens `chunk` of feature `row`
  static __device__ __forceinline__ int value(int row, int chunk) { return kKeys + 16 * (8 * row + (chunk ^ ((row >> 1) & 7))); }
};

// kTerms, kWeights: fp16 terms of q and of the weights.
template <int kC, int kTerms, int kWeights>
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
  const int tid = threadIdx.x, lane = tid & 63, wave = uniform(tid >> 6), i = lane & 31, f = lane >> 5;
  const int D = a.c.D, pieces = D / 16, group = a.Hq / a.c.H;
  const float sign = a.scale < 0.0f ? -1.0f : 1.0f;
  // (features past D stay zeros, and the first product with the values meets no stray NaN)
  for (int x = 16 * tid; x < 2 * L::kBuffer; x += 16 * kThreads) *reinterpret_cast<uint4*>(lds + x) = uint4{};

  // Each wave brings one block of a step: its 16-byte units `lane + 64 n` (the last
  // one several times where there are fewer than lanes), and where they go as fp16.
  int unit_at[kLoads], key_at[kLoads], value_at[kLoads];
#pragma unroll
  for (int n = 0; n < kLoads; ++n) {
    const int y = min(lane + 64 * n, D - 1), t = y & 15;
    unit_at[n] = 16 * y;
    // token 8 f + 4 s + r of the block is row 8 s + 4 f + r
    key_at[n] = L::key(16 * wave + ((t & 3) | ((t & 4) << 1) | ((t & 8) >> 1)), 2 * (y >> 4));
    value_at[n] = L::value(y, 2 * wave);
  }
  int64_t left = uniform64(plan.first(block + 1) - plan.first(block));
  const Start start = scratch.starts[block];
  int seq = uniform(start.seq), h = uniform(start.head), tile_number = uniform(start.tile), s0 = uniform(start.step);
  Rows r = uniform(rows_of(a.c, seq));
  int tiles = tiles_of(a, r);
  bool first_part = true;

  while (left > 0) {
    const Tile tile(a, r, tile_number);
    const Steps steps = tile.steps(a);
    const int count = steps.count(), s1 = (int)min((int64_t)count, s0 + left);

    // A step's page, then its scales and bytes, then those as fp16 in a buffer: each is
    // asked for a step before the next needs it.  Steps past the last are the last one
    // again, so that nothing here branches.
    const int32_t* table = a.c.table + (size_t)seq * a.c.table_width;
    const uint32_t page_blocks = (uint32_t)a.c.H << a.c.block_shift, h_blocks = (uint32_t)h << a.c.block_shift;
    const int in_page = (1 << a.c.block_shift) - 1, window_shift = steps.from - steps.head;
    int page_next, page_after;       // of the blocks to be asked for next
    uint32_t block_now, block_next;  // blocks (fewer than 2^31 in a cache) whose values, and keys, are asked for next
    bool good;
    uint4 kw[kLoads], vw[kLoads];
    float ks, vs;
    auto step_at = [&](int s) {
      s = min(s, s1 - 1);
      return s < steps.head ? s : s + window_shift;
    };
    auto page_of_step = [&](int s) { return table[min((4 * step_at(s) + wave) >> a.c.block_shift, a.c.table_width - 1)]; };
    auto find_block = [&](int s) {
      const int sb = 4 * step_at(s) + wave;
      const uint32_t p = uniform(page_next);
      good = p < (uint32_t)a.c.pages && sb >> a.c.block_shift < a.c.table_width;
      block_next = (good ? p : 0) * page_blocks + h_blocks + (sb & in_page);
    };
    auto load_keys = [&]() {
      const uint8_t* from = a.c.k + (uint64_t)block_next * (uint32_t)(16 * D);
#pragma unroll
      for (int n = 0; n < kLoads; ++n) kw[n] = *reinterpret_cast<const uint4*>(from + (uint32_t)unit_at[n]);
      ks = a.c.k_scale[block_next];
      vs = a.c.v_scale[block_next];
      if (!good) ks = __builtin_nanf(""), vs = 0.0f;
    };
    auto load_values = [&]() {
      const uint8_t* from = a.c.v + (uint64_t)block_now * (uint32_t)(16 * D);
#pragma unroll
      for (int n = 0; n < kLoads; ++n) vw[n] = *reinterpret_cast<const uint4*>(from + (uint32_t)unit_at[n]);
    };
    // a block that is not valid has a key scale of NaN; one that is not or whose scale is
    // not finite a value scale of 0
    auto store_scales = [&](int buffer) {
      const float k = vs == vs ? ks : vs, v = vs < __builtin_inff() ? vs : 0.0f;
      if (lane < 2) scales[buffer][4 * lane + wave] = lane ? v : k;
    };
    // 8 of a thread's keys, or of its values
    auto store_keys = [&](int buffer, int n, int half) {
      *reinterpret_cast<h8*>(lds + buffer + (key_at[n] ^ (16 * half))) =
          half ? halves8(kw[n].z, kw[n].w) : halves8(kw[n].x, kw[n].y);
    };
    auto store_values = [&](int buffer, int n, int half) {
      *reinterpret_cast<h8*>(lds + buffer + (value_at[n] ^ (16 * half))) =
          half ? halves8(vw[n].z, vw[n].w) : halves8(vw[n].x, vw[n].y);
    };

    // maximum, this lane's part of the sum (NaN for all of a sequence longer than its
    // table, also where a window hides what the table has room for), largest value scale
    // that the query has seen, features of the output in `unit`
    float m = -__builtin_inff(), l = r.len > room_of(a) ? __builtin_nanf("") : 0.0f, unit = 0x1p-126f;
    f16v o[kTiles];
#pragma unroll
    for (int t = 0; t < kTiles; ++t) o[t] = f16v{};
    h8 p[kWeights][4];           // the last step's weights
#pragma unroll
    for (int n = 0; n < kWeights; ++n)
#pragma unroll
      for (int u = 0; u < 4; ++u) p[n][u] = h8{};
    // The products in slots: their operands from LDS are read kAhead slots before, and
    // each slot brings a share of other work for the vector units (`beside`).
    constexpr int kSlots = 8 * kC, kAhead = 4;
    auto in_slots = [&](auto read, auto product, auto beside) {
      h8 operand[kAhead];
#pragma unroll
      for (int j = 0; j < kAhead; ++j) operand[j] = read(j);
#pragma unroll
      for (int j = 0; j < kSlots; ++j) {
        product(j, operand[j % kAhead]);
        if (j + kAhead < kSlots) operand[j % kAhead] = read(j + kAhead);
        beside(j);
        __builtin_amdgcn_sched_barrier(0);
      }
    };
    // LDS addresses: a row's chunks differ in one exclusive or, rows and buffers in the offset
    const int key_row = L::key(i, f), value_row = L::value(i, f);
    auto add_values = [&](int buffer, auto beside) {
      const int base = value_row + buffer;
      in_slots([&](int j) { return *reinterpret_cast<const h8*>(lds + (base ^ (32 * (j / kTiles))) + 4096 * (j % kTiles)); },
               [&](int j, h8 v) {
#pragma unroll
                 for (int n = 0; n < kWeights; ++n)
                   o[j % kTiles] = __builtin_amdgcn_mfma_f32_32x32x16_f16(v, p[n][j / kTiles], o[j % kTiles], 0, 0, 0);
               },
               beside);
    };

    page_next = page_of_step(s0);
    page_after = page_of_step(s0 + 1);
    find_block(s0);
    load_keys();
    block_now = block_next;
    load_values();
    page_next = page_after;
    page_after = page_of_step(s0 + 2);

    // queries: features 16 c + 8 f .. of row i
    const int row = kRows * tile_number + kWaveRows * wave + i, token = row / group;
    const bool in = token < r.n;
    const int pos = in ? r.len - r.n + token : -1;
    h8 q[kTerms][4 * kC];
    float factor;
    {
      const size_t from = (size_t)(r.row0 + (in ? token : 0)) * a.q_stride +
                          (size_t)(h * group + (in ? row - token * group : 0)) * D + 8 * f;
      float top = 0.0f;
      RawValues<2> bytes[4 * kC];
#pragma unroll
      for (int c = 0; c < 4 * kC; ++c) bytes[c].load(a.q, from + 16 * min(c, pieces - 1), a.c.dtype);
      auto value = [&](int c, int j) { return in && c < pieces ? bytes[c].get(j, a.c.dtype) : f4{}; };
#pragma unroll
      for (int c = 0; c < 4 * kC; ++c)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const f4 x = value(c, j);
#pragma unroll
          for (int b = 0; b < 4; ++b) top = fmaxf(top, fabsf(x[b]));
        }
      top = fmaxf(top, __shfl_xor(top, 32));
      const float times = row_scale(top) * sign;
      factor = a.scale * kLog2E / times;        // (positive: the sign is in q)
#pragma unroll
      for (int c = 0; c < 4 * kC; ++c)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const f4 x = value(c, j) * times;
#pragma unroll
          for (int b = 0; b < 4; ++b) {
            const _Float16 hi = (_Float16)x[b];
            q[0][c][4 * j + b] = hi;
            if constexpr (kTerms == 2) q[kTerms - 1][c][4 * j + b] = (_Float16)(x[b] - (float)hi);
          }
        }
    }

    lds_barrier();               // (the zeros, or what the last unit reads)
    store_scales(0);
#pragma unroll
    for (int n = 0; n < 2 * kLoads; ++n) store_keys(0, n / 2, n % 2);
    find_block(s0 + 1);
    load_keys();
    block_now = block_next;
    page_next = page_after;
    page_after = page_of_step(s0 + 3);
    lds_barrier();
    // In step s: its scores, while the next keys and its values are turned to fp16; then
    // its weights, while the last step's meet their values.
    for (int s = s0, buffer = 0; s < s1; ++s, buffer ^= 1) {
      const int here = buffer * L::kBuffer, there = L::kBuffer - here;
      const int t0 = kStep * step_at(s);
      float by[4], value_scale[4];        // a block's; by: the factor of its scores
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        by[u] = factor * scales[buffer][u];
        value_scale[u] = scales[buffer][4 + u];
      }
      f16v sc[2] = {f16v{}, f16v{}};
      store_scales(buffer ^ 1);
      const int base = key_row + here;
      in_slots([&](int j) { return *reinterpret_cast<const h8*>(lds + (base ^ (32 * (j / 2))) + 32 * 16 * L::kChunks * (j % 2)); },
               [&](int j, h8 k) {
#pragma unroll
                 for (int n = 0; n < kTerms; ++n)
                   sc[j % 2] = __builtin_amdgcn_mfma_f32_32x32x16_f16(k, q[n][j / 2], sc[j % 2], 0, 0, 0);
               },
               [&](int j) {
                 if (j % 2) return;
                 const int n = j / 8, part = j / 2 % 4;
                 if (part < 2) store_keys(there, n, part);
                 else store_values(here, n, part - 2);
               });
      load_values();
      find_block(s + 2);
      load_keys();
      block_now = block_next;
      page_next = page_after;
      page_after = page_of_step(s + 4);
      float unit_now = unit;
      if (sees_all(a, t0, tile.low, tile.high)) {
#pragma unroll
        for (int u = 0; u < 4; ++u) unit_now = fmaxf(unit_now, value_scale[u]);
      } else {
        asm volatile("");       // (a branch, not 32 selections in every step)
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          // seen tokens of a block that is not valid give NaN, hidden ones nothing: no
          // factor of NaN, or of 0, may meet their -infinity
          const bool bad = by[u] != by[u];
          const int ahead = pos - (t0 + 16 * u + 8 * f);       // of the first of these tokens
          const int behind = pos - (t0 + 16 * u);              // of the block's first
          if (behind >= 0 && (a.window == 0 || behind - 15 < a.window || t0 + 16 * u < a.sinks))
            unit_now = fmaxf(unit_now, value_scale[u]);
#pragma unroll
          for (int b = 0; b < 8; ++b) {
            const float x = sc[u / 2][8 * (u % 2) + b];
            sc[u / 2][8 * (u % 2) + b] = ahead < b ? -__builtin_inff() : bad ? by[u] : x;
          }
          if (a.window > 0) {
#pragma unroll
            for (int b = 0; b < 8; ++b)
              if (ahead - b >= a.window && t0 + 16 * u + 8 * f + b >= a.sinks) sc[u / 2][8 * (u % 2) + b] = -__builtin_inff();
          }
          by[u] = bad ? 1.0f : fmaxf(by[u], 0x1p-120f);
        }
      }
      // weights under the maximum so far; where that is too low for them, or a query has
      // seen nothing yet, again under a new one
      float sum = 0.0f, ratio[4];
      h8 next[kWeights][4];
      // (a block that the query does not see may have any scale: its weights are 0)
      auto ratios = [&](float of) {
#pragma unroll
        for (int u = 0; u < 4; ++u) ratio[u] = fminf(value_scale[u] * __builtin_amdgcn_rcpf(of), 1.0f);
      };
      auto weight = [&](int x, float exponent) {
        const float e = __builtin_amdgcn_exp2f(exponent);
        sum += e;
        const float v = e * ratio[x / 8];
        const _Float16 hi = (_Float16)v;
        next[0][x / 8][x % 8] = hi;
        if constexpr (kWeights == 2) next[kWeights - 1][x / 8][x % 8] = (_Float16)(v - (float)hi);
      };
      ratios(unit);
      const float floor = above(m) - kWeightExponent;
      add_values(there, [&](int j) {
#pragma unroll
        for (int x = j * 32 / kSlots; x < (j + 1) * 32 / kSlots; ++x)
          weight(x, fmaf(sc[x / 16][x % 16], by[x / 8], -floor));
      });
      // (no weight is larger than their sum; one of at most 2^15 stays in fp16's range)
      if (__any(sum > 0x1p15f || (pos >= 0 && m == -__builtin_inff()) || unit_now > unit)) {
        float top = -__builtin_inff();
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          float best = sc[u / 2][8 * (u % 2)];
#pragma unroll
          for (int b = 1; b < 8; ++b) best = fmaxf(best, sc[u / 2][8 * (u % 2) + b]);
          top = fmaxf(top, best * by[u]);
        }
        const float now = fmaxf(m, fmaxf(top, __shfl_xor(top, 32)));
        const float keep = __builtin_amdgcn_exp2f(m - above(now)), scaled = keep * unit * __builtin_amdgcn_rcpf(unit_now);
        l *= keep;
#pragma unroll
        for (int t = 0; t < kTiles; ++t) o[t] *= scaled;
        m = now;
        unit = unit_now;
        sum = 0.0f;
        ratios(unit);
        // (the products rounded as the maximum is: a fused one would leave half a step of
        // the score, which from 2^28 on is more than a weight's exponent has room for)
        const float again = above(m) - kWeightExponent;
#pragma unroll
        for (int x = 0; x < 32; ++x) {
#pragma clang fp contract(off)
          const float score = sc[x / 16][x % 16] * by[x / 8];
          weight(x, score - again);
        }
      }
      l += sum;
#pragma unroll
      for (int n = 0; n < kWeights; ++n)
#pragma unroll
        for (int u = 0; u < 4; ++u) p[n][u] = next[n][u];
      lds_barrier();
    }
    add_values(((s1 - s0 - 1) & 1) * L::kBuffer, [](int) {});

    l += __shfl_xor(l, 32);
    const float times = l == 0.0f ? 0.0f : 1.0f / l;      // (and then `unit`: their product may be subnormal)
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
              store4_as(a.y, to * D + d, a.c.dtype, f4{o[t][4 * b], o[t][4 * b + 1], o[t][4 * b + 2], o[t][4 * b + 3]} * times * unit);
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
                f4{o[t][4 * b], o[t][4 * b + 1], o[t][4 * b + 2], o[t][4 * b + 3]} * times * unit;
        }
      if (f == 0) part[kRows * D + line] = lse2;
    }
    left -= s1 - s0;
    first_part = false;
    s0 = 0;
    if (++tile_number == tiles) {
      tile_number = 0;
      if (++h == a.c.H) {
        h = 0;
        do {
          ++seq;
          if (seq >= a.c.S) break;
          r = uniform(rows_of(a.c, seq));
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
    // four parts asked for at a time, the last one again where there are fewer
    float m = -__builtin_inff(), l = 0.0f;
    f4 y{};
    for (int n0 = 0; n0 < parts; n0 += 4) {
      float lse[4];
      f4 v[4];
#pragma unroll
      for (int n = 0; n < 4; ++n) {
        const float* from = part(min(n0 + n, parts - 1));
        lse[n] = from[kRows * D + line];
        v[n] = *reinterpret_cast<const f4*>(from + (size_t)line * D + d);
      }
      float now = m;
#pragma unroll
      for (int n = 0; n < 4; ++n) {
        if (n0 + n >= parts) lse[n] = -__builtin_inff();
        now = fmaxf(now, lse[n]);
      }
      const float had = l * __builtin_amdgcn_exp2f(m - above(now));
      float e[4];
      l = had;
#pragma unroll
      for (int n = 0; n < 4; ++n) l += e[n] = n0 + n < parts ? __builtin_amdgcn_exp2f(lse[n] - above(now)) : 0.0f;
      const float times = l == 0.0f ? 0.0f : 1.0f / l;      // (a mean throughout: a sum of values might pass fp32's range)
      y *= had * times;
#pragma unroll
      for (int n = 0; n < 4; ++n) y += n0 + n < parts ? e[n] * times * v[n] : f4{};
      m = now;
    }
    const size_t to = (size_t)(r.row0 + token) * a.Hq + next.head * group + row - token * group;
    store4_as(a.y, to * D + d, a.c.dtype, y);
    if (a.lse && d == 0) a.lse[to] = (m + __builtin_amdgcn_logf(l)) * kLn2;
  }
}

template <int kC, int kTerms, int kWeights>
hipError_t launch_tiles(const AttentionArgs& a, hipStream_t stream) {
  constexpr int blocks = blocks_of_kernel(kC);
  attention_tiles_kernel<kC, kTerms, kWeights><<<blocks, kThreads, 0, stream>>>(a, blocks);
  return hipGetLastError();
}

template <int kTerms, int kWeights>
hipError_t launch_terms(const AttentionArgs& a, hipStream_t stream) {
  switch ((a.c.D + 63) / 64) {
    case 1: return launch_tiles<1, kTerms, kWeights>(a, stream);
    case 2: return launch_tiles<2, kTerms, kWeights>(a, stream);
    case 3: return launch_tiles<3, kTerms, kWeights>(a, stream);
    default: return launch_tiles<4, kTerms, kWeights>(a, stream);
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
  e = a.c.dtype == SHERRY_F32   ? launch_terms<2, 2>(a, stream)
      : a.c.dtype == SHERRY_F16 ? launch_terms<1, 2>(a, stream)
                                : launch_terms<1, 1>(a, stream);
  if (e != hipSuccess) return e;
  attention_tiles_join_kernel<<<dim3(blocks, 8), kThreads, 0, stream>>>(a, blocks);
  return hipGetLastError();
}

}  // namespace sherry
