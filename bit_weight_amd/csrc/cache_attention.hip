// Causal attention of each sequence's newest tokens over its 8-bit pages:
//   s_j = scale q . k_j for the visible j,  y = sum_j e^(s_j - m) v_j / l,
//   l = sum_j e^(s_j - m),  m = max_j s_j,  lse = m + log l.
// Token j is visible to the query at position p where j <= p, and with a window
// where p - j < window or j < sinks.
//
// One pass over the keys with a running maximum and sum.  A step is 64 tokens,
// four 16-token blocks.  Scores are taken transposed, keys times queries: lane
// (query i, group g) of the product then holds 16 scores of one query, and with
// the keys' rows dealt so that row 4 g + r of product n is token 4 n + r of
// block g they are the 16 tokens of block g, which is what the product with the
// values takes as its operand from the same lane: nothing crosses lanes but the
// maximum, and each lane has one key and one value scale a step.
//
// 8-bit values are exact in fp16, so the products run on fp16 operands with fp32
// sums: q under a power of two per row, e^(s - m) times the value scale over the
// largest one so far (a power of two too) times 2^7.  A 16-bit q is exact in one
// fp16 term, an fp32 one takes a high and a low one (2^-22).  A weight's rounding comes
// to y as that of the values would: one term (half a step: 2^-11) for bf16, whose own
// half step of 2^-8 hides it (the error's mean square grows by up to 1.4 %), two for fp16,
// where one made the error 1.2 to 1.4 times that of the last rounding, and for fp32 (2^-22).
//
// Measured: 64 sequences of up to 8192 tokens, one query each, 32 heads over 8 of 128 in
// bf16: 133 us for 680 MB (5.1 TB/s, what a copy reaches); one of 1000 tokens 11.0 us, all
// of it launch, the chain page -> keys -> values -> parts -> join.
#include "sherry_attention.h"

namespace sherry {
namespace {

constexpr int kRows = 16;                // queries of a unit

// A workgroup's waves take its steps in turn.  Two workgroups a CU, or one where D > 128
// wants the registers: a unit is short beside its beginning and end, which are mostly
// waits, and one workgroup's run under the other's steps (one of eight waves a CU: 256
// sequences of up to 100 tokens 50 us, 34 so).
constexpr int kWaves = 4;
constexpr int kThreads = 64 * kWaves;
constexpr int kBlocks = 2 * kCUs;
constexpr int blocks_of_kernel(int kC) { return kC <= 2 ? kBlocks : kBlocks / 2; }

// Units of a sequence: each head's tiles of 16 rows; a row is a token and one of
// the query heads that share the head.
__device__ __forceinline__ int tiles_of(const AttentionArgs& a, const Rows& r) {
  return (r.n * (a.Hq / a.c.H) + kRows - 1) / kRows;
}

// What a unit looks at.
__device__ __forceinline__ Steps steps_of(const AttentionArgs& a, const Rows& r, int tile) {
  const int group = a.Hq / a.c.H, first = r.len - r.n;
  const bool begins = tile == 0, ends = kRows * (tile + 1) >= r.n * group;       // (no division where all is one unit)
  return Steps(a, begins ? first : first + kRows * tile / group, ends ? r.len - 1 : first + (kRows * tile + kRows - 1) / group);
}

// A unit's steps are cut into equal pieces of at most `most` steps, but no more than
// kParts of them (as many as its sequence's last unit, which looks at the most but for
// one):
//   kShort, and units of up to kMiddle not at all, where half of the workgroups get one;
//   kMiddle where every piece has a workgroup of its own;
//   1 where a workgroup has kMany steps or more;
//   as many as a workgroup has on average where that gives every piece one of its own;
//   else kLong, so that short units are not cut.
// (One sequence of 1000 tokens: 12.6 us in pieces of 8, 11.0 of 4; of 16000: 21 us in 63
// parts, 15.8 in 31; 64 of 125 to 500 tokens: 32 us in even shares, 16 in pieces; 16
// windows of 4096 tokens: 32 us in pieces of 16, 24 of the average.)  All pieces, one
// after another (by sequence, head and tile), are dealt evenly: workgroup w takes `each`
// of them from piece first(w) on; those of one unit it takes together.  Even are the
// pieces: a causal prompt's earlier units have its last one's number of them and fewer
// steps, so that the workgroups of a prompt without history have from none to twice
// the average.
constexpr int kShort = 4, kMiddle = 8, kLong = 16, kMany = 24, kParts = 32;
struct Deal {
  int64_t total;
  int each;
  __device__ __forceinline__ explicit Deal(int64_t t, int blocks) : total(t) {
    each = (int)min(quotient(t + blocks - 1, blocks), (int64_t)1 << 30);
  }
  __device__ __forceinline__ int64_t first(int w) const { return (int64_t)each * w; }
  __device__ __forceinline__ int owner(int64_t piece) const { return (int)quotient(piece, each); }
};
__device__ __forceinline__ int pieces_of(int steps, int most) {
  if (most == kShort && steps <= kMiddle) return 1;
  return most == 1 ? steps : min((steps + most - 1) / most, kParts);
}

__device__ __forceinline__ int64_t pieces_of(const AttentionArgs& a, const Rows& r, int most) {
  return r.n > 0 ? (int64_t)a.c.H * tiles_of(a, r) * pieces_of(steps_of(a, r, tiles_of(a, r) - 1).count(), most) : 0;
}

__device__ __forceinline__ float max_of_groups(float v) {
  v = fmaxf(v, __shfl_xor(v, 16));
  return fmaxf(v, __shfl_xor(v, 32));
}

__device__ __forceinline__ float inverse(float sum) { return sum == 0.0f ? 0.0f : 1.0f / sum; }      // (of weights: none, y is 0)

__device__ __forceinline__ float sum_of_groups(float v) {
  v += __shfl_xor(v, 16);
  return v + __shfl_xor(v, 32);
}

// Parts pass from one XCD to another, whose L2 are not one: relaxed atomics of the
// agent's scope go past them.  (A release and an acquire at that scope write back and
// drop the whole L2 each time: 64 sequences of 2600 to 8192 tokens took 307 us with them,
// 131 without.)
__device__ __forceinline__ void share(float* p, float v) { __hip_atomic_store(p, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT); }
__device__ __forceinline__ float shared_value(const float* p) {
  return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ void share(float* p, f4 v) {      // (8 bytes aligned)
  const uint4 u = __builtin_bit_cast(uint4, v);
  uint64_t* to = reinterpret_cast<uint64_t*>(p);
  __hip_atomic_store(to, u.x | (uint64_t)u.y << 32, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  __hip_atomic_store(to + 1, u.z | (uint64_t)u.w << 32, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ f4 shared_four(const float* p) {
  const uint64_t* from = reinterpret_cast<const uint64_t*>(p);
  const uint64_t a = __hip_atomic_load(from, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  const uint64_t b = __hip_atomic_load(from + 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  return __builtin_bit_cast(f4, make_uint4((uint32_t)a, (uint32_t)(a >> 32), (uint32_t)b, (uint32_t)(b >> 32)));
}
// Every store of this wave has arrived before anything that follows is issued.
__device__ __forceinline__ void all_arrived() {
  asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
}

// A part of a unit in scratch: [16][D] of y over these steps alone, then the 16 maxima and sums.
__host__ __device__ inline size_t part_floats(int D) { return (size_t)kRows * (D + 2); }

// A workgroup's share of a unit: pieces p0 .. p1 - 1 of `pieces`, steps s0 .. s1 - 1.
struct Share {
  int seq, h, tile, p0, p1, pieces, s0, s1;
  Rows r;
  Steps steps;
  __device__ __forceinline__ void cut(int64_t left) {
    const int count = steps.count(), each = count / pieces, more = count - each * pieces;
    p1 = (int)min((int64_t)pieces, p0 + left);
    s0 = each * p0 + min(p0, more);
    s1 = each * p1 + min(p1, more);
  }
  // `rest` of the sequence's pieces come before, `left` are this workgroup's from there on
  __device__ __forceinline__ Share(const AttentionArgs& a, int seq_, const Rows& r_, int64_t rest, int64_t left, int most)
      : seq(seq_), r(r_), steps(steps_of(a, r_, tiles_of(a, r_) - 1)) {
    pieces = pieces_of(steps.count(), most);
    const int tiles = tiles_of(a, r), unit = (int)quotient(rest, pieces);
    h = unit / tiles;
    tile = unit - h * tiles;
    steps = steps_of(a, r, tile);
    p0 = (int)(rest - (int64_t)unit * pieces);
    cut(left);
  }
  // the unit after this one, of which `left` pieces are this workgroup's (more than 0)
  __device__ __forceinline__ void advance(const AttentionArgs& a, int64_t left, int most) {
    p0 = 0;
    const int tiles = tiles_of(a, r);
    if (++tile == tiles) {
      tile = 0;
      if (++h == a.c.H) {
        h = 0;
        do r = uniform(rows_of(a.c, ++seq));
        while (r.n == 0);
        pieces = pieces_of(steps_of(a, r, tiles_of(a, r) - 1).count(), most);
      }
    }
    steps = steps_of(a, r, tile);
    cut(left);
  }
};

// kC: D / 64 rounded up.  kFull: D is 64 kC.  kTerms, kWeights: fp16 terms of q and of the weights.
template <int kC, bool kFull, int kTerms, int kWeights>
__global__ __launch_bounds__(kThreads, kC <= 2 ? 2 : 1) void attention_kernel(AttentionArgs a) {
  constexpr int kGrid = blocks_of_kernel(kC);
  constexpr int kTiles = 4 * kC;        // of 16 features
  constexpr int kPitch = 64 * kC + 4;
  constexpr float kWeight = 128.0f;     // 2^kWeightExponent
  __shared__ float join[kWaves][kRows][kPitch];
  __shared__ float maxima[kWaves][kRows], sums[kWaves][kRows];
  __shared__ int64_t scan[kWaves], found_rest;
  __shared__ int found_seq, is_last;
  __shared__ Rows found_rows;
  const int tid = threadIdx.x, lane = tid & 63, wave = uniform(tid >> 6), i = lane & 15, g = lane >> 4;
  const int block = blockIdx.x, group = a.Hq / a.c.H, D = a.c.D, pieces = D / 16;

  // Where this workgroup's pieces begin: up to 64 sequences a lane each, in every wave;
  // more of them a thread each, 64 kWaves at a time.
  const bool few = a.c.S <= 64;
  int64_t total = 0, before = 0, own = 0;
  int round = few ? 0 : 2, most = few ? kShort : 1;      // (steps of a piece)
  Rows mine{};
  auto look_at = [&](int seq) {
    mine = {};
    if (seq < a.c.S) mine = rows_of(a.c, seq);
    own = pieces_of(a, mine, most);
  };
  if (few) look_at(lane);
  for (;;) {
    if (few) {
      own = pieces_of(a, mine, most);
      int64_t sum = own;
#pragma unroll
      for (int d = 1; d < 64; d *= 2) {
        const int64_t v = shfl_up64(sum, d);
        if (lane >= d) sum += v;
      }
      before = sum - own;
      total = ((int64_t)__builtin_amdgcn_readlane((int)(sum >> 32), 63) << 32) | (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)sum, 63);
    } else {
      total = 0;
      for (int base = 0; base < a.c.S; base += kThreads) {
        look_at(base + tid);
        total += block_scan<kWaves>(own, before, scan);
      }
      total = uniform64(total);
    }
    if (round == 4 || (round == 2 ? total >= kMany * kGrid : total <= (round == 0 ? kGrid / 2 : kGrid))) break;
    most = round == 0 ? kMiddle : round == 1 ? 1 : round == 2 ? max(kMiddle, (int)quotient(total, kGrid) + 1) : kLong;
    ++round;
  }
  if (total == 0) return;
  const Deal deal(total, kGrid);
  const int64_t begin = deal.first(block);
  if (begin >= total) return;
  int64_t left = min(total - begin, (int64_t)deal.each);
  int first_seq;
  int64_t first_rest;
  Rows first_rows;
  if (few) {
    const int at = __ffsll((unsigned long long)__ballot(begin >= before && begin < before + own)) - 1;
    first_seq = at;
    first_rows = {__builtin_amdgcn_readlane(mine.row0, at), __builtin_amdgcn_readlane(mine.n, at), __builtin_amdgcn_readlane(mine.len, at)};
    first_rest = begin - (((int64_t)__builtin_amdgcn_readlane((int)(before >> 32), at) << 32) |
                          (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)before, at));
  } else {
    int64_t past = 0;
    for (int base = 0; past <= begin; base += kThreads) {       // (begin < total, so a sequence has it)
      look_at(base + tid);
      const int64_t all = block_scan<kWaves>(own, before, scan);
      before += past;
      if (begin >= before && begin < before + own) {
        found_seq = base + tid;
        found_rows = mine;
        found_rest = begin - before;
      }
      past += all;
    }
    __syncthreads();
    first_seq = uniform(found_seq);
    first_rows = uniform(found_rows);
    first_rest = uniform64(found_rest);
  }
  Share now(a, first_seq, first_rows, first_rest, left, most);
  int64_t here = begin;        // the share's first piece
  bool first_part = true;

  // A wave's next step: its pages, then its bytes, each asked for a step before it is
  // needed, also when that is in the next unit.  Where there is none, block 0 of the
  // cache is read, so that nothing here branches.
  // Keys: lane (row 4 g' + r, group g) takes features 16 (4 c + g) .. of token 4 n + r of
  // block g', so that lane (query i, group g) of the product has the 16 tokens of block
  // g.  Values: tokens 16 g .. of feature 16 t + i.
  int key_page, value_page;
  uint4 kw[4][kC], vw[kTiles];
  float ks, vs;
  uint32_t value_block;       // (a cache has fewer than 2^31 blocks)
  bool value_good;
  const uint32_t page_blocks = (uint32_t)a.c.H << a.c.block_shift;
  auto load_pages = [&](int seq, int step) {
    const int32_t* table = a.c.table + (size_t)seq * a.c.table_width;
    key_page = table[min((4 * step + i / 4) >> a.c.block_shift, a.c.table_width - 1)];
    value_page = table[min((4 * step + g) >> a.c.block_shift, a.c.table_width - 1)];
  };
  auto load_keys = [&](bool any, int h, int step) {
    const int kb = 4 * step + i / 4, vb = 4 * step + g, in_page = (1 << a.c.block_shift) - 1;
    const uint32_t h_blocks = (uint32_t)h << a.c.block_shift;
    auto good = [&](int page, int b) {
      return any && (uint32_t)page < (uint32_t)a.c.pages && b >> a.c.block_shift < a.c.table_width;
    };
    value_good = good(value_page, vb);
    value_block = value_good ? (uint32_t)value_page * page_blocks + h_blocks + (vb & in_page) : 0;
    const uint32_t key_block = good(key_page, kb) ? (uint32_t)key_page * page_blocks + h_blocks + (kb & in_page) : 0;
    const uint8_t* from = a.c.k + (uint64_t)key_block * (uint32_t)(16 * D) + 16 * (i & 3) + (kFull ? 256 * g : 0);
#pragma unroll
    for (int n = 0; n < 4; ++n)
#pragma unroll
      for (int c = 0; c < kC; ++c)      // (pieces past D: the last one again, which meets zeros of q)
        kw[n][c] = *reinterpret_cast<const uint4*>(from + (kFull ? 1024 * c : 256 * min(4 * c + g, pieces - 1)) + 64 * n);
    ks = a.c.k_scale[value_block];      // (of the block whose scores this lane will have)
    vs = a.c.v_scale[value_block];
  };
  auto load_values = [&]() {
    const uint8_t* from = a.c.v + (uint64_t)value_block * (uint32_t)(16 * D) + 16 * i;
#pragma unroll
    for (int t = 0; t < kTiles; ++t) vw[t] = *reinterpret_cast<const uint4*>(from + 256 * (kFull ? t : min(t, pieces - 1)));
  };
  // The wave's steps in turn, the next unit's after this one's: sequence, head and
  // token step of the one after s, or of the first; none: step 0 of the same.
  struct At {
    bool any;
    int seq, h, step;
  };
  {
    const int s = now.s0 + wave;
    load_pages(now.seq, s < now.s1 ? now.steps.at(s) : 0);
    load_keys(s < now.s1, now.h, s < now.s1 ? now.steps.at(s) : 0);
  }
  load_values();

  for (;;) {
    const Rows r = now.r;
    const int h = now.h, tile = now.tile, s0 = now.s0, s1 = now.s1;
    left -= now.p1 - now.p0;
    Share next = now;
    if (left > 0) next.advance(a, left, most);
    else next.s0 = next.s1 = 0;
    auto after = [&](int s) {
      const bool same = s + kWaves < s1;
      const int to = same ? s + kWaves : next.s0 + wave, head = same ? now.steps.head : next.steps.head,
                from = same ? now.steps.from : next.steps.from;
      const bool any = same || to < next.s1;
      return At{any, same ? now.seq : next.seq, same ? h : next.h, !any ? 0 : to < head ? to : from + to - head};
    };
    if (s0 + wave < s1) {
      const At x = after(s0 + wave);
      load_pages(x.seq, x.step);
    } else {        // (this wave has no step of this unit: what it has asked for is the next unit's first)
      const int s = next.s0 + wave;
      load_pages(next.seq, s < next.s1 ? next.steps.at(s) : 0);
      load_keys(s < next.s1, next.h, s < next.s1 ? next.steps.at(s) : 0);
      load_values();
    }
    {
      // queries, exact as fp16 under 2^e per row (the row's largest near 2^13)
      const int row = kRows * tile + i, token = row / group, position = r.len - r.n;
      const bool in = token < r.n;
      const int pos = in ? position + token : -1;
      const int low = position + kRows * tile / group, high = position + min((kRows * tile + kRows - 1) / group, r.n - 1);
      h8 q[kTerms][kC][2];
      float factor;
      {
        const size_t at = (size_t)(r.row0 + (in ? token : 0)) * a.q_stride +
                          (size_t)(h * group + (in ? row - token * group : 0)) * D;
        RawValues<4> raw[kC];
        float top = 0.0f;
#pragma unroll
        for (int c = 0; c < kC; ++c) raw[c].load(a.q, at + 16 * min(4 * c + g, pieces - 1), a.c.dtype);
        f4 x[kC][4];
#pragma unroll
        for (int c = 0; c < kC; ++c)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            x[c][j] = in && 4 * c + g < pieces ? raw[c].get(j, a.c.dtype) : f4{};
#pragma unroll
            for (int b = 0; b < 4; ++b) top = fmaxf(top, fabsf(x[c][j][b]));
          }
        const float times = row_scale(max_of_groups(top));
        factor = a.scale * kLog2E / times;
#pragma unroll
        for (int c = 0; c < kC; ++c)
#pragma unroll
          for (int half = 0; half < 2; ++half)
#pragma unroll
            for (int b = 0; b < 8; ++b) {
              const float v = x[c][2 * half + b / 4][b % 4] * times;
              const _Float16 hi = (_Float16)v;
              q[0][c][half][b] = hi;
              if constexpr (kTerms == 2) q[kTerms - 1][c][half][b] = (_Float16)(v - (float)hi);
            }
      }

      // maximum, this lane's part of the sum (NaN for all of a sequence longer than its
      // table, also where a window hides what the table has room for), largest value scale
      // so far, features 16 t + 4 g + r of query i in `unit` / kWeight
      float m = -__builtin_inff(), l = r.len > room_of(a) ? __builtin_nanf("") : 0.0f, unit = 0x1p-126f;
      f4 o[kTiles];
#pragma unroll
      for (int t = 0; t < kTiles; ++t) o[t] = f4{};
      for (int s = s0 + wave; s < s1; s += kWaves) {
        const int t0 = kStep * now.steps.at(s);
        f4 sc[4];
#pragma unroll
        for (int n = 0; n < 4; ++n) {
          sc[n] = f4{};
#pragma unroll
          for (int c = 0; c < kC; ++c) {
            const h8 k0 = halves8(kw[n][c].x, kw[n][c].y), k1 = halves8(kw[n][c].z, kw[n][c].w);
#pragma unroll
            for (int t = 0; t < kTerms; ++t) {
              sc[n] = __builtin_amdgcn_mfma_f32_16x16x32_f16(k0, q[t][c][0], sc[n], 0, 0, 0);
              sc[n] = __builtin_amdgcn_mfma_f32_16x16x32_f16(k1, q[t][c][1], sc[n], 0, 0, 0);
            }
          }
        }
        const float scale_now = vs, by = factor * (value_good && vs == vs ? ks : __builtin_nanf(""));   // not valid: NaN for whoever sees it
        const At then = after(s);
        load_keys(then.any, then.h, then.step);
        const At later = after(s + kWaves < s1 ? s + kWaves : s);     // (past this unit its own first step asks)
        load_pages(later.seq, later.step);
        float top = -__builtin_inff();
#pragma unroll
        for (int n = 0; n < 4; ++n) sc[n] *= by;
        if (!sees_all(a, t0, low, high)) {
          asm volatile("");       // (a branch, not selections in every step)
#pragma unroll
          for (int n = 0; n < 4; ++n)
#pragma unroll
            for (int b = 0; b < 4; ++b)
              if (!sees(a, t0 + 16 * g + 4 * n + b, pos)) sc[n][b] = -__builtin_inff();
        }
#pragma unroll
        for (int n = 0; n < 4; ++n)
#pragma unroll
          for (int b = 0; b < 4; ++b) top = fmaxf(top, sc[n][b]);
        // (the scale of a block that is not seen may be anything)
        const float scale_top = max_of_groups(fmaxf(unit, top > -__builtin_inff() && scale_now < __builtin_inff() ? scale_now : 0.0f));
        top = max_of_groups(top);
        if (__any(top > m + kSlack || scale_top > unit)) {
          const float peak = fmaxf(m, top);
          const float keep = __builtin_amdgcn_exp2f(m - above(peak));      // (0 where nothing was seen so far)
          l *= keep;
          const float scaled = keep * unit * __builtin_amdgcn_rcpf(scale_top);
#pragma unroll
          for (int t = 0; t < kTiles; ++t) o[t] *= scaled;
          m = peak;
          unit = scale_top;
        }
        const float base = above(m), w = kWeight * (scale_now * __builtin_amdgcn_rcpf(unit));
        h8 p[kWeights][2];
#pragma unroll
        for (int n = 0; n < 4; ++n)
#pragma unroll
          for (int b = 0; b < 4; ++b) {
            const float e = __builtin_amdgcn_exp2f(sc[n][b] - base);
            l += e;
            const float v = sc[n][b] == -__builtin_inff() ? 0.0f : e * w;
            const _Float16 hi = (_Float16)v;
            p[0][n / 2][4 * (n % 2) + b] = hi;
            if constexpr (kWeights == 2) p[kWeights - 1][n / 2][4 * (n % 2) + b] = (_Float16)(v - (float)hi);
          }
#pragma unroll
        for (int t = 0; t < kTiles; ++t) {
          const h8 v0 = halves8(vw[t].x, vw[t].y), v1 = halves8(vw[t].z, vw[t].w);
#pragma unroll
          for (int n = 0; n < kWeights; ++n) {
            o[t] = __builtin_amdgcn_mfma_f32_16x16x32_f16(v0, p[n][0], o[t], 0, 0, 0);
            o[t] = __builtin_amdgcn_mfma_f32_16x16x32_f16(v1, p[n][1], o[t], 0, 0, 0);
          }
        }
        load_values();
      }

      // the waves' parts, each a mean of values: sums of them might pass fp32's range
      l = sum_of_groups(l);
      const float times = inverse(kWeight * l);
      __syncthreads();
#pragma unroll
      for (int t = 0; t < kTiles; ++t)
        *reinterpret_cast<f4*>(&join[wave][i][16 * t + 4 * g]) = o[t] * times * unit;
      if (g == 0) {
        maxima[wave][i] = m;
        sums[wave][i] = l;
      }
      __syncthreads();
      const bool whole = now.p0 == 0 && now.p1 == now.pieces;
      const int quads = D / 4, rows = min(kRows, r.n * group - kRows * tile);
      // of the first `count` of `join`, a line's four features; their maximum and sum
      auto mean_of = [&](int count, int line, int d, float& top, float& sum) {
        float e[kWaves];
        top = maxima[0][line];
        sum = 0.0f;
#pragma unroll
        for (int v = 1; v < kWaves; ++v) top = fmaxf(top, v < count ? maxima[v][line] : top);
#pragma unroll
        for (int v = 0; v < kWaves; ++v)
          sum += e[v] = v < count ? __builtin_amdgcn_exp2f(maxima[v][line] - above(top)) * sums[v][line] : 0.0f;
        const float times = inverse(sum);
        f4 y{};
#pragma unroll
        for (int v = 0; v < kWaves; ++v) y += v < count ? e[v] * times * *reinterpret_cast<const f4*>(&join[v][line][d]) : f4{};
        return y;
      };
      auto put = [&](int of_tile, int d, f4 y, float top, float sum) {
        const int line = kRows * tile + of_tile, of = line / group;
        const size_t at = (size_t)(r.row0 + of) * a.Hq + h * group + line - of * group;
        store4_as(a.y, at * D + d, a.c.dtype, y);
        if (a.lse && d == 0) a.lse[at] = (top + __builtin_amdgcn_logf(sum)) * kLn2;
      };
      float* part = a.scratch + (size_t)(2 * block + (first_part ? 0 : 1)) * part_floats(D);
      for (int x = tid; x < rows * quads; x += kThreads) {
        const int line = x / quads, d = 4 * (x - line * quads);
        float top, sum;
        const f4 y = mean_of(kWaves, line, d, top, sum);
        if (whole) {
          put(line, d, y, top, sum);
        } else {
          share(part + (size_t)line * D + d, y);
          if (d == 0) {
            share(part + kRows * D + line, top);
            share(part + kRows * D + kRows + line, sum);
          }
        }
      }
      if (!whole) {
        // The unit's parts are in as many workgroups as its pieces are dealt to; the one
        // that is done last joins them, always in their order.  Only one unit that begins
        // in a workgroup goes on in the next: that workgroup's counter is the unit's.
        const int64_t unit_first = here - now.p0;
        const int w0 = deal.owner(unit_first), w1 = deal.owner(unit_first + now.pieces - 1);
        all_arrived();
        __syncthreads();
        if (tid == 0)
          is_last = __hip_atomic_fetch_add(&a.counters[w0], 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) == w1 - w0;
        __syncthreads();
        if (is_last) {
          if (tid == 0) __hip_atomic_store(&a.counters[w0], 0, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
          auto part_of = [&](int w) {
            return a.scratch + (size_t)(2 * w + (deal.first(w) < unit_first ? 1 : 0)) * part_floats(D);
          };
          // the threads share the parts too (each a trip to memory), eight asked for at once
          const int outputs = rows * quads, sharers = max(1, min(kWaves, kThreads / outputs));
          for (int base = 0; base < outputs; base += kThreads) {
            const int sharer = sharers > 1 ? tid / outputs : 0, x = base + tid - sharer * outputs;
            const bool has = sharer < sharers && x < outputs;
            const int line = x / quads, d = 4 * (x - line * quads);
            float top = -__builtin_inff(), sum = 0.0f;
            f4 y{};
            for (int w = w0 + sharer; has && w <= w1; w += 8 * sharers) {
              float tops[8], sums_of[8];
              f4 ys[8];
#pragma unroll
              for (int k = 0; k < 8; ++k) {
                const float* from = part_of(min(w + k * sharers, w1));
                tops[k] = shared_value(from + kRows * D + line);
                sums_of[k] = shared_value(from + kRows * D + kRows + line);
                ys[k] = shared_four(from + (size_t)line * D + d);
              }
              float peak = top;
#pragma unroll
              for (int k = 0; k < 8; ++k) peak = fmaxf(peak, w + k * sharers <= w1 ? tops[k] : top);
              const float had = sum * __builtin_amdgcn_exp2f(top - above(peak));
              float e[8];
              sum = had;
#pragma unroll
              for (int k = 0; k < 8; ++k)
                sum += e[k] = w + k * sharers <= w1 ? __builtin_amdgcn_exp2f(tops[k] - above(peak)) * sums_of[k] : 0.0f;
              const float times = inverse(sum);
              y *= had * times;
#pragma unroll
              for (int k = 0; k < 8; ++k) y += w + k * sharers <= w1 ? e[k] * times * ys[k] : f4{};
              top = peak;
            }
            if (sharers > 1) {
              if (has) {
                *reinterpret_cast<f4*>(&join[sharer][line][d]) = y;
                if (d == 0) {
                  maxima[sharer][line] = top;
                  sums[sharer][line] = sum;
                }
              }
              __syncthreads();
              if (sharer == 0 && has) y = mean_of(sharers, line, d, top, sum);
            }
            if (sharer == 0 && has) put(line, d, y, top, sum);
          }
        }
      }
      first_part = false;
    }
    if (left == 0) break;
    here += now.p1 - now.p0;
    now = next;
  }
}

template <int kC, int kTerms, int kWeights>
void launch_full(const AttentionArgs& a, hipStream_t stream) {
  if (a.c.D == 64 * kC) attention_kernel<kC, true, kTerms, kWeights><<<blocks_of_kernel(kC), kThreads, 0, stream>>>(a);
  else attention_kernel<kC, false, kTerms, kWeights><<<blocks_of_kernel(kC), kThreads, 0, stream>>>(a);
}

template <int kTerms, int kWeights>
void launch_terms(const AttentionArgs& a, hipStream_t stream) {
  switch ((a.c.D + 63) / 64) {
    case 1: return launch_full<1, kTerms, kWeights>(a, stream);
    case 2: return launch_full<2, kTerms, kWeights>(a, stream);
    case 3: return launch_full<3, kTerms, kWeights>(a, stream);
    default: return launch_full<4, kTerms, kWeights>(a, stream);
  }
}

}  // namespace

// Whether the kernel that shares a step's keys and values between 128 rows pays: where
// sequences have 64 rows or more on average, and the steps of 16 rows that all of them take
// are many (counted with the longest sequence that the table has room for, or the window:
// the host knows no lengths).  One kernel takes all sequences of a call: a prompt among
// many single tokens (4000 tokens among 299: 1060 us, apart 280 and 167) goes to 16-row
// units with them.  Beside those the tiles' own start, deal and join take 40 us.  Prompts
// behind 1700 tokens, 32 heads over 8 of 128, in units and in tiles, us: of 361 (24000
// steps) 57 and 75 in bf16, 63 and 104 in fp32; of 460 (31000) 67 and 74, 74 and 101; of
// 600 (43000) 82 and 83, 94 and 118; of 800 (64000) 106 and 85, 120 and 125.
constexpr int64_t kTilesPay = 32000;
static bool tiles_pay(const AttentionArgs& a) {
  const int64_t T = a.c.T, S = a.c.S, group = a.Hq / a.c.H;
  if (T * group < 64 * S) return false;
  int64_t seen = (int64_t)a.c.table_width << (a.c.block_shift + 4);
  if (a.window > 0) seen = std::min<int64_t>(seen, (int64_t)a.window + a.sinks);
  return T * a.Hq / 16 * (seen / kStep + 1) >= kTilesPay;
}

size_t cache_attention_scratch_bytes(int T, int S, int Hq, int H, int D) {
  const size_t rows = (size_t)2 * kBlocks * part_floats(D) * sizeof(float);
  return (int64_t)T * (Hq / H) >= 64 * (int64_t)S ? std::max(rows, attention_tiles_scratch_bytes(S, D)) : rows;
}

size_t cache_attention_workspace_bytes() { return kBlocks * sizeof(int); }

hipError_t launch_cache_attention(const AttentionArgs& a, hipStream_t stream, bool* partial) {
  if (tiles_pay(a)) return launch_attention_tiles(a, stream, partial);
  if (a.c.dtype == SHERRY_F32) launch_terms<2, 2>(a, stream);
  else if (a.c.dtype == SHERRY_F16) launch_terms<1, 2>(a, stream);
  else launch_terms<1, 1>(a, stream);
  return hipGetLastError();
}

}  // namespace sherry
