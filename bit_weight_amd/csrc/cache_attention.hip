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
// largest one so far (a power of two too) times 2^7.  One fp16 term of each
// for 16-bit queries (q is exact, the weights off by 2^-12), a high and a low
// one for fp32 queries (2^-23).
#include "sherry_attention.h"

namespace sherry {
namespace {

constexpr int kWaves = 4;
constexpr int kThreads = 64 * kWaves;
constexpr int kRows = 16;                // queries of a unit
constexpr int kBlocks = 2 * kCUs;        // workgroups
constexpr int kLeast = 2 * kWaves;       // steps that a workgroup takes at least
constexpr float kWeight = 128.0f;        // 2^kWeightExponent

// Units of a sequence: each head's tiles of 16 rows; a row is a token and one of
// the query heads that share the head.
__device__ __forceinline__ int tiles_of(const AttentionArgs& a, const Rows& r) {
  return (r.n * (a.Hq / a.c.H) + kRows - 1) / kRows;
}

// All of a sequence's units look at the same steps.
__device__ __forceinline__ Steps steps_of(const AttentionArgs& a, const Rows& r) {
  return Steps(a, r.len - r.n, r.len - 1);
}

__device__ __forceinline__ int64_t cost_of(const AttentionArgs& a, int i) {
  const Rows r = rows_of(a.c, i);
  return r.n == 0 ? 0 : (int64_t)a.c.H * tiles_of(a, r) * steps_of(a, r).count();
}

// All units' steps, one after another, are dealt evenly: workgroup w of `used`
// takes steps w total / used up to the next one's first.
struct Deal {
  int64_t total;
  int used;
  __device__ __forceinline__ explicit Deal(int64_t t) : total(t) {
    const int64_t most = (t + kLeast - 1) / kLeast;
    used = (int)(most < kBlocks ? most : kBlocks);
  }
  __device__ __forceinline__ int64_t first(int w) const { return total * w / used; }
  // the workgroup that has step s
  __device__ __forceinline__ int owner(int64_t s) const {
    int w = (int)(s * used / total);
    while (w + 1 < used && first(w + 1) <= s) ++w;
    return w;
  }
};

__device__ __forceinline__ float max_of_groups(float v) {
  v = fmaxf(v, __shfl_xor(v, 16));
  return fmaxf(v, __shfl_xor(v, 32));
}

__device__ __forceinline__ float sum_of_groups(float v) {
  v += __shfl_xor(v, 16);
  return v + __shfl_xor(v, 32);
}

// kC: D / 64 rounded up.  kTerms: fp16 terms of q and of the weights.
template <int kC, int kTerms>
struct Wave {
  static constexpr int kTiles = 4 * kC;     // of 16 features
  const AttentionArgs& a;
  int lane, i, g;
  int seq, h, pieces;
  Rows r;
  int pos;              // of this lane's query
  int low, high;        // of the tile's queries
  float factor;         // of q's power of two and the scale, for base 2
  h8 q[kTerms][kC][2];
  // running
  float m, l, unit;     // maximum, this lane's part of the sum, largest value scale
  f4 o[kTiles];         // features 16 t + 4 g + r of query i, in `unit` / kWeight

  __device__ __forceinline__ Wave(const AttentionArgs& args) : a(args) {
    lane = threadIdx.x & 63;
    i = lane & 15;
    g = lane >> 4;
    pieces = a.c.D / 16;
  }

  // The queries of tile `tile`: exact as fp16 under 2^e per row, the row's largest near 2^14.
  __device__ __forceinline__ void load_queries(int tile) {
    const int group = a.Hq / a.c.H, row = kRows * tile + i, token = row / group;
    const bool in = token < r.n;
    const size_t at = (size_t)(r.row0 + (in ? token : 0)) * a.q_stride +
                      (size_t)(h * group + (in ? row - token * group : 0)) * a.c.D;
    const int first = r.len - r.n;
    pos = in ? first + token : -1;
    low = first + kRows * tile / group;
    high = first + min((kRows * tile + kRows - 1) / group, r.n - 1);
    f4 raw[kC][4];
    float top = 0.0f;
#pragma unroll
    for (int c = 0; c < kC; ++c)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        raw[c][j] = f4{};
        if (in && 4 * c + g < pieces) raw[c][j] = load4_as(a.q, at + 64 * c + 16 * g + 4 * j, a.c.dtype);
#pragma unroll
        for (int b = 0; b < 4; ++b) top = fmaxf(top, fabsf(raw[c][j][b]));
      }
    top = max_of_groups(top);
    const float times = row_scale(top);
    factor = a.scale * kLog2E / times;
    if (r.len > room_of(a)) factor = __builtin_nanf("");     // tokens without pages
#pragma unroll
    for (int c = 0; c < kC; ++c)
#pragma unroll
      for (int half = 0; half < 2; ++half)
#pragma unroll
        for (int b = 0; b < 8; ++b) {
          const float v = raw[c][2 * half + b / 4][b % 4] * times;
          const _Float16 hi = (_Float16)v;
          q[0][c][half][b] = hi;
          if constexpr (kTerms == 2) q[kTerms - 1][c][half][b] = (_Float16)(v - (float)hi);
        }
  }

  __device__ __forceinline__ void reset() {
    m = -__builtin_inff();
    l = 0.0f;
    unit = 0x1p-126f;
#pragma unroll
    for (int t = 0; t < kTiles; ++t) o[t] = f4{};
  }

  __device__ __forceinline__ void step(int ts) {
    // keys: lane (row 4 g' + r, group g) takes features 16 (4 c + g) .. of token 4 n + r of block g'
    const int key_page = page_of(a.c, seq, 4 * ts + i / 4), page = page_of(a.c, seq, 4 * ts + g);
    const size_t key_block = block_of(a.c, max(key_page, 0), h, 4 * ts + i / 4);
    const size_t block = block_of(a.c, max(page, 0), h, 4 * ts + g);
    const uint8_t* keys = a.c.k + key_block * (16 * a.c.D) + 16 * (i & 3);
    const uint8_t* values = a.c.v + block * (16 * a.c.D) + 16 * i;
    uint4 kw[4][kC], vw[kTiles];
#pragma unroll
    for (int n = 0; n < 4; ++n)
#pragma unroll
      for (int c = 0; c < kC; ++c)
        kw[n][c] = *reinterpret_cast<const uint4*>(keys + 256 * min(4 * c + g, pieces - 1) + 64 * n);
    float ks = a.c.k_scale[block], vs = a.c.v_scale[block];
#pragma unroll
    for (int t = 0; t < kTiles; ++t)
      if (t < pieces) vw[t] = *reinterpret_cast<const uint4*>(values + 256 * t);
    if (page < 0 || vs != vs) ks = __builtin_nanf("");      // whoever sees it gives NaN

    f4 s[4];
#pragma unroll
    for (int n = 0; n < 4; ++n) {
      s[n] = f4{};
#pragma unroll
      for (int c = 0; c < kC; ++c) {
        const h8 k0 = halves8(kw[n][c].x, kw[n][c].y), k1 = halves8(kw[n][c].z, kw[n][c].w);
#pragma unroll
        for (int t = 0; t < kTerms; ++t) {
          s[n] = __builtin_amdgcn_mfma_f32_16x16x32_f16(k0, q[t][c][0], s[n], 0, 0, 0);
          s[n] = __builtin_amdgcn_mfma_f32_16x16x32_f16(k1, q[t][c][1], s[n], 0, 0, 0);
        }
      }
    }
    // (the pieces past D that the keys' loads repeat meet zeros of q)
    const float f = factor * ks;
    const int t0 = kStep * ts;
    const bool all = sees_all(a, t0, low, high);
    float top = -__builtin_inff();
#pragma unroll
    for (int n = 0; n < 4; ++n)
#pragma unroll
      for (int b = 0; b < 4; ++b) {
        s[n][b] *= f;
        if (!all) {
          const int j = t0 + 16 * g + 4 * n + b;
          s[n][b] = sees(a, j, pos) ? s[n][b] : -__builtin_inff();
        }
        top = fmaxf(top, s[n][b]);
      }
    // (the scale of a block that is not seen may be anything)
    const float scale_top = max_of_groups(fmaxf(unit, top > -__builtin_inff() && vs < __builtin_inff() ? vs : 0.0f));
    top = max_of_groups(top);
    if (__any(top > m + kSlack || scale_top > unit)) {
      const float now = fmaxf(m, top);
      const float keep = __builtin_amdgcn_exp2f(m - above(now));      // (0 where nothing was seen so far)
      l *= keep;
      const float scaled = keep * (unit / scale_top);
#pragma unroll
      for (int t = 0; t < kTiles; ++t) o[t] *= scaled;
      m = now;
      unit = scale_top;
    }
    const float base = above(m), w = vs * (kWeight / unit);
    h8 p[kTerms][2];
#pragma unroll
    for (int n = 0; n < 4; ++n)
#pragma unroll
      for (int b = 0; b < 4; ++b) {
        const float e = __builtin_amdgcn_exp2f(s[n][b] - base);
        l += e;
        const float v = s[n][b] == -__builtin_inff() ? 0.0f : e * w;
        const _Float16 hi = (_Float16)v;
        p[0][n / 2][4 * (n % 2) + b] = hi;
        if constexpr (kTerms == 2) p[kTerms - 1][n / 2][4 * (n % 2) + b] = (_Float16)(v - (float)hi);
      }
#pragma unroll
    for (int t = 0; t < kTiles; ++t) {
      if (t < pieces) {
        const h8 v0 = halves8(vw[t].x, vw[t].y), v1 = halves8(vw[t].z, vw[t].w);
#pragma unroll
        for (int u = 0; u < kTerms; ++u) {
          o[t] = __builtin_amdgcn_mfma_f32_16x16x32_f16(v0, p[u][0], o[t], 0, 0, 0);
          o[t] = __builtin_amdgcn_mfma_f32_16x16x32_f16(v1, p[u][1], o[t], 0, 0, 0);
        }
      }
    }
  }
};

// A part of a unit in scratch: [16][D] of y over these steps alone, then the 16 maxima and sums.
__host__ __device__ inline size_t part_floats(int D) { return (size_t)kRows * (D + 2); }

template <int kC, int kTerms>
__global__ __launch_bounds__(kThreads) void attention_kernel(AttentionArgs a) {
  constexpr int kPitch = 64 * kC + 4;
  __shared__ float join[kWaves][kRows][kPitch];
  __shared__ float maxima[kWaves][kRows], sums[kWaves][kRows];
  __shared__ int64_t parts[kWaves];
  __shared__ int64_t found_rest;
  __shared__ int found_seq;
  const int wave = threadIdx.x >> 6, block = blockIdx.x, group = a.Hq / a.c.H;

  int64_t total = 0, before;
  for (int base = 0; base < a.c.S; base += kThreads) {
    const int i = base + threadIdx.x;
    total += block_scan<kWaves>(i < a.c.S ? cost_of(a, i) : 0, before, parts);
  }
  if (total == 0) return;
  const Deal deal(total);
  if (block >= deal.used) return;
  const int64_t begin = deal.first(block);
  int64_t left = deal.first(block + 1) - begin, past = 0;
  for (int base = 0;; base += kThreads) {       // (begin < total, so a sequence has it)
    const int i = base + threadIdx.x;
    const int64_t own = i < a.c.S ? cost_of(a, i) : 0, all = block_scan<kWaves>(own, before, parts);
    before += past;
    if (begin >= before && begin < before + own) {
      found_seq = i;
      found_rest = begin - before;
    }
    past += all;
    if (past > begin) break;
  }
  __syncthreads();
  int seq = found_seq;
  int64_t rest = found_rest;

  Wave<kC, kTerms> w(a);
  bool first_part = true;
  while (left > 0) {
    w.seq = seq;
    w.r = rows_of(a.c, seq);
    const Steps steps = steps_of(a, w.r);
    const int count = steps.count(), tiles = tiles_of(a, w.r), units = w.r.n == 0 ? 0 : a.c.H * tiles;
    for (int u = (int)(rest / count); u < units && left > 0; ++u) {
      const int s0 = (int)(rest - (int64_t)u * count), s1 = (int)min((int64_t)count, s0 + left);
      const int tile = u % tiles;
      w.h = u / tiles;
      w.load_queries(tile);
      w.reset();
      for (int s = s0 + wave; s < s1; s += kWaves) w.step(steps.at(s));
      // the waves' parts
      const float sum = sum_of_groups(w.l);
      __syncthreads();
#pragma unroll
      for (int t = 0; t < 4 * kC; ++t)
        if (t < w.pieces)
          *reinterpret_cast<f4*>(&join[wave][w.i][16 * t + 4 * w.g]) = w.o[t] * (w.unit * (1.0f / kWeight));
      if (w.g == 0) {
        maxima[wave][w.i] = w.m;
        sums[wave][w.i] = sum;
      }
      __syncthreads();
      const bool whole = s0 == 0 && s1 == count;
      float* part = a.scratch + (size_t)(2 * block + (first_part ? 0 : 1)) * part_floats(a.c.D);
      const int quads = a.c.D / 4;
      for (int x = threadIdx.x; x < kRows * quads; x += kThreads) {
        const int row = x / quads, d = 4 * (x - row * quads), line = kRows * tile + row, token = line / group;
        float m = maxima[0][row];
#pragma unroll
        for (int v = 1; v < kWaves; ++v) m = fmaxf(m, maxima[v][row]);
        float l = 0.0f;
        f4 y{};
#pragma unroll
        for (int v = 0; v < kWaves; ++v) {
          const float e = __builtin_amdgcn_exp2f(maxima[v][row] - above(m));
          l += e * sums[v][row];
          y += e * *reinterpret_cast<const f4*>(&join[v][row][d]);
        }
        y = l == 0.0f ? f4{} : y / l;
        if (whole) {
          if (token < w.r.n) {
            const size_t at = (size_t)(w.r.row0 + token) * a.Hq + w.h * group + line - token * group;
            store4_as(a.y, at * a.c.D + d, a.c.dtype, y);
            if (a.lse && d == 0) a.lse[at] = (m + __builtin_amdgcn_logf(l)) * kLn2;
          }
        } else {
          *reinterpret_cast<f4*>(part + (size_t)row * a.c.D + d) = y;
          if (d == 0) {
            part[kRows * a.c.D + row] = m;
            part[kRows * a.c.D + kRows + row] = l;
          }
        }
      }
      left -= s1 - s0;
      rest += s1 - s0;
      first_part = false;
    }
    ++seq;
    rest = 0;
  }
}

// Joins the parts of the units that more than one workgroup had, always in the same order.
__global__ __launch_bounds__(kThreads) void attention_join_kernel(AttentionArgs a) {
  __shared__ int64_t parts[kWaves];
  __shared__ int64_t found_before;
  __shared__ int found_seq;
  const int t = blockIdx.x, h = blockIdx.y, group = a.Hq / a.c.H;
  if (threadIdx.x == 0) found_seq = -1;
  int64_t total = 0, before;
  for (int base = 0; base < a.c.S; base += kThreads) {
    const int i = base + threadIdx.x;
    const int64_t own = i < a.c.S ? cost_of(a, i) : 0, all = block_scan<kWaves>(own, before, parts);
    if (own > 0) {
      const Rows r = rows_of(a.c, i);
      if (t >= r.row0 && t < r.row0 + r.n) {
        found_seq = i;
        found_before = total + before;
      }
    }
    total += all;
  }
  __syncthreads();
  const int seq = found_seq;
  if (seq < 0) return;
  const Rows r = rows_of(a.c, seq);
  const int count = steps_of(a, r).count(), tiles = tiles_of(a, r);
  const Deal deal(total);
  const int quads = a.c.D / 4;
  for (int x = threadIdx.x; x < group * quads; x += kThreads) {
    const int head = x / quads, d = 4 * (x - head * quads), line = (t - r.row0) * group + head;
    const int64_t first = found_before + (int64_t)(h * tiles + line / kRows) * count;
    const int w0 = deal.owner(first), w1 = deal.owner(first + count - 1), row = line % kRows;
    if (w0 == w1) continue;
    float m = -__builtin_inff(), l = 0.0f;
    for (int w = w0; w <= w1; ++w) {
      const float* part = a.scratch + (size_t)(2 * w + (deal.first(w) < first ? 1 : 0)) * part_floats(a.c.D);
      m = fmaxf(m, part[kRows * a.c.D + row]);
    }
    f4 y{};
    for (int w = w0; w <= w1; ++w) {
      const float* part = a.scratch + (size_t)(2 * w + (deal.first(w) < first ? 1 : 0)) * part_floats(a.c.D);
      const float e = __builtin_amdgcn_exp2f(part[kRows * a.c.D + row] - above(m)) * part[kRows * a.c.D + kRows + row];
      l += e;
      y += e * *reinterpret_cast<const f4*>(part + (size_t)row * a.c.D + d);
    }
    y = l == 0.0f ? f4{} : y / l;
    const size_t at = (size_t)t * a.Hq + h * group + head;
    store4_as(a.y, at * a.c.D + d, a.c.dtype, y);
    if (a.lse && d == 0) a.lse[at] = (m + __builtin_amdgcn_logf(l)) * kLn2;
  }
}

template <int kTerms>
void launch_terms(const AttentionArgs& a, hipStream_t stream) {
  switch ((a.c.D + 63) / 64) {
    case 1: attention_kernel<1, kTerms><<<kBlocks, kThreads, 0, stream>>>(a); break;
    case 2: attention_kernel<2, kTerms><<<kBlocks, kThreads, 0, stream>>>(a); break;
    case 3: attention_kernel<3, kTerms><<<kBlocks, kThreads, 0, stream>>>(a); break;
    default: attention_kernel<4, kTerms><<<kBlocks, kThreads, 0, stream>>>(a); break;
  }
}

}  // namespace

// Many rows a sequence: the kernel that shares a step's keys and values between 128 rows.
static bool tiles_pay(int T, int S, int Hq, int H) { return (int64_t)T * (Hq / H) >= 64 * (int64_t)S; }

size_t cache_attention_scratch_bytes(int T, int S, int Hq, int H, int D) {
  if (tiles_pay(T, S, Hq, H)) return attention_tiles_scratch_bytes(S, D);
  return (size_t)2 * kBlocks * part_floats(D) * sizeof(float);
}

hipError_t launch_cache_attention(const AttentionArgs& a, hipStream_t stream, bool* partial) {
  if (tiles_pay(a.c.T, a.c.S, a.Hq, a.c.H)) return launch_attention_tiles(a, stream, partial);
  if (a.c.dtype == SHERRY_F32) launch_terms<2>(a, stream);
  else launch_terms<1>(a, stream);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  *partial = true;
  attention_join_kernel<<<dim3(a.c.T, a.c.H), kThreads, 0, stream>>>(a);
  return hipGetLastError();
}

}  // namespace sherry
