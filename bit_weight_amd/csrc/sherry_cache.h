// The paged 8-bit cache of keys and values, as its kernels see it.
//
// A page holds `page` tokens of every head, in blocks of 16 tokens; a block of
// one head is 16 D bytes and has one scale.  Keys lie as [D / 16][16 tokens][16
// features] and values as [D / 16][16 features][16 tokens]: the 16 bytes that a
// matrix-core lane takes of either are contiguous, and 16 lanes' are 256 bytes.
// The block of page p, head h, number b is number (p H + h) blocks + b.
//
// Sequence i owns rows starts[i] .. starts[i + 1] - 1 of what a call brings or
// asks for; they are its last tokens, at positions up to lens[i] - 1.  Position
// t lies in page table[i][t / page].  What these arrays say is never trusted:
// rows, table slots and pages are checked before they become addresses.
#pragma once

#include "sherry_device.h"
#include "sherry_launch.h"
#include "sherry_types.h"

namespace sherry {

constexpr int kBlockTokens = 16;

struct Rows {       // a sequence's part of a call
  int row0, n;      // its rows
  int len;          // tokens it has (with the call's)
};

__device__ __forceinline__ Rows rows_of(const CacheArgs& c, int i) {
  const int a = min(max(c.starts[i], 0), c.T), b = min(max(c.starts[i + 1], a), c.T);
  return {a, b - a, min(max(c.lens[i], 0), 1 << 30)};
}

// The page of 16-token block sb of sequence i, or -1.
__device__ __forceinline__ int page_of(const CacheArgs& c, int i, int sb) {
  const int slot = sb >> c.block_shift;
  if (sb < 0 || slot >= c.table_width) return -1;
  const int p = c.table[(size_t)i * c.table_width + slot];
  return p >= 0 && p < c.pages ? p : -1;
}

// Number of the block sb of a page and head.
__device__ __forceinline__ size_t block_of(const CacheArgs& c, int page, int h, int sb) {
  return (((size_t)page * c.H + h) << c.block_shift) + (sb & ((1 << c.block_shift) - 1));
}

// Blocks that the rows of a sequence lie in: the first and how many (also at
// positions below 0, which no page has).
__device__ __forceinline__ int2 blocks_of(const Rows& r) {
  if (r.n == 0) return make_int2(0, 0);
  const int first = (r.len - r.n) >> 4;
  return make_int2(first, ((r.len - 1) >> 4) - first + 1);
}

// Item w of those that the sequences have count(i) of, one after another: its
// sequence and number there, or false past the last.  A wave's lanes count 64
// sequences at a time; the answer is the same in every lane.
template <typename F>
__device__ __forceinline__ bool find_item(int S, int w, F count, int& seq, int& number) {
  const int lane = threadIdx.x & 63;
  for (int base = 0; base < S; base += 64) {
    const int own = base + lane < S ? count(base + lane) : 0;
    int sum = own;
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
      const int v = __shfl_up(sum, d);
      if (lane >= d) sum += v;
    }
    const uint64_t past = __ballot(sum > w);
    if (past) {
      const int at = __ffsll((unsigned long long)past) - 1;
      seq = base + at;
      number = w - (__builtin_amdgcn_readlane(sum, at) - __builtin_amdgcn_readlane(own, at));
      return number >= 0 && number < __builtin_amdgcn_readlane(own, at);
    }
    w -= __builtin_amdgcn_readlane(sum, 63);
  }
  return false;
}

}  // namespace sherry
