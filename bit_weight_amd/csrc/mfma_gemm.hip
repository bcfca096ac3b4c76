// Kernel 4: large-M (prefill) product.  The 5-bit codes are decoded to int8
// {-1,0,+1} and contracted with the int8 activations on the gfx950 matrix
// cores (v_mfma_i32_16x16x64_i8, int32 accumulation), followed by the same
// float rescale as the lookup path: y = ((float)acc * s_x[m]) * alpha[n].
// Decoding inside the int8 GEMM's prologue follows the fused
// decode-then-int8-GEMM structure the OdysseyLLM FastGEMM review describes
// for W4A8 (xllm-io page, FastGEMM section).
//
// Workgroup tile: BM = 128 activation rows x BN = 256 weight rows (4 format
// row tiles), k-steps of one format k-tile (128 inputs); 8 waves, two per
// SIMD: wave (kh, w) takes the k-tiles of phase kh (2j + kh) of row tile w,
// i.e. 64 weight rows = 4 MFMA column blocks, against all 128 activation
// rows = 8 MFMA row blocks (8 x 4 accumulators); the two phases' sums are
// added in the epilogue.  On a small grid the 8 waves split instead into 2
// row tiles x KP = 4 k-phases (BN = 128, k-tiles 4j + kh): twice the
// workgroups, each a quarter of K per wave; BM = 64 halves the tile again.
// A decoded weight operand therefore feeds 8 MFMAs and an activation
// fragment 4, which keeps the LDS work per k-tile (pair-table lookups plus
// activation fragments) well below the matrix-core time.
//  * activations: 128 x 128 int8 per k-step, copied once per workgroup
//    straight from global memory into LDS by buffer loads with LDS return
//    (no registers on the way), 8 lanes per 128-byte row so every load reads
//    whole lines; rows sit in a row-major tile whose 16-byte chunks are
//    XOR-swizzled (see a_off) so the MFMA A reads (16 rows, one chunk) hit 16
//    different bank groups.  Three buffers per phase: the copy for k-step
//    j+2 starts right after the barrier of step j, once every wave is done
//    with the buffer it overwrites, and has two steps to land (two buffers
//    and one step with BM = 128 and 4 phases, whose 12 x 16 KB would not
//    fit LDS; with BM = 64 four buffers and one barrier per two steps);
//  * weights: each wave decodes exactly the B operands it consumes.  It loads
//    its row tile's 1280-byte k-tile coalesced (lane l = slot l, 16 + 4
//    bytes), which by the format's design already holds, for column block t,
//    weight row 16t + l%16 and, for lane group g = l/16, codes 8g..8g+7 of
//    the k-tile (inputs 32g..32g+31: the first half in MFMA sub-step 0, the
//    second in sub-step 1): dword t and byte t of the slot's last dword.  The
//    A operands use the same input order, which a dot product does not see.
//    A 1024-entry LDS table maps a 10-bit code pair to its 8 int8 weights,
//    so 4 codes cost two 8-byte lookups;
//  * codes come through a buffer descriptor into two register stages used
//    in turn; a k-step's codes are decoded (table lookups) between the
//    MFMAs of the step before it, so the LDS lookups overlap matrix-core
//    work, and the 64 MFMAs of a step run back to back with the A reads two
//    row blocks ahead.  The barrier waits for exactly the activation copy of
//    its own step (a counted vmcnt), so the newer loads stay in flight
//    across it.
// The same kernel with another epilogue (EP) forms the feed-forward products:
// bias, activation and residual; the gated block, whose workgroup pairs the
// gate's and the up matrix's row tiles of the same outputs, so act(g) u is
// formed where both sums meet and neither is ever written; and the backward
// passes' recomputed sums, whose epilogue writes the pre-activations'
// gradients in scaled fp16 and partial column sums of dalpha and dbias.  The
// epilogue takes its sums through LDS 16 rows at a time, its other inputs
// requested together ahead of it.  The main loop bounds all of them (bf16,
// K = 4096, N = 14336: gated M=512 59.5 us, 2.02 POP/s; its backward sums at
// M=2048 254 us, 1.89 POP/s with the epilogue; K = 14336, N = 4096, M=512
// 33 us, 1.8 POP/s; the vendor's int8 product reaches 2.70 POP/s at 8192^3,
// and 1.54 and 2.26 on the two gated shapes).
// Tiles are numbered so that the 8 XCDs (workgroups are dealt round-robin)
// each own a slab of weight rows, which then stays in that XCD's L2 for all
// activation tiles.
#include "sherry_device.h"
#include "sherry_grad.h"
#include "sherry_launch.h"
#include "sherry_types.h"

namespace sherry {
namespace {

typedef int v4i __attribute__((ext_vector_type(4)));
typedef unsigned int v4u __attribute__((ext_vector_type(4)));

constexpr int kNT = kTileRows / 16;             // 4 column blocks per wave (one row tile)
constexpr int kBK = kTileK;                     // 128
constexpr int kThreads = 512;                   // 8 waves: row tiles x k-phases

// The sizes that follow from the tile height BM (128 or 64 activation rows)
// and the number of k-phases KP (2 or 4).
template <int BM, int KP>
struct Tiling {
  static_assert(KP == 2 || KP == 4, "k-phases: 2 or 4");
  // 64-row tiles: one barrier per two k-steps, four activation buffers per
  // k-phase, the copies for steps j+2 and j+3 issued in step j (measured at
  // K=4096: M=128, N=14336 14.5 -> 13.6 us; M=320, N=11008 20.9 -> 20.5;
  // no faster with 128-row tiles).  Else a barrier per k-step with three
  // buffers (the copy for step j+2 issued in step j), or two with 128-row
  // tiles and 4 phases, whose 4 x 3 x 16 KB would not fit LDS (the copy for
  // step j+1 issued in step j).
  static constexpr bool kPair = BM <= 64;
  static constexpr int kABufs = kPair ? 4 : (BM == 128 && KP == 4 ? 2 : 3);
  static constexpr int kRT = kThreads / 64 / KP;       // row tiles per workgroup (4 or 2)
  static constexpr int kBN = kRT * kTileRows;          // workgroup tile width (256 or 128 weight rows)
  // Words per row of the epilogue tiles.  One sums write (an accumulator
  // register of every lane) puts rows r, r+4, r+8, r+12 of an MFMA block in
  // lanes 0-15, 16-31, 32-47, 48-63; a pitch of 4 (mod 16) words spaces
  // those rows 16 banks apart, so no two lanes of a write share a bank.  (At
  // kBN + 16 the four rows were 1088 words, a multiple of 64, apart: measured
  // with the padded pitch, M=512, N=14336, K=4096 31.4 -> 31.1 us; M=256
  // 20.5 -> 19.9; M=128 13.7 -> 13.5.)
  static constexpr int kOutLd = kBN + 4;
  static constexpr int kLdsOut = KP * 32 * kOutLd * 4; // epilogue tiles (32 rows, every phase)
  static constexpr int kLdsTile = KP * 16 * kOutLd * 4;   // 16 rows of them (epilogues other than kEpNone)
  static constexpr int kMT = BM / 16;                  // row blocks per wave (8 or 4)
  static constexpr int kAStage = BM * kBK;             // activation bytes per k-step
  static constexpr int kRowsPerWave = BM / kRT;        // rows each wave of a phase copies
  static constexpr int kACopies = kRowsPerWave / 8;    // 1 KB copies (8 rows) per wave per k-step
  static constexpr int kLdsMain = KP * kABufs * kAStage;  // activation buffers x phases
  static constexpr int kLdsBytes = kLdsMain > kLdsOut ? kLdsMain : kLdsOut;
  // vector-memory ops a wave issues between a k-step's activation copy and
  // that step's barrier: with three buffers the codes three steps ahead of
  // it (2), the next step's copy, and the codes four steps ahead (2); with
  // two, the codes two steps ahead of it (2); with a barrier per two steps
  // (the copy of steps j, j+1 issued at step j-2), the codes of steps j+1
  // and j+2 (2 + 2)
  static constexpr int kNewerLoads = kPair ? 4 : (kABufs == 3 ? 2 + kACopies + 2 : 2);
};

template <int I>
using Const = std::integral_constant<int, I>;

// Activation tile in LDS, row-major with 128-byte rows: the 16-byte chunk c
// of row r sits at chunk position c ^ ((r >> 1) & 7).  A fragment read (16
// consecutive rows, one chunk) then spreads over all 16 bank groups of a
// 256-byte bank period, and 8 lanes copying one row fill one row.
__device__ __forceinline__ int a_off(int r, int c) { return (r * 8 + (c ^ ((r >> 1) & 7))) * 16; }

// s_waitcnt operand: vmcnt(vm), lgkmcnt(0), expcnt not waited.
constexpr int waitcnt_vm_lgkm0(int vm) { return (vm & 15) | ((vm >> 4) << 14) | 0x70; }

// B operands of one column block and sub-step: 4 codes (20 bits of v) as
// two code pairs, one 8-byte table entry each.
__device__ __forceinline__ v4i mg_decode4(uint32_t v, const uint8_t* dec2) {
  const uint2 e0 = *reinterpret_cast<const uint2*>(dec2 + ((v << 3) & 0x1FF8u));
  const uint2 e1 = *reinterpret_cast<const uint2*>(dec2 + ((v >> 7) & 0x1FF8u));
  return v4i{(int)e0.x, (int)e0.y, (int)e1.x, (int)e1.y};
}

// The 2 x MT x 4 MFMAs of one k-step (sub-steps s = 0, 1 read A chunk 2g+s
// of the tile at `as`, with B operands b0 / b1), and the table lookups that
// decode the next k-step's codes (f0 / f1) into n0 / n1: those of sub-step
// 0 spread over the groups of 8 MFMAs of sub-step 1 (b0 is dead by then, so
// n0 can take its registers), those of sub-step 1 after the MFMAs.  The A
// fragments of the next two row blocks are requested before the MFMAs of
// the current two, so the LDS latency hides behind 8 MFMAs.
template <bool kLive, int kMT>
__device__ __forceinline__ void mg_mfma(v4i (&acc)[kMT][kNT], const v4i (&b0)[kNT],
                                        const v4i (&b1)[kNT], const int8_t* as, int l16, int g,
                                        const uint32_t (&f0)[kNT], const uint32_t (&f1)[kNT],
                                        v4i (&n0)[kNT], v4i (&n1)[kNT], const uint8_t* dec2) {
  auto frag = [&](int u) {   // u = kMT s + row block
    return *reinterpret_cast<const v4i*>(as + a_off(16 * (u % kMT) + l16, 2 * g + u / kMT));
  };
  constexpr int kDecPerGroup = kNT / (kMT / 2);   // sub-step-0 lookups per group of sub-step 1
  v4i a0{0, 0, 0, 0}, a1{0, 0, 0, 0};
  if constexpr (kLive) {
    a0 = frag(0);
    a1 = frag(1);
  }
#pragma unroll
  for (int u = 0; u < 2 * kMT; u += 2) {
    v4i p0 = a0, p1 = a1;
    if (kLive && u + 2 < 2 * kMT) {
      p0 = frag(u + 2);
      p1 = frag(u + 3);
    }
    if (u >= kMT) {
#pragma unroll
      for (int d = 0; d < kDecPerGroup; ++d) {
        const int t = ((u - kMT) >> 1) * kDecPerGroup + d;
        n0[t] = mg_decode4(f0[t], dec2);
      }
    }
    __builtin_amdgcn_sched_barrier(0);
    if constexpr (kLive) {
      const int i = u % kMT;
#pragma unroll
      for (int c = 0; c < kNT; ++c)
        acc[i][c] = __builtin_amdgcn_mfma_i32_16x16x64_i8(a0, u < kMT ? b0[c] : b1[c], acc[i][c], 0, 0, 0);
#pragma unroll
      for (int c = 0; c < kNT; ++c)
        acc[i + 1][c] = __builtin_amdgcn_mfma_i32_16x16x64_i8(a1, u < kMT ? b0[c] : b1[c], acc[i + 1][c], 0, 0, 0);
    }
    __builtin_amdgcn_sched_barrier(0);
    a0 = p0;
    a1 = p1;
  }
#pragma unroll
  for (int t = 0; t < kNT; ++t) n1[t] = mg_decode4(f1[t], dec2);
}

// 16 bytes per lane from the buffer at byte `voffset` straight into LDS at
// dst + 16 * lane (a buffer load with LDS return).  A plain function, not a
// lambda inside the kernel template: there the host pass rejects the LDS
// address-space cast and silently drops the kernel's host-side stub.
__device__ __forceinline__ void copy16_to_lds(__amdgpu_buffer_rsrc_t r, int8_t* dst, int voffset) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (__attribute__((address_space(3))) void*)dst, 16, voffset, 0, 0,
                                           0);
}

__device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer_rsrc(const void* base, size_t bytes) {
  const int n = bytes > 0x7FFFFFFFull ? 0x7FFFFFFF : (int)bytes;
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), 0, n, 0x00020000);
}

// One workgroup's tile (mt_idx, nt_idx) of the product.  kAgain: the gradients
// of a token tile whose scale the first pass found too small (backward only).
template <int BM, int KP, int EP, bool kAgain>
__device__ __forceinline__ void product_tile(GemmArgs a, EpilogueOf<EP> e, int M, int N, int K, int mt_idx, int nt_idx) {
  using T = Tiling<BM, KP>;
  constexpr int kBM = BM, kMT = T::kMT, kAStage = T::kAStage, kACopies = T::kACopies;
  constexpr int kLdsBytes = T::kLdsBytes, kNewerLoads = T::kNewerLoads;
  constexpr int kRT = T::kRT, kBN = T::kBN, kOutLd = T::kOutLd;
  constexpr bool kOwn = EP != kEpNone;
  constexpr int kABufs = kOwn && T::kABufs == 3 ? 4 : T::kABufs;
  constexpr bool kPair = T::kPair;
  // gated: half of the workgroup's row tiles are the gate's, half the up
  // matrix's of the same kBNO outputs
  constexpr bool kGlu = ep_glu(EP);
  constexpr int kRTO = kGlu ? kRT / 2 : kRT, kBNO = kRTO * kTileRows;
  // the activation buffers [buffer][phase]; after the main loop the
  // epilogue tile reuses them
  // (32-bit words: every view below is a character type or 32-bit lanes)
  // With an epilogue every buffer is an array of its own, picked by a
  // constant, the first one large enough for the epilogue tile: the compiler
  // then sees that a step's fragment reads cannot touch what the copies in
  // flight write.  From one array it waits, before a step's first fragment,
  // for the copies that step has just issued.  (Measured, with 16 instead of
  // 32 rows per epilogue turn: 64-token tiles, M=512, K=14336, N=4096 39.3 ->
  // 34.4 us; 128-token tiles, M=512, K=4096, gated N=14336 62.5 -> 62.0.)
  constexpr int kBuf = KP * kAStage / 4, kFirst = kBuf * 4 > T::kLdsTile ? kBuf : T::kLdsTile / 4;
  __shared__ __attribute__((aligned(16))) uint32_t lds[kOwn ? kFirst : kLdsBytes / 4];
  __shared__ __attribute__((aligned(16))) uint32_t lds1[kOwn ? kBuf : 4];
  __shared__ __attribute__((aligned(16))) uint32_t lds2[kOwn && kABufs > 2 ? kBuf : 4];
  __shared__ __attribute__((aligned(16))) uint32_t lds3[kOwn && kABufs > 3 ? kBuf : 4];
  // the pair table in an array of its own: the compiler then sees that its
  // lookups cannot read what an activation copy in flight is writing.  Its
  // alignment places it first in LDS, below 64 KB, so a lookup's table base
  // folds into the instruction's offset field instead of costing a VALU OR
  // per lookup (measured at M=512, K=4096, N=14336: 32.7 -> 31.9 us)
  __shared__ __attribute__((aligned(1024))) uint2 dec2[1024];
  __shared__ float sxs[kBM];   // s_x of this tile's rows (epilogue)
  // with an epilogue, also its other factors, loaded ahead of the main loop:
  // the gradients' scales, and alpha and alpha2 (or the bias) of the outputs
  constexpr bool kBack = ep_back(EP);
  __shared__ float inv_rows[kBack ? kBM : 1];
  __shared__ __attribute__((aligned(16))) float cols[2][kOwn ? kBNO : 4];
  // the largest |z| of each row in this tile (as the float's bits)
  constexpr bool kTops = kBack && !kAgain;
  __shared__ unsigned row_tops[kTops ? kBM : 1];
  // arrivals at the step barrier of each k-tile parity (128-row tiles)
  __shared__ unsigned parity_arrivals[KP];

  const int KT = k_tiles(K), RT = row_tiles(N);
  const int m0 = mt_idx * kBM, n0 = nt_idx * kBNO;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wv = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wave = wv % kRT, kh = wv / kRT;        // row tile, k-phase
  const int l16 = lane & 15, g = lane >> 4;

  if (tid < KP) parity_arrivals[tid] = 0u;   // published by the prologue's barrier
  if constexpr (kTops) {
    if (tid < kBM) row_tops[tid] = 0u;
  }
  // decode table: code pair (c0 | c1 << 5) -> the 8 int8 weights of both
  for (int i = tid; i < 1024; i += kThreads)
    dec2[i] = make_uint2(code_word(i & 31), code_word(i >> 5));

  // This wave's row tile.  One wholly past N (N not a multiple of 256)
  // streams the last row tile again and stores nothing.  In a ragged last
  // row tile (N % 64 != 0) the padding rows decode code 0, the block
  // (0,+1,+1,+1), and form sums of their own: only the n < N mask of the
  // epilogue's stores keeps them out of the output.
  const int rt_raw = n0 / kTileRows + wave % kRTO;
  const bool n_live = rt_raw < RT;
  const int rt = n_live ? rt_raw : RT - 1;
  const uint8_t* codes = a.packed;
  if constexpr (kGlu) codes = wave < kRTO ? a.packed : e.packed2;
  const __amdgpu_buffer_rsrc_t rc =
      buffer_rsrc(codes + tile_offset(rt, 0, KT), (size_t)KT * kTileBytes);
  const __amdgpu_buffer_rsrc_t ra =
      buffer_rsrc(a.x + (size_t)m0 * K, (size_t)(M - m0) * (size_t)K);

  // activations: the kRT waves of a phase copy its k-tile, BM rows x 128
  // bytes; copy jj of wave `wave` fills rows (BM/kRT) wave + 8 jj .. +7, lane
  // L taking chunk (L & 7) ^ swizzle of row L >> 3 (its LDS position is
  // fixed at 16 L).  Rows past M read row M-1 (they feed only unstored rows).
  int a_v[kACopies];
#pragma unroll
  for (int jj = 0; jj < kACopies; ++jj) {
    const int row = T::kRowsPerWave * wave + 8 * jj + (lane >> 3);
    const int c = (lane & 7) ^ ((row >> 1) & 7);
    a_v[jj] = min(row, M - 1 - m0) * K + c * 16;
  }
  // first input of a copy's chunk in its k-step: the swizzle (row >> 1) & 7
  // of row (BM/kRT) wave + 8 jj + (lane >> 3) is 4 (jj & 1) + (lane >> 4)
  // (BM/kRT is a multiple of 16)
  static_assert(T::kRowsPerWave % 16 == 0, "rows per wave: a multiple of 16");
  int a_k[2];
#pragma unroll
  for (int p = 0; p < 2; ++p) a_k[p] = 16 * ((lane & 7) ^ (4 * p + (lane >> 4)));
  // an offset the descriptor's range check rejects (the copy writes zeros)
  const int a_oob = (size_t)(M - m0) * (size_t)K > 0x7FFFFFFFull ? 0x7FFFFFFF : (M - m0) * K;
  auto a_buf = [&](int b) { return reinterpret_cast<int8_t*>(lds) + (b * KP + kh) * kAStage; };
  auto own_buf = [&](auto b) __attribute__((always_inline)) {
    constexpr int i = decltype(b)::value % kABufs;
    return reinterpret_cast<int8_t*>(i == 0 ? lds : i == 1 ? lds1 : i == 2 ? lds2 : lds3) + kh * kAStage;
  };

  v4i acc[kMT][kNT];
#pragma unroll
  for (int i = 0; i < kMT; ++i)
#pragma unroll
    for (int t = 0; t < kNT; ++t) acc[i][t] = v4i{0, 0, 0, 0};

  // this wave's k-tile of step j (KP j + kh, clamped: a prefetch past the
  // end re-reads the last k-tile)
  const int KJ = (KT + KP - 1) / KP;
  auto ktile = [&](int j) { return min(KP * j + kh, KT - 1); };
  // codes, coalesced (lane = tile row)
  auto load_codes = [&](int j, v4u& w, uint32_t& h) __attribute__((always_inline)) {
    const int ks = ktile(j) * kTileBytes;
    w = __builtin_amdgcn_raw_buffer_load_b128(rc, 16 * lane, ks, 0);
    h = __builtin_amdgcn_raw_buffer_load_b32(rc, kTileHiOff + 4 * lane, ks, 0);
  };
  // this wave's share of the activation tile of step j into buffer b
  auto copy_a = [&](int j, int8_t* buf) __attribute__((always_inline)) {
    const int ka = ktile(j) * kBK;
    int8_t* dst = buf + T::kRowsPerWave * wave * kBK;
    // (the k-step offset is added to the lane offset, not passed as the
    // scalar offset, so the descriptor's range check sees the whole offset;
    // chunks past K, in a ragged last k-tile whose codes are padding, take
    // an out-of-range offset and land as zeros)
#pragma unroll
    for (int jj = 0; jj < kACopies; ++jj)
      copy16_to_lds(ra, dst + 8 * jj * kBK, ka + a_k[jj & 1] < K ? a_v[jj] + ka : a_oob);
  };
  const uint8_t* d2 = reinterpret_cast<const uint8_t*>(dec2);
  // the 20-bit code groups of one register stage: lane (l16, g) of block t
  // holds codes 8g..8g+3 of row 16t+l16 (sub-step 0) in the low 20 bits of
  // dword t, and codes 8g+4..8g+7 (sub-step 1) in its top 12 bits and byte t
  // of h.  The empty asm statements make the compiler form both halves here,
  // in registers of their own: left to itself it reads f0 out of the stage
  // registers and forms f1 late, so the code load into the stage that
  // follows gets fresh registers and the loop's back edge copies them back
  // after waiting for every load (measured at N=14336, K=4096: M=128 22.9
  // against 20.5 us with them).
  auto split = [&](const v4u& w, uint32_t h, uint32_t (&f0)[kNT], uint32_t (&f1)[kNT]) __attribute__((always_inline)) {
    const uint32_t wt[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int t = 0; t < kNT; ++t) {
      f0[t] = wt[t];
      f1[t] = __builtin_amdgcn_alignbit(h >> (8 * t), wt[t], 20);
      asm volatile("" : "+v"(f0[t]), "+v"(f1[t]));
    }
  };
  // Step j (activation buffer b = j % kABufs): its B operands bc0 / bc1 were
  // decoded during step j-1; the register stage (wn, hn) holds the codes of
  // step j+1, decoded during this step's MFMAs into bn0 / bn1 and then
  // refilled with the codes of step j+3.
  // The step barrier.  With 128-row tiles it joins only the kRT waves of
  // this wave's k-phase, which share that phase's activation buffers and
  // nothing else until the epilogue: an LDS arrival count per phase, so the
  // phases' waves (two to a SIMD) need not leave each step together
  // (measured at N=14336, K=4096: M=512 31.7 -> 30.6 us, M=1024 66.6 ->
  // 60.6; with 64-row tiles it was 2 % slower, so those keep s_barrier).
  // The arrival and the polls are LDS instructions in asm: as built-ins the
  // compiler cannot tell them from the activation copies in flight and waits
  // for those first.  The poll is bounded (~0.3 s), so a wave always leaves.
  auto parity_barrier = [&](int j) __attribute__((always_inline)) {   // j: the barrier's index
    const uint32_t pa = (uint32_t)(size_t)((__attribute__((address_space(3))) unsigned*)&parity_arrivals[kh]);
    if (lane == 0) asm volatile("ds_add_u32 %0, %1" ::"v"(pa), "v"(1u) : "memory");
    const unsigned target = (unsigned)kRT * (unsigned)(j + 1);
#pragma unroll 1
    for (int spin = 0; spin < (1 << 22); ++spin) {
      unsigned c;
      asm volatile("ds_read_b32 %0, %1\n\ts_waitcnt lgkmcnt(0)" : "=v"(c) : "v"(pa) : "memory");
      if (__builtin_amdgcn_readfirstlane(c) >= target) break;
      __builtin_amdgcn_s_sleep(1);
    }
  };
  // `even`: j is even (a constant at every call), so with a barrier per two
  // steps the odd steps fold to the decode and the MFMAs.
  // `as`: the buffer it reads; `to`, `to2`: those its copies go to.
  auto step_on = [&](int j, const int8_t* as, int8_t* to, int8_t* to2, bool even, v4u& wn, uint32_t& hn, const v4i (&bc0)[kNT],
                  const v4i (&bc1)[kNT], v4i (&bn0)[kNT], v4i (&bn1)[kNT]) __attribute__((always_inline)) {
    // every wave's copy of step j (and j+1) has landed and its earlier LDS
    // reads are done; then the buffer of step j-1 is free for the copy of
    // step j+2 (those of j-2, j-1 for j+2, j+3)
    if (!kPair || even) {
      __builtin_amdgcn_sched_barrier(0);
      __builtin_amdgcn_s_waitcnt(waitcnt_vm_lgkm0(kNewerLoads));
      __builtin_amdgcn_sched_barrier(0);
      if constexpr (BM == 128)
        parity_barrier(j);
      else
        __builtin_amdgcn_s_barrier();
      __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
      __builtin_amdgcn_sched_barrier(0);
      if constexpr (kPair) {
        copy_a(min(j + 2, KJ - 1), to);
        copy_a(min(j + 3, KJ - 1), to2);
      } else if constexpr (kABufs >= 3) {
        copy_a(min(j + 2, KJ - 1), to);
      } else {
        copy_a(min(j + 1, KJ - 1), to);
      }
      __builtin_amdgcn_sched_barrier(0);
    }
    uint32_t f0[kNT], f1[kNT];
    split(wn, hn, f0, f1);
    load_codes(min(j + 3, KJ - 1), wn, hn);
    __builtin_amdgcn_sched_barrier(0);
    if (KP * j + kh < KT)    // KT not a multiple of KP: the last step is short
      mg_mfma<true, kMT>(acc, bc0, bc1, as, l16, g, f0, f1, bn0, bn1, d2);
    else
      mg_mfma<false, kMT>(acc, bc0, bc1, as, l16, g, f0, f1, bn0, bn1, d2);
  };
  auto step = [&](int j, int b, bool even, v4u& wn, uint32_t& hn, const v4i (&bc0)[kNT],
                  const v4i (&bc1)[kNT], v4i (&bn0)[kNT], v4i (&bn1)[kNT]) {
    int8_t* to = a_buf(kPair ? (b + 2) & 3 : kABufs == 3 ? (b == 0 ? 2 : b - 1) : b ^ 1);
    step_on(j, a_buf(b), to, kPair ? a_buf((b + 3) & 3) : to, even, wn, hn, bc0, bc1, bn0, bn1);
  };

  // Two register stages of codes and two sets of B operands, ping-pong.
  // Issue order (the barrier's vmcnt counts on it): codes 0, copy 0,
  // codes 1, copy 1 (three buffers only), codes 2, then per step j:
  // barrier, copy j+2 (j+1 with two buffers), codes j+3.  With a barrier
  // per two steps: codes 0, copy 0, copy 1, codes 1, codes 2, then per
  // even step j: barrier, copies j+2 and j+3, codes j+3; per odd step:
  // codes j+3.
  v4u w0, w1;
  uint32_t h0, h1;
  v4i bA0[kNT], bA1[kNT], bB0[kNT], bB1[kNT];
  float sx_in = 0.0f, al_in = 0.0f, al2_in = 0.0f;
  GradRow row_in{};
  float tops_in[3] = {0.0f, 0.0f, 0.0f};
  uint32_t largest_in = 0u;
  if constexpr (kOwn) {
    const int mi = min(m0 + tid, M - 1), ni = min(n0 + tid, N - 1);
    if (tid < kBM) {
      sx_in = a.s_x[mi];
      if constexpr (kBack) row_in = e.grad.rows[mi];
      if constexpr (kAgain) largest_in = e.grad.largest[mi];
    }
    if (tid < kBNO) {
      al_in = a.alpha[ni];
      if constexpr (kGlu) al2_in = e.alpha2[ni];
      else if (e.bias) al2_in = e.bias[ni];
    }
    if constexpr (kBack) {
#pragma unroll
      for (int i = 0; i < 3; ++i) tops_in[i] = e.grad.tops[i];
    }
    __builtin_amdgcn_sched_barrier(0);
  }
  load_codes(0, w0, h0);
  __builtin_amdgcn_sched_barrier(0);
  copy_a(0, kOwn ? own_buf(Const<0>{}) : a_buf(0));
  __builtin_amdgcn_sched_barrier(0);
  if constexpr (kPair) {
    copy_a(min(1, KJ - 1), kOwn ? own_buf(Const<1>{}) : a_buf(1));
    __builtin_amdgcn_sched_barrier(0);
  }
  load_codes(min(1, KJ - 1), w1, h1);
  __builtin_amdgcn_sched_barrier(0);
  if constexpr (!kPair && kABufs >= 3) copy_a(min(1, KJ - 1), kOwn ? own_buf(Const<1>{}) : a_buf(1));
  __builtin_amdgcn_sched_barrier(0);
  if constexpr (kOwn) {
    if (tid < kBM) {
      sxs[tid] = sx_in;
      if constexpr (kBack) {
        int exponent = first_exponent(row_in, sx_in, tops_in, e.act, kGlu);
        if constexpr (kAgain)
          exponent = last_exponent(exponent, largest_in, row_in, sx_in, tops_in, e.act, kGlu, e.grad.terms);
        inv_rows[tid] = exp2_of(exponent);
      }
    }
    if (tid < kBNO) {
      cols[0][tid] = al_in;
      cols[1][tid] = al2_in;
    }
    __builtin_amdgcn_sched_barrier(0);
  }
  // decode table written (LDS only: the copies stay in flight)
  __builtin_amdgcn_s_waitcnt(waitcnt_vm_lgkm0(63));
  __builtin_amdgcn_s_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
  __builtin_amdgcn_sched_barrier(0);
  {
    uint32_t f0[kNT], f1[kNT];
    split(w0, h0, f0, f1);
#pragma unroll
    for (int t = 0; t < kNT; ++t) {
      bA0[t] = mg_decode4(f0[t], d2);
      bA1[t] = mg_decode4(f1[t], d2);
    }
    load_codes(min(2, KJ - 1), w0, h0);
    __builtin_amdgcn_sched_barrier(0);
  }

  if constexpr (kOwn) {
    // steps in turns of kABufs, a multiple of the 2 register stages (with
    // 128 x 256 tiles four buffers, not three, for that)
    static_assert(kABufs % 2 == 0, "a step's register stage follows from its buffer");
    auto own_step = [&](int j, auto u) __attribute__((always_inline)) {
      constexpr int i = decltype(u)::value;
      int8_t* as = own_buf(u);
      int8_t* to = own_buf(Const<i + (kABufs == 2 ? 1 : 2)>{});
      int8_t* to2 = own_buf(Const<i + 3>{});
      if constexpr (i % 2 == 0) step_on(j, as, to, to2, true, w1, h1, bA0, bA1, bB0, bB1);
      else step_on(j, as, to, to2, false, w0, h0, bB0, bB1, bA0, bA1);
    };
    int j = 0;
    for (; j + kABufs <= KJ; j += kABufs) {
      own_step(j, Const<0>{});
      own_step(j + 1, Const<1>{});
      if constexpr (kABufs > 2) {
        own_step(j + 2, Const<2>{});
        own_step(j + 3, Const<3>{});
      }
    }
    if (j < KJ) own_step(j, Const<0>{});
    if constexpr (kABufs > 2) {
      if (j + 1 < KJ) own_step(j + 1, Const<1>{});
      if (j + 2 < KJ) own_step(j + 2, Const<2>{});
    }
  } else {
    int j = 0, b = 0;
    for (; j + 2 <= KJ; j += 2) {
      step(j, b, true, w1, h1, bA0, bA1, bB0, bB1);
      b = b + 1 == kABufs ? 0 : b + 1;
      step(j + 1, b, false, w0, h0, bB0, bB1, bA0, bA1);
      b = b + 1 == kABufs ? 0 : b + 1;
    }
    if (j < KJ) step(j, b, true, w1, h1, bA0, bA1, bB0, bB1);
  }
  // the clamped copies past the end may still be landing in LDS, which the
  // epilogue reuses
  __builtin_amdgcn_s_waitcnt(waitcnt_vm_lgkm0(0));

  // Epilogue, 32 rows (two row blocks) at a time, 16 in the forms other than
  // kEpNone: every wave writes its raw int32 sums into its phase's row-major LDS tile, then each thread adds
  // the KP phases for 4 consecutive columns of one row and stores
  // y = ((float)acc * s_x[m]) * alpha[n] (or the int32 sum), 16 bytes per
  // lane, so each store instruction writes whole 128-byte lines, marked
  // non-temporal (the output is not read again here: measured 7 % faster at
  // M=512, N=14336, K=4096, where the 29 MB of fp32 output bound it).  Lane
  // (l16, g) of a 16 x 16 MFMA block holds column l16, rows 4g..4g+3.  The
  // scales are read once, before the first barrier.
  // The sums of the qq-th kTurnRows rows (row blocks) into this phase's LDS tile.
  constexpr int kTurnRows = kOwn ? 16 : 32, kTurnBlocks = kTurnRows / 16;
  int* ot = reinterpret_cast<int*>(lds);       // [phase][kTurnRows][kOutLd] sums
  int* mine = ot + kh * kTurnRows * kOutLd;
  auto put_sums = [&](int qq) {
#pragma unroll
    for (int ii = 0; ii < kTurnBlocks; ++ii)
#pragma unroll
      for (int r = 0; r < 4; ++r)
#pragma unroll
        for (int t = 0; t < kNT; ++t)
          mine[(16 * ii + 4 * g + r) * kOutLd + wave * kTileRows + 16 * t + l16] = acc[kTurnBlocks * qq + ii][t][r];
  };
  if constexpr (EP == kEpNone) {
    const bool want_y = a.y != nullptr;
    const int c4 = tid & (kBN / 4 - 1);          // this thread's 4 columns
    const int n = n0 + 4 * c4;
    float4 al4 = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    if (want_y && n < N) al4 = make_float4(a.alpha[n], a.alpha[n + 1], a.alpha[n + 2], a.alpha[n + 3]);
    if (want_y && tid < kBM) sxs[tid] = a.s_x[min(m0 + tid, M - 1)];
    // The scale loads complete here, before the first output store.  The
    // memory counter counts stores as well as loads, so a wait for alpha
    // placed after a store also waits for that store; left to itself the
    // compiler puts such a wait before every row's scaling, and the tile's
    // 16 rows of stores then leave one round trip at a time.
    __builtin_amdgcn_s_waitcnt(waitcnt_vm_lgkm0(0));
#pragma unroll
    for (int qq = 0; qq < kMT / 2; ++qq) {
      __syncthreads();  // the previous use of the LDS area is finished
      put_sums(qq);
      __syncthreads();
#pragma unroll
      for (int k = 0; k < 32 * (kBN / 4) / kThreads; ++k) {
        const int ml = tid / (kBN / 4) + (kThreads / (kBN / 4)) * k;   // row within the 32
        const int m = m0 + 32 * qq + ml;
        v4i sum = *reinterpret_cast<const v4i*>(&ot[ml * kOutLd + 4 * c4]);
#pragma unroll
        for (int ph = 1; ph < KP; ++ph) sum += *reinterpret_cast<const v4i*>(&ot[(ph * 32 + ml) * kOutLd + 4 * c4]);
        if (m < M && n < N) {
          if (want_y) {
            const float sx = sxs[32 * qq + ml];
            const float4 v = make_float4(((float)sum.x * sx) * al4.x, ((float)sum.y * sx) * al4.y,
                                         ((float)sum.z * sx) * al4.z, ((float)sum.w * sx) * al4.w);
            __builtin_nontemporal_store(__builtin_bit_cast(v4u, v), reinterpret_cast<v4u*>(a.y + (size_t)m * N + n));
          } else {
            __builtin_nontemporal_store(sum, reinterpret_cast<v4i*>(a.acc + (size_t)m * N + n));
          }
        }
      }
    }
  } else {
    constexpr int kCols = kBNO / 4;             // threads across a row: 4 outputs each
    constexpr int kRowStep = kThreads / kCols;  // rows the workgroup takes at a time
    static_assert(kRowStep <= kTurnRows ? kTurnRows % kRowStep == 0 : kRowStep == 2 * kTurnRows, "rows per turn");
    // (a row narrower than the workgroup can take in one turn: half the threads rest)
    constexpr int kTurns = kRowStep <= kTurnRows ? kTurnRows / kRowStep : 1;
    constexpr int kAll = kBM / kTurnRows * kTurns;   // rows per thread
    const int c4 = tid % kCols, r0 = tid / kCols;
    const int n = n0 + 4 * c4;
    // this thread's residuals or output gradients, all requested before the
    // first is used (up to four turns of them in 128 x 256 tiles' registers)
    constexpr int kAhead = kAll < 8 ? kAll : 8;
    u4 io[kAhead];
    const void* in = kBack ? e.grad.dy : e.residual;
    const bool has_in = !(EP == kEpGlu) && in && n < N && r0 < kTurnRows;
    const bool wide_in = e.dtype == SHERRY_F32;
    auto row_of = [&](int i) { return m0 + kTurnRows * (i / kTurns) + r0 + kRowStep * (i % kTurns); };
    auto load_in = [&](int first) __attribute__((always_inline)) {
#pragma unroll
      for (int i = 0; i < kAhead; ++i) io[i] = u4{0u, 0u, 0u, 0u};
      if (has_in && wide_in) {
#pragma unroll
        for (int i = 0; i < kAhead; ++i)
          if (row_of(first + i) < M) io[i] = load4_raw(in, (size_t)row_of(first + i) * N + n, SHERRY_F32);
      } else if (has_in) {
#pragma unroll
        for (int i = 0; i < kAhead; ++i)
          if (row_of(first + i) < M)   // (either 16-bit type)
            io[i] = load4_raw(in, (size_t)row_of(first + i) * N + n, SHERRY_F16);
      }
    };
    load_in(0);
    const f4 al = *reinterpret_cast<const f4*>(&cols[0][4 * c4]);
    const f4 second = *reinterpret_cast<const f4*>(&cols[1][4 * c4]);   // alpha2, or the bias
    const f4 al2 = kGlu ? second : f4{0.0f, 0.0f, 0.0f, 0.0f}, bias = second;
    f4 sum0{0.0f, 0.0f, 0.0f, 0.0f}, sum1 = sum0;   // this thread's share of dalpha and dalpha2 / dbias
    const int RT64 = RT * kTileRows;
    const size_t zrow = (size_t)e.grad.terms * (kGlu ? 2 : 1) * RT64;
#pragma unroll
    for (int qq = 0; qq < kMT / kTurnBlocks; ++qq) {
      if constexpr (kAll > kAhead) {
        if (qq > 0 && qq * kTurns % kAhead == 0) load_in(qq * kTurns);
      }
      __syncthreads();  // the previous use of the LDS area is finished
      put_sums(qq);
      __syncthreads();
#pragma unroll
      for (int k = 0; k < kTurns; ++k) {
        const int ml = r0 + kRowStep * k;
        const int m = m0 + kTurnRows * qq + ml;
        float top = 0.0f;   // largest |z| of this thread's columns
        if (m < M && n < (kBack ? RT64 : N) && r0 < kTurnRows) {
          v4i s1{0, 0, 0, 0}, s2{0, 0, 0, 0};
#pragma unroll
          for (int ph = 0; ph < KP; ++ph) {
            s1 += *reinterpret_cast<const v4i*>(&ot[(ph * kTurnRows + ml) * kOutLd + 4 * c4]);
            if constexpr (kGlu)
              s2 += *reinterpret_cast<const v4i*>(&ot[(ph * kTurnRows + ml) * kOutLd + kBNO + 4 * c4]);
          }
          const float sx = sxs[kTurnRows * qq + ml];
          const f4 in4 = as_f4(io[(qq * kTurns + k) % kAhead], e.dtype);
          f4 o{0.0f, 0.0f, 0.0f, 0.0f}, o2 = o;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float p1 = (float)s1[i] * sx, p2 = (float)s2[i] * sx;
            const float z = kGlu ? p1 * al[i] : p1 * al[i] + bias[i];
            if constexpr (EP == kEpFused) {
              o[i] = act_value(z, e.act) + in4[i];
            } else if constexpr (EP == kEpGlu) {
              o[i] = act_value(z, e.act) * (p2 * al2[i]);
            } else if constexpr (EP == kEpFusedBack) {
              float slope;
              activate<true>(z, e.act, slope);
              const float dz = in4[i] * slope;
              sum0[i] += dz * p1;
              sum1[i] += dz;
              o[i] = dz * al[i];
            } else {
              float slope;
              const float du = in4[i] * activate<true>(z, e.act, slope);
              const float dg = in4[i] * (p2 * al2[i]) * slope;
              sum0[i] += dg * p1;
              sum1[i] += du * p2;
              o[i] = dg * al[i];
              o2[i] = du * al2[i];
            }
          }
          if constexpr (!kBack) {
            store4_as(e.out, (size_t)m * N + n, e.dtype, o);
          } else {
            // rows past N inside the last row tile: zeros, so the padding adds nothing
            if (n >= N) o = o2 = f4{0.0f, 0.0f, 0.0f, 0.0f};
            _Float16* z = reinterpret_cast<_Float16*>(e.grad.z) + (size_t)m * zrow + n;
            const float scale = inv_rows[kTurnRows * qq + ml];
            store_terms(z, o * scale, e.grad.terms, (kGlu ? 2 : 1) * RT64);
            if constexpr (kGlu) store_terms(z + RT64, o2 * scale, e.grad.terms, 2 * RT64);
            if constexpr (kTops) {   // (a NaN does not count)
#pragma unroll
              for (int i = 0; i < 4; ++i) top = fmaxf(top, fmaxf(fabsf(o[i]), fabsf(o2[i])));
            }
          }
        }
        if constexpr (kTops) {
          // 16 lanes on 64 columns of one row, a row tile's: all in or all out
          top = row16_max(top);
          if (c4 % 16 == 0 && r0 < kTurnRows) atomicMax(&row_tops[kTurnRows * qq + ml], __builtin_bit_cast(unsigned, top));
        }
      }
    }
    if constexpr (kTops) {
      __syncthreads();
      if (tid < kBM && m0 + tid < M)
        __hip_atomic_fetch_max(e.grad.largest + m0 + tid, row_tops[tid], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      // the column sums of this token tile, its rows' threads joined in order
      f4* red = reinterpret_cast<f4*>(lds);
#pragma unroll
      for (int which = 0; which < 2; ++which) {
        __syncthreads();
        red[tid] = which ? sum1 : sum0;
        __syncthreads();
        float* part = which ? e.grad.part1 : e.grad.part0;
        if (r0 == 0 && n < N && part) {
          f4 t = red[c4];
#pragma unroll
          for (int r = 1; r < kRowStep; ++r) t += red[r * kCols + c4];
          float* p = part + (size_t)mt_idx * N + n;
          for (int i = 0; i < 4; ++i) p[i] = t[i];
        }
      }
    }
  }
}

template <int BM, int KP, int EP>
__global__ __launch_bounds__(kThreads) void mfma_gemm_kernel(const uint8_t* packed, const int8_t* x,
                                                             const float* xf, int M, int N, int K,
                                                             int n_tiles, int /*unused*/, const float* s_x,
                                                             const float* alpha, float* y, int32_t* acc_out,
                                                             int32_t* partials, EpilogueOf<EP> e) {
  const GemmArgs a = product_args(packed, x, xf, M, N, K, s_x, alpha, y, acc_out, partials);
  // tile id -> (m tile, n tile): consecutive ids of one XCD share n tiles
  const int id = blockIdx.x;
  const int mt_count = (M + BM - 1) / BM;
  const int xcd = id & 7, slot = id >> 3;
  const int per_xcd = (n_tiles + 7) / 8;            // n tiles owned by one XCD
  const int owned = slot / mt_count;
  const int mt_idx = slot - owned * mt_count;
  const int nt_idx = xcd * per_xcd + owned;
  if (nt_idx >= n_tiles || mt_idx >= mt_count) return;  // padding ids
  product_tile<BM, KP, EP, false>(a, e, M, N, K, mt_idx, nt_idx);
}

// The backward's gradients once more, for the token tiles with a token whose
// largest |z| passes fp16's range under its first scale, or lies so far below
// that the range costs it digits (sherry_grad.h): now under a scale of its own.  The others, as a rule
// all of them, are left after a look at their tokens; so that this look costs
// little, a grid of one round walks the tiles, `share` workgroups to a token
// tile: 4.7 us at M=2048, N=14336 gated, of 599, and 3.8 at M=77, N=1300, of 29.
// (As many workgroups as tiles would come and go in 14 rounds there.)  Where
// every token needs it, K=4096, fp32, relu2, two rows' scales 32 times the
// others', it takes 403 us of 1286.
constexpr int kAgainBM = 64, kAgainKP = 4;
template <int EP>
__global__ __launch_bounds__(kThreads) void gradients_again_kernel(GemmArgs a, int n_tiles, int share, EpilogueArgs e) {
  __shared__ int wanted;
  const int mt_count = (a.M + kAgainBM - 1) / kAgainBM, at_once = gridDim.x / share;
  const int tid = threadIdx.x;
  for (int mt = blockIdx.x / share; mt < mt_count; mt += at_once) {
    if (tid < 64) {
      const int m = min(kAgainBM * mt + tid, a.M - 1);
      const GradRow row = e.grad.rows[m];
      const int first = first_exponent(row, a.s_x[m], e.grad.tops, e.act, ep_glu(EP));
      const int last =
          last_exponent(first, e.grad.largest[m], row, a.s_x[m], e.grad.tops, e.act, ep_glu(EP), e.grad.terms);
      if (blockIdx.x % share == 0) e.grad.back[m] = 0.5f * exp2_of(-last);   // (the last token's by several, alike)
      const unsigned long long any = __ballot(first != last);
      if (tid == 0) wanted = any != 0;
    }
    __syncthreads();
    const bool go = wanted;
    __syncthreads();
    if (!go) continue;
    for (int nt = blockIdx.x % share; nt < n_tiles; nt += share) {
      product_tile<kAgainBM, kAgainKP, EP, true>(a, e, a.M, a.N, a.K, mt, nt);
      __builtin_amdgcn_s_waitcnt(waitcnt_vm_lgkm0(0));   // (its counted waits start from none in flight)
      __syncthreads();   // the next tile's copies reuse the LDS
    }
  }
}

template <int BM, int KP, int EP>
hipError_t launch_tiles(const GemmPlan& p, const GemmArgs& a, hipStream_t stream, EpilogueOf<EP> e) {
  constexpr int kBNO = Tiling<BM, KP>::kBN / (ep_glu(EP) ? 2 : 1);   // outputs per tile
  const int nt = (a.N + kBNO - 1) / kBNO;
  launch_product_kernel(mfma_gemm_kernel<BM, KP, EP>, dim3(p.grid), dim3(kThreads), 0, stream, a, nt, 0, e);
  return hipGetLastError();
}

template <int EP>
hipError_t launch_again(const GemmArgs& a, const EpilogueArgs& e, hipStream_t stream) {
  static_assert(kAgainBM == 64, "a wave looks at a tile's tokens");
  constexpr int kBNO = Tiling<kAgainBM, kAgainKP>::kBN / (ep_glu(EP) ? 2 : 1);
  const int nt = (a.N + kBNO - 1) / kBNO, mt = (a.M + kAgainBM - 1) / kAgainBM;
  const int share = mt >= kCUs ? 1 : nt < kCUs / mt ? nt : kCUs / mt;
  hipLaunchKernelGGL(gradients_again_kernel<EP>, dim3(mt >= kCUs ? kCUs : mt * share), dim3(kThreads), 0, stream, a,
                     nt, share, e);
  return hipGetLastError();
}

// plan.rw carries the tile height in units of 64 activation rows (1 or 2; 0: 32
// rows, the backward epilogues only), plan.ch the k-phases (2 or 4).
template <int EP>
hipError_t launch_ep(const GemmPlan& p, const GemmArgs& a, hipStream_t stream, const EpilogueOf<EP>& e) {
  if constexpr (ep_back(EP)) {
    if (p.rw == 0 && p.ch == 4) return launch_tiles<32, 4, EP>(p, a, stream, e);
  }
  if (p.rw == 1 && p.ch == 4) return launch_tiles<64, 4, EP>(p, a, stream, e);
  if (p.rw == 1 && p.ch == 2) return launch_tiles<64, 2, EP>(p, a, stream, e);
  if (p.rw == 2 && p.ch == 4) return launch_tiles<128, 4, EP>(p, a, stream, e);
  if (p.rw == 2 && p.ch == 2) return launch_tiles<128, 2, EP>(p, a, stream, e);
  return hipErrorInvalidValue;
}

}  // namespace

// Static LDS per workgroup: activation buffers (or epilogue tiles), the pair
// table, the tile's s_x and, with 128-row tiles, the phase counters.
int mfma_gemm_lds_bytes(int bm, int kp) {
  const int main_bytes = bm == 128 ? (kp == 4 ? Tiling<128, 4>::kLdsBytes : Tiling<128, 2>::kLdsBytes)
                         : kp == 4 ? Tiling<64, 4>::kLdsBytes
                                   : Tiling<64, 2>::kLdsBytes;
  return main_bytes + 1024 * 8 + bm * 4 + (bm == 128 ? 4 * kp : 0);
}

int mfma_gemm_threads() { return kThreads; }

int mfma_gemm_grid(int M, int N, int bm, int kp) {
  const int bn = kThreads / 64 / kp * kTileRows;
  const int mt = (M + bm - 1) / bm, nt = (N + bn - 1) / bn;
  const int per_xcd = (nt + 7) / 8;
  return 8 * per_xcd * mt;
}

hipError_t launch_mfma_gemm(const GemmPlan& p, const GemmArgs& a, hipStream_t stream) {
  return launch_ep<kEpNone>(p, a, stream, NoEpilogueArgs{});
}

hipError_t launch_mfma_gemm_epilogue(const GemmPlan& p, const GemmArgs& a, int ep, const EpilogueArgs& e,
                                     hipStream_t stream) {
  switch (ep) {
    case kEpFused: return launch_ep<kEpFused>(p, a, stream, e);
    case kEpGlu: return launch_ep<kEpGlu>(p, a, stream, e);
    case kEpFusedBack: return launch_ep<kEpFusedBack>(p, a, stream, e);
    case kEpGluBack: return launch_ep<kEpGluBack>(p, a, stream, e);
    default: return hipErrorInvalidValue;
  }
}

hipError_t launch_gradients_again(const GemmArgs& a, int ep, const EpilogueArgs& e, hipStream_t stream) {
  return ep_glu(ep) ? launch_again<kEpGluBack>(a, e, stream) : launch_again<kEpFusedBack>(a, e, stream);
}

}  // namespace sherry
