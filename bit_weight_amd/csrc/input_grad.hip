// Gradients of the products with an epilogue.  Three steps, the scratch
// memory between them:
//  1. grad_prepare_kernel reads what the size of the finite gradients follows
//     from (per token max|dy|, sum|q| and sum q^2, per matrix max|alpha|, the
//     largest positive bias) and lays the weight codes out for step 3;
//  2. the forward's prefill kernel recomputes the exact sums (1.25 bits per
//     weight: cheaper than saving M x N fp32 values in the forward) and its
//     epilogue writes z = dz alpha in scaled fp16 (sherry_grad.h) and partial
//     sums of dalpha, dbias; gradients_again_kernel then writes z again for
//     tokens whose scale came out too small, and every token's factor back;
//  3. input_grad_kernel forms dx = sum over rows n of z[m,n] T[n,k] on the
//     fp16 matrix cores, both matrices of the gated block in one sum;
// and grad_finish_kernel adds partial sums where a step left some.
// Matrix-core time bounds the sum at many tokens (bf16, K = 4096, N = 14336,
// gated, M=2048: 26 + 254 + 5 + 300 + 14 us, 1.9 POP/s int8 and 1.6 PFLOP/s fp16
// in steps 2 and 3), the five launches at few (M=77, K=1040, N=1300: 29 us).
//
// Step 3's weights.  The product contracts over weight rows, but a 5-bit
// code covers 4 columns of one row, so no operand of the matrix instruction
// can be decoded from a code alone.  Step 1 therefore writes T at 2 bits a
// weight in operand order: for a 64-row x 64-column half tile, lane (i, g)
// of a wave holds the weights of columns 4i .. 4i+3 and, for sub-step s = 0,
// 1, rows 32 s + 8 g .. + 7, 16 bytes in all.  Weight w is the sign and the
// top exponent bit of the fp16 number 2 w (0xC000, 0x4000 or 0), 8 such pairs
// in each half of a dword, so an operand register is one shift and one mask:
// no table, no LDS.  The factor 2 is taken back with the token's scale.
// Consecutive row tiles of a column half are consecutive in memory.
#include "sherry_device.h"
#include "sherry_grad.h"
#include "sherry_launch.h"
#include "sherry_types.h"

namespace sherry {
namespace {

typedef _Float16 h8 __attribute__((ext_vector_type(8)));
typedef unsigned int v4u __attribute__((ext_vector_type(4)));

template <int I>
using Const = std::integral_constant<int, I>;

constexpr int kPrepThreads = 256;
constexpr int kHalfBytes = 1024;   // a 64-row x 64-column half tile in operand order

// ------------------------------------------------------------------ step 1
// Blocks 0 to 2 read alpha, alpha2 and bias; the next M one token each; the
// rest four tiles each, a wave per tile.
struct PrepareArgs {
  const uint8_t* packed[2];
  const float* vec[3];    // alpha, alpha2, bias (nullptr: none)
  const void* dy;
  const int8_t* q;
  uint8_t* codes;         // [2 k tiles][parts x row tiles][kHalfBytes]
  GradRow* rows;
  float* tops;
  uint32_t* largest;
  int parts, dtype, M, N, K;
};

// |v|, or 0 where v is infinite or NaN.
__device__ __forceinline__ float finite_abs(float v) {
  const float t = fabsf(v);
  return t <= 3.402823466e38f ? t : 0.0f;
}

__device__ __forceinline__ float block_top(float v, float* red) {
  v = wave_max(v);
  __syncthreads();
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
  __syncthreads();
  float r = red[0];
  for (int i = 1; i < kPrepThreads / 64; ++i) r = fmaxf(r, red[i]);
  return r;
}

// The four weights of code c as 2-bit fields in a byte (two's complement:
// weight j in bits 2j, 2j + 1, i.e. nonzero and sign).
__device__ __forceinline__ uint32_t code_fields(uint32_t c) {
  const uint32_t w = code_word(c) & 0x03030303u;
  return (w | w >> 6 | w >> 12 | w >> 18) & 255u;
}

__global__ __launch_bounds__(kPrepThreads) void grad_prepare_kernel(PrepareArgs a) {
  constexpr int kPitch = 36;   // bytes per row of the staged tile
  __shared__ __attribute__((aligned(16))) uint8_t tile[kPrepThreads / 64][kTileRows * kPitch];
  __shared__ uint8_t fields[32];
  __shared__ float red[kPrepThreads / 64];
  __shared__ float2 sums[kPrepThreads / 64];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  // maxima: kAhead loads in flight per thread (a load a turn, waited for,
  // made block 0 the launch's last: 54 us at N = 14336)
  constexpr int kAhead = 16;
  if (blockIdx.x < 3) {
    const float* vec = a.vec[blockIdx.x];
    float t = 0.0f;
    for (int n0 = tid; vec && n0 < a.N; n0 += kAhead * kPrepThreads) {
      float v[kAhead];
#pragma unroll
      for (int i = 0; i < kAhead; ++i) v[i] = vec[min(n0 + i * kPrepThreads, a.N - 1)];
#pragma unroll
      for (int i = 0; i < kAhead; ++i) t = fmaxf(t, blockIdx.x == 2 && v[i] < 0.0f ? 0.0f : finite_abs(v[i]));
    }
    t = block_top(t, red);
    if (tid == 0) a.tops[blockIdx.x] = t;
    return;
  }
  const int block = blockIdx.x - 3;
  if (block < a.M) {
    const int m = block;
    float t = 0.0f;
    for (int n0 = 4 * tid; n0 < a.N; n0 += kAhead * kPrepThreads) {
      f4 v[kAhead / 4];
#pragma unroll
      for (int i = 0; i < kAhead / 4; ++i)
        v[i] = load4_as(a.dy, (size_t)m * a.N + min(n0 + 4 * i * kPrepThreads, a.N - 4), a.dtype);
#pragma unroll
      for (int i = 0; i < kAhead / 4; ++i)
        t = fmaxf(fmaxf(t, fmaxf(finite_abs(v[i][0]), finite_abs(v[i][1]))),
                  fmaxf(finite_abs(v[i][2]), finite_abs(v[i][3])));
    }
    int s = 0, squares = 0;
    const int4* q = reinterpret_cast<const int4*>(a.q + (size_t)m * a.K);
    for (int k = tid; k < a.K / 16; k += kPrepThreads) {
      const int4 v = q[k];
      const int w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int b = 0; b < 4; ++b) {
          const int x = (w[i] << (24 - 8 * b)) >> 24;
          s += abs(x);
          squares += x * x;
        }
    }
    t = block_top(t, red);
    // (a lane's sums stay below 2^19 and 2^26: K / kPrepThreads values)
    const float2 total = make_float2(wave_sum((float)s), wave_sum((float)squares));
    __syncthreads();
    if (lane == 0) sums[wave] = total;
    __syncthreads();
    if (tid == 0) {
      const float sum = (sums[0].x + sums[1].x) + (sums[2].x + sums[3].x);
      const float square = (sums[0].y + sums[1].y) + (sums[2].y + sums[3].y);
      a.rows[m] = GradRow{t, sum, fminf(sum, kSpread * sqrtf(0.75f * square)), 0.0f};
      a.largest[m] = 0u;
    }
    return;
  }
  const int KT = k_tiles(a.K), RT = row_tiles(a.N);
  const int id = (block - a.M) * (kPrepThreads / 64) + wave;
  const bool live = id < a.parts * RT * KT;
  const int r = live ? id / KT : 0, kt = live ? id - r * KT : 0;   // r: row tile over both matrices
  const int part = r >= RT ? 1 : 0, rt = r - part * RT;
  if (tid < 32) fields[tid] = (uint8_t)code_fields(tid);
  __syncthreads();
  {
    const uint8_t* src = a.packed[part] + tile_offset(rt, kt, KT);
    const uint4 lo = *reinterpret_cast<const uint4*>(src + 16 * lane);
    const uint32_t hi = *reinterpret_cast<const uint32_t*>(src + kTileHiOff + 4 * lane);
    const uint32_t w[4] = {lo.x, lo.y, lo.z, lo.w};
    const int i = lane & 15, g = lane >> 4;
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      const bool row_ok = rt * kTileRows + 16 * t + i < a.N;
      uint32_t f[2] = {0, 0};
#pragma unroll
      for (int jj = 0; jj < 8; ++jj) {
        const bool ok = row_ok && kt * kTileK + 4 * (8 * g + jj) < a.K;
        const uint32_t c = fields[group_code(w[t], (hi >> (8 * t)) & 255u, jj)];
        f[jj >> 2] |= (ok ? c : 0u) << (8 * (jj & 3));
      }
      uint32_t* dst = reinterpret_cast<uint32_t*>(&tile[wave][(16 * t + i) * kPitch + 8 * g]);
      dst[0] = f[0];
      dst[1] = f[1];
    }
  }
  __syncthreads();
  if (!live) return;
  const int i = lane & 15, g = lane >> 4;
  const size_t R = (size_t)a.parts * RT;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    uint32_t out[4];
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      uint32_t d0 = 0, d1 = 0;   // columns 0, 1 and 2, 3
#pragma unroll
      for (int p = 0; p < 4; ++p) {
        // rows 2p and 2p + 1 in the two halves; the field of column jl at
        // entry e = 4 jl + p: bits 14 - 2e of its half
        const uint8_t* src = &tile[wave][(32 * s + 8 * g + 2 * p) * kPitch + 16 * h + i];
        const uint32_t f = (uint32_t)src[0] | (uint32_t)src[kPitch] << 16;
        d0 |= (f & 0x00030003u) << (14 - 2 * p) | ((f >> 2) & 0x00030003u) << (6 - 2 * p);
        d1 |= ((f >> 4) & 0x00030003u) << (14 - 2 * p) | ((f >> 6) & 0x00030003u) << (6 - 2 * p);
      }
      out[2 * s] = d0;
      out[2 * s + 1] = d1;
    }
    *reinterpret_cast<uint4*>(a.codes + ((2 * (size_t)kt + h) * R + r) * kHalfBytes + 16 * lane) =
        make_uint4(out[0], out[1], out[2], out[3]);
  }
}

// ------------------------------------------------------------------ step 3
// Workgroup: 8 waves, 2 x 4; a wave forms 16 MT tokens x 64 columns, the
// workgroup BM = 32 MT tokens x 256 columns, over a share of the row tiles
// (64 contraction indices a step, 128 bytes of z per token).
//  * z: copied once per workgroup straight into LDS (buffer loads with LDS
//    return), four buffers, up to three steps ahead; rows of 128 bytes whose
//    16-byte chunks are XOR-swizzled so 16 rows' reads of one chunk hit 16
//    bank groups.  A buffer is an array of its own, picked by a constant: the
//    compiler then sees that a step's reads cannot touch what the copies in
//    flight write (from one array it waits for every copy before the first
//    read of each step).
//  * T: each wave loads its half tile's 16 bytes a lane three steps ahead and
//    makes its operands with shifts and masks between the MFMAs.
//  * A step is two sub-steps.  Between them a wave waits for its copies of the
//    next step (counted vmcnt, the newer loads stay in flight) and joins the
//    barrier; behind it are the copies into the buffer every wave has left by
//    then, and the next step's first fragments and operands, under the second
//    sub-step's MFMAs.  A step so starts with MFMAs (with the barrier in front
//    of the step and three buffers: M=2048, K=4096, 448 row tiles 330 us; so
//    317, 1.52 PFLOP/s, what the vendor's fp16 product of 8192^3 reaches).
// Workgroups of one XCD take neighbouring column tiles of the same tokens,
// so a z tile is read from HBM once and then from that XCD's L2.
constexpr int kGradThreads = 512;
constexpr int kGradBN = 256;
constexpr int kStepK = 64;
constexpr int kMaxSplits = 64;     // of the contraction

struct InputGradArgs {
  const uint8_t* codes;
  const _Float16* z;
  const float* back;
  void* dx;          // [M,K] of type dtype (one split), or
  float* part;       // [splits][M][K]
  int dtype, terms;
  int M, K, R;       // R: row tiles of all matrices
  int splits, r_per_split;
};

__device__ __forceinline__ int z_off(int r, int c) { return (r * 8 + (c ^ ((r >> 1) & 7))) * 16; }

// s_waitcnt operand: vmcnt(vm) only.
constexpr int wait_vm(int vm) { return (vm & 15) | ((vm >> 4) << 14) | 0x0F70; }

__device__ __forceinline__ void z_to_lds(__amdgpu_buffer_rsrc_t r, uint8_t* dst, int voffset, int soffset) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (__attribute__((address_space(3))) void*)dst, 16, voffset, soffset,
                                           0, 0);
}

// 2^31 bytes from base on.  The range check sees the lanes' offsets, here below
// 2^31, and not the scalar one added to them: 256 tokens' z, whose last bytes
// lie 2^31 behind the first, is within it either way.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t all_of(const void* base) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), 0, (int)0x80000000u, 0x00020000);
}

template <int MT>
__global__ __launch_bounds__(kGradThreads) void input_grad_kernel(InputGradArgs a) {
  constexpr int BM = 32 * MT;
  constexpr int kStage = BM * 128;                       // bytes of z per step
  static_assert(MT % 2 == 0, "fragments are taken in pairs");
  constexpr int kCopies = MT / 2;                        // 8-row copies per wave and step
  constexpr int kDecode = MT >= 8 ? 1 : 8 / MT;          // column blocks decoded per pair of fragments
  __shared__ __attribute__((aligned(1024))) uint8_t z0[kStage], z1[kStage], z2[kStage], z3[kStage];
  __shared__ float back[BM];   // 2^-e / 2 of each token

  const int NT = (a.K + kGradBN - 1) / kGradBN, MTiles = (a.M + BM - 1) / BM;
  const int total = NT * MTiles * a.splits, per = (total + 7) / 8;
  const int id = (blockIdx.x & 7) * per + (blockIdx.x >> 3);
  if ((int)(blockIdx.x >> 3) >= per || id >= total) return;
  // (quotients come from the vector unit; made scalar, the buffer descriptors
  // that follow from them stay scalar)
  const int group = __builtin_amdgcn_readfirstlane(id / NT), nt = id - group * NT;
  const int mt = __builtin_amdgcn_readfirstlane(group / a.splits), split = group - mt * a.splits;
  const int m0 = mt * BM;
  const int r0 = split * a.r_per_split, r1 = min(a.R, r0 + a.r_per_split);
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave >> 2, wn = wave & 3;
  const int l16 = lane & 15, g = lane >> 4;

  for (int t = tid; t < BM; t += kGradThreads) {
    const int m = min(m0 + t, a.M - 1);
    back[t] = a.back[m];
  }

  // this wave's 64 columns (past the last k tile: the last half again, not stored)
  const int halves = 2 * k_tiles(a.K);
  const int col0 = nt * kGradBN + 64 * wn;
  const int half = min(col0 / 64, halves - 1);
  const __amdgpu_buffer_rsrc_t rw = all_of(a.codes + (size_t)half * a.R * kHalfBytes);
  const size_t zrow = (size_t)a.terms * a.R * kStepK;    // fp16 elements per token
  const __amdgpu_buffer_rsrc_t rz = all_of(a.z + (size_t)m0 * zrow);
  // copy jj of this wave: 8 rows of 128 bytes, lane L the chunk that belongs
  // at LDS position 16 L; tokens past M re-read the last one (not stored).
  // Lane offsets stay below 2^31: 255 rows of at most 2^23 bytes.
  int z_v[kCopies], z_row[kCopies];
#pragma unroll
  for (int jj = 0; jj < kCopies; ++jj) {
    z_row[jj] = 8 * (wave * kCopies + jj);
    const int row = z_row[jj] + (lane >> 3);
    const int c = (lane & 7) ^ ((row >> 1) & 7);
    z_v[jj] = min(row, a.M - 1 - m0) * (int)(2 * zrow) + 16 * c;
  }
  // steps: row tile r0 + st / terms, term st % terms
  const int steps = (r1 - r0) * a.terms, shift = a.terms - 1;
  auto load_w = [&](int st, v4u& w) {
    w = __builtin_amdgcn_raw_buffer_load_b128(rw, 16 * lane, (r0 + (min(st, steps - 1) >> shift)) * kHalfBytes, 0);
  };
  auto copy_z = [&](int st, uint8_t* buf) {
    const int s = min(st, steps - 1);
    const int col = (((s & shift) * a.R) + r0 + (s >> shift)) * 128;
#pragma unroll
    for (int jj = 0; jj < kCopies; ++jj) z_to_lds(rz, buf + z_row[jj] * 128, z_v[jj], col);
    __builtin_amdgcn_sched_barrier(0);
  };

  f4 acc[MT][4];
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[i][j] = f4{0.0f, 0.0f, 0.0f, 0.0f};

  auto frag = [&](const uint8_t* buf, int u) __attribute__((always_inline)) {   // u = MT s + row block
    return *reinterpret_cast<const h8*>(buf + z_off(16 * (MT * wm + u % MT) + l16, 4 * (u / MT) + g));
  };
  auto decode = [&](const v4u& w, int s, int j) __attribute__((always_inline)) {
    const uint32_t d = w[2 * s + (j >> 1)];
    v4u o;
#pragma unroll
    for (int p = 0; p < 4; ++p) o[p] = (d << (2 * (4 * (j & 1) + p))) & 0xC000C000u;
    return __builtin_bit_cast(h8, o);
  };
  h8 f0, f1, even[4], odd[4];   // fragments; operands of sub-steps 0 and 1
  // sub-step s on `now`: per pair of fragments its 8 MFMAs, the request of the
  // fragments two ahead and a share of decoding the sub-step after it
  auto sub_step = [&](auto sc, const uint8_t* buf, const uint8_t* next, const h8 (&now)[4], h8 (&then)[4],
                  const v4u& w) __attribute__((always_inline)) {
    constexpr int s = decltype(sc)::value;
#pragma unroll
    for (int i = 0; i < MT; i += 2) {
      const int u = MT * s + i;
      const h8 p0 = u + 2 < 2 * MT ? frag(buf, u + 2) : frag(next, u + 2 - 2 * MT);
      const h8 p1 = u + 3 < 2 * MT ? frag(buf, u + 3) : frag(next, u + 3 - 2 * MT);
#pragma unroll
      for (int d = 0; d < kDecode; ++d) {
        const int j = (i / 2) * kDecode + d;
        if (j < 4) then[j] = decode(w, 1 - s, j);
      }
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_f16(f0, now[j], acc[i][j], 0, 0, 0);
#pragma unroll
      for (int j = 0; j < 4; ++j)
        acc[i + 1][j] = __builtin_amdgcn_mfma_f32_16x16x32_f16(f1, now[j], acc[i + 1][j], 0, 0, 0);
      __builtin_amdgcn_sched_barrier(0);
      f0 = p0;
      f1 = p1;
    }
  };
  // Step st on buffer buf with weights w; next / wn are the next step's, far /
  // wf those that step st + 3 goes to.
  auto step = [&](int st, const uint8_t* buf, const uint8_t* next, uint8_t* far, const v4u& w, const v4u& wn,
                  v4u& wf) __attribute__((always_inline)) {
    sub_step(Const<0>{}, buf, next, even, odd, w);
    // newer than the next step's copies: its weights, the copies after them
    // and theirs
    __builtin_amdgcn_s_waitcnt(wait_vm(kCopies + 2));
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
    __builtin_amdgcn_sched_barrier(0);
    copy_z(st + 3, far);
    load_w(st + 3, wf);
    __builtin_amdgcn_sched_barrier(0);
    sub_step(Const<1>{}, buf, next, odd, even, wn);
  };

  v4u w0, w1, w2, w3;
  copy_z(0, z0);
  load_w(0, w0);
  __builtin_amdgcn_sched_barrier(0);
  copy_z(1, z1);
  load_w(1, w1);
  __builtin_amdgcn_sched_barrier(0);
  copy_z(2, z2);
  load_w(2, w2);
  __builtin_amdgcn_sched_barrier(0);
  __builtin_amdgcn_s_waitcnt(wait_vm(2 * kCopies + 3));
  __builtin_amdgcn_s_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
  __builtin_amdgcn_sched_barrier(0);
  f0 = frag(z0, 0);
  f1 = frag(z0, 1);
#pragma unroll
  for (int j = 0; j < 4; ++j) even[j] = decode(w0, 0, j);
  int st = 0;
  for (; st + 4 <= steps; st += 4) {
    step(st, z0, z1, z3, w0, w1, w3);
    step(st + 1, z1, z2, z0, w1, w2, w0);
    step(st + 2, z2, z3, z1, w2, w3, w1);
    step(st + 3, z3, z0, z2, w3, w0, w2);
  }
  if (st < steps) step(st, z0, z1, z3, w0, w1, w3);
  if (st + 1 < steps) step(st + 1, z1, z2, z0, w1, w2, w0);
  if (st + 2 < steps) step(st + 2, z2, z3, z1, w2, w3, w1);
  // the clamped copies past the end land before the workgroup's LDS is freed
  __builtin_amdgcn_s_waitcnt(wait_vm(0));
  __syncthreads();

  // lane (l16, g) of accumulator (i, j): rows 4g .. 4g+3 of row block i,
  // column 4 l16 + j of this wave's 64
  const int col = col0 + 4 * l16;
  auto put = [&](auto* out) {
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int row = 16 * (MT * wm + i) + 4 * g + r, m = m0 + row;
        if (m < a.M && col < a.K)
          store4(out + (size_t)m * a.K + col, f4{acc[i][0][r], acc[i][1][r], acc[i][2][r], acc[i][3][r]} * back[row]);
      }
  };
  if (a.part) put(a.part + (size_t)split * a.M * a.K);
  else if (a.dtype == SHERRY_F32) put(static_cast<float*>(a.dx));
  else if (a.dtype == SHERRY_F16) put(static_cast<_Float16*>(a.dx));
  else put(static_cast<__bf16*>(a.dx));
}

// Partial sums joined in order: dx over the splits, dalpha and dbias over
// the token tiles.
struct FinishArgs {
  const float* dx_part;    // nullptr: dx is already written
  void* dx;
  const float* cols[2];    // [tiles][N], nullptr: already written (or not wanted)
  float* out[2];
  int dtype, splits, tiles, M, N, K, dx_blocks;
};

__global__ __launch_bounds__(256) void grad_finish_kernel(FinishArgs a) {
  __shared__ float red[4][64];
  if ((int)blockIdx.x < a.dx_blocks) {
    const size_t n4 = (size_t)a.M * a.K / 4;
    for (size_t i = (size_t)blockIdx.x * 256 + threadIdx.x; i < n4; i += (size_t)a.dx_blocks * 256) {
      // eight splits' loads in flight at a time, added in order
      f4 t = load4(a.dx_part + 4 * i);
      for (int s0 = 1; s0 < a.splits; s0 += 8) {
        f4 v[8];
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (s0 + j < a.splits) v[j] = load4(a.dx_part + (size_t)(s0 + j) * 4 * n4 + 4 * i);
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (s0 + j < a.splits) t += v[j];
      }
      store4_as(a.dx, 4 * i, a.dtype, t);
    }
    return;
  }
  const int col_blocks = (a.N + 63) / 64, c = blockIdx.x - a.dx_blocks;
  const int which = c >= col_blocks;
  const float* part = a.cols[which];
  if (!part) return;
  const int lane = threadIdx.x & 63, share = threadIdx.x >> 6;
  const int n = (c - which * col_blocks) * 64 + lane;
  float t = 0.0f;
  if (n < a.N) {
#pragma unroll 4
    for (int r = share; r < a.tiles; r += 4) t += part[(size_t)r * a.N + n];
  }
  red[share][lane] = t;
  __syncthreads();
  if (share == 0 && n < a.N) a.out[which][n] = (red[0][lane] + red[1][lane]) + (red[2][lane] + red[3][lane]);
}

size_t up256(size_t n) { return (n + 255) / 256 * 256; }

}  // namespace

// Tokens per workgroup tile (32 MT) and contraction splits: the pair with the
// least estimated time.  A workgroup takes a fixed time and a time per step
// (us, measured with one workgroup per CU, 56 and 448 steps: MT = 2 36 and
// 248, MT = 4 52 and 366, MT = 8 90 and 660); larger tiles read less z and T
// per multiply-add, smaller ones waste less of few tokens and fill the CUs
// with fewer splits, whose partial results are written and read again at
// about 6 TB/s.  (Against 256 tokens from 385 on, 128 from 65 on and as many
// splits as fill the CUs, whole backward pass, bf16: M=512, N=K=4096 55.4 -> 46.2
// us; M=128 gated there 41.9 -> 39.5; M=512 gated, N=11008 160.9 -> 155.8; fp16
// M=1500, N=K=2048 63.6 -> 59.6.)
void plan_tiles(int M, int K, GradPlan& p) {
  constexpr struct { int mt; double fixed, step; } kTiles[] = {{2, 5.5, 0.54}, {4, 7.0, 0.80}, {8, 9.0, 1.45}};
  double best = 0.0;
  for (const auto& t : kTiles) {
    const double tiles = (double)((M + 32 * t.mt - 1) / (32 * t.mt)) * ((K + kGradBN - 1) / kGradBN);
    for (int s = 1; s <= kMaxSplits && s <= p.R; ++s) {
      const int r = (p.R + s - 1) / s;
      if ((p.R + r - 1) / r != s) continue;   // no empty split
      double time = ceil(tiles * s / kCUs) * (t.fixed + (double)r * p.terms * t.step);
      if (s > 1) time += 2.0 + (double)s * M * K * 8.0 / 6.0e6;
      if (best == 0.0 || time < best) {
        best = time;
        p.mt = t.mt;
        p.splits = s;
        p.r_per_split = r;
      }
    }
  }
}

GradPlan plan_grad(const GemmPlan& product, int M, int N, int K, int parts, int dtype) {
  GradPlan p{};
  p.terms = dtype == SHERRY_BF16 ? 1 : 2;
  p.R = parts * row_tiles(N);
  plan_tiles(M, K, p);
  const int bm = product.rw ? 64 * product.rw : 32;   // tokens per tile of the recomputing product
  p.token_tiles = (M + bm - 1) / bm;
  size_t at = 0;
  auto take = [&](size_t bytes) {
    const size_t here = at;
    at += up256(bytes);
    return here;
  };
  p.tops = take(3 * sizeof(float));
  p.rows = take((size_t)M * sizeof(GradRow));
  p.largest = take((size_t)M * sizeof(uint32_t));
  p.back = take((size_t)M * sizeof(float));
  p.codes = take(2 * (size_t)k_tiles(K) * p.R * kHalfBytes);
  p.z = take((size_t)M * p.terms * p.R * kStepK * sizeof(uint16_t));
  p.cols = take(p.token_tiles > 1 ? 2 * (size_t)p.token_tiles * N * sizeof(float) : 0);
  p.dx_part = take(p.splits > 1 ? (size_t)p.splits * M * K * sizeof(float) : 0);
  p.bytes = at;
  return p;
}

hipError_t launch_backward(const GemmPlan& product, const GradPlan& p, const GemmArgs& a, int ep, EpilogueArgs e,
                           void* dx, float* d0, float* d1, void* scratch, hipStream_t stream, bool* partial) {
  *partial = false;
  const bool glu = ep_glu(ep);
  const int parts = glu ? 2 : 1;
  char* base = static_cast<char*>(scratch);
  PrepareArgs pa{};
  pa.packed[0] = a.packed;
  pa.packed[1] = e.packed2;
  pa.vec[0] = a.alpha;
  pa.vec[1] = e.alpha2;
  pa.vec[2] = e.bias;
  pa.dy = e.grad.dy;
  pa.q = a.x;
  pa.codes = reinterpret_cast<uint8_t*>(base + p.codes);
  pa.rows = reinterpret_cast<GradRow*>(base + p.rows);
  pa.tops = reinterpret_cast<float*>(base + p.tops);
  pa.largest = reinterpret_cast<uint32_t*>(base + p.largest);
  pa.parts = parts;
  pa.dtype = e.dtype;
  pa.M = a.M;
  pa.N = a.N;
  pa.K = a.K;
  const size_t tiles = (size_t)p.R * k_tiles(a.K);
  hipLaunchKernelGGL(grad_prepare_kernel, dim3((unsigned)(3 + a.M + (tiles + 3) / 4)), dim3(kPrepThreads), 0, stream, pa);
  hipError_t err = hipGetLastError();
  if (err != hipSuccess) return err;
  *partial = true;

  const bool direct = p.token_tiles == 1;   // one token tile: its sums are the results
  float* cols = reinterpret_cast<float*>(base + p.cols);
  e.grad.rows = pa.rows;
  e.grad.tops = pa.tops;
  e.grad.largest = pa.largest;
  e.grad.back = reinterpret_cast<float*>(base + p.back);
  e.grad.z = reinterpret_cast<uint16_t*>(base + p.z);
  e.grad.terms = p.terms;
  e.grad.part0 = !d0 ? nullptr : direct ? d0 : cols;
  e.grad.part1 = !d1 ? nullptr : direct ? d1 : cols + (size_t)p.token_tiles * a.N;
  err = launch_mfma_gemm_epilogue(product, a, ep, e, stream);
  if (err != hipSuccess) return err;
  err = launch_gradients_again(a, ep, e, stream);
  if (err != hipSuccess) return err;

  InputGradArgs g{};
  g.codes = pa.codes;
  g.z = reinterpret_cast<const _Float16*>(base + p.z);
  g.back = e.grad.back;
  g.dx = dx;
  g.part = p.splits > 1 ? reinterpret_cast<float*>(base + p.dx_part) : nullptr;
  g.dtype = e.dtype;
  g.terms = p.terms;
  g.M = a.M;
  g.K = a.K;
  g.R = p.R;
  g.splits = p.splits;
  g.r_per_split = p.r_per_split;
  const int bm = 32 * p.mt;
  const int total = ((a.K + kGradBN - 1) / kGradBN) * ((a.M + bm - 1) / bm) * p.splits;
  const dim3 grid(8 * ((total + 7) / 8)), block(kGradThreads);
  switch (p.mt) {
    case 2: hipLaunchKernelGGL(input_grad_kernel<2>, grid, block, 0, stream, g); break;
    case 4: hipLaunchKernelGGL(input_grad_kernel<4>, grid, block, 0, stream, g); break;
    default: hipLaunchKernelGGL(input_grad_kernel<8>, grid, block, 0, stream, g); break;
  }
  err = hipGetLastError();
  if (err != hipSuccess) return err;

  const bool join_cols = !direct && (d0 || d1);
  if (!g.part && !join_cols) return hipSuccess;
  FinishArgs f{};
  f.dx_part = g.part;
  f.dx = dx;
  f.cols[0] = direct ? nullptr : e.grad.part0;
  f.cols[1] = direct ? nullptr : e.grad.part1;
  f.out[0] = d0;
  f.out[1] = d1;
  f.dtype = e.dtype;
  f.splits = p.splits;
  f.tiles = p.token_tiles;
  f.M = a.M;
  f.N = a.N;
  f.K = a.K;
  const size_t dx_blocks = ((size_t)a.M * a.K / 4 + 255) / 256;
  f.dx_blocks = g.part ? (int)(dx_blocks < 4096 ? dx_blocks : 4096) : 0;
  const int col_blocks = join_cols ? 2 * ((a.N + 63) / 64) : 0;
  hipLaunchKernelGGL(grad_finish_kernel, dim3(f.dx_blocks + col_blocks), dim3(256), 0, stream, f);
  return hipGetLastError();
}

}  // namespace sherry
