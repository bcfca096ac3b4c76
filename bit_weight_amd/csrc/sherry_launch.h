// Internal launch interface between the C ABI (sherry_abi.hip) and the
// kernel translation units.  Shapes are validated by the caller.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>
#include <type_traits>

namespace sherry {

// Launch plan of the product for one shape (host-side, pure).
struct GemmPlan {
  int path;          // 0 = lookup-table GEMV, 1 = decode + int8 MFMA GEMM,
                     // 2 = decode + int8 MFMA GEMV (M <= 64)
  int grid;          // workgroups
  int block;         // threads per workgroup
  int splits;        // K-splits per row group (GEMV)
  int kt_per_split;  // format k-tiles per K-split (GEMV)
  int rw;            // LUT GEMV: row tiles per workgroup; matrix-core GEMV: waves per
                     // row tile; prefill GEMM: tile height in units of 64 activation rows
  int ch;            // LUT GEMV: k-tiles per LDS table stage; prefill GEMM: k-phases (2 or 4)
  int groups;        // output row groups (GEMV)
  int lds_bytes;     // dynamic LDS per workgroup
  size_t ws_bytes;   // workspace bytes required
  int chunk;         // tokens per launch (0 = all M in one launch)
};

constexpr int kLutMaxM = 16;          // M <= 16 takes a GEMV path
constexpr int kGemvMaxM = 64;         // 16 < M <= 64: the matrix-core GEMV, unless path 1 is forced
constexpr int kChunkMaxM = 128;       // 64 < M <= 128: the prefill GEMM, or the GEMV in
constexpr int kChunkMaxGrid = 64;     //   launches of 64 tokens where the prefill grid is at
                                      //   most 64 workgroups (chunk_max_m)
constexpr int kGemvWaves = 4;         // waves per GEMV workgroup
constexpr int kCUs = 256;             // MI355X compute units: one round of one workgroup each
constexpr int kDefaultSmallMPath = 2;  // M <= 16: 0 = lookup tables, 2 = matrix-core GEMV
constexpr int kGluMaxSplits = 255;     // gated product: arrivals a split-K cell counts
constexpr int kFuseMaxM = 4;           // fused quantization: at most 4 tokens,
constexpr int kFuseMaxMK = 16384;      //   M*K elements read per workgroup for the scales,
constexpr int kFuseMaxSpan = 32;       //   and k-tiles per K-split held in LDS as int8

// Tuning override of the GEMV plan (path -1 / others 0 = built-in choice),
// see sherry.h.
void set_plan_override(int path, int rw, int ch, int splits);

GemmPlan plan_gemm(int M, int N, int K);

// Backward: what the size of a token's gradients follows from.
struct GradRow {
  float dy;        // max |dy|
  float sum;       // sum |q|: no product of the token and a weight row is larger
  float likely;    // what none of them passes unless the row takes the token's signs
  float unused;
};

// Backward: what the recomputing product writes and scales by.
struct GradArgs {
  const void* dy;          // [M,N] of type dtype
  const GradRow* rows;     // per token
  const float* tops;       // max |alpha|, max |alpha2|, max(bias, 0)
  uint16_t* z;             // fp16 [M][terms][parts][64 row tiles]: the scaled gradients
  uint32_t* largest;       // per token: bits of the largest |dz alpha| (0 before the product)
  float* back;             // per token: what takes its sums of 2 T z back (written by the second pass)
  int terms;               // fp16 terms per gradient: 1, or 2 (high and low parts)
  float* part0;            // [token tiles][N] partial sums of dalpha
  float* part1;            // the same of dalpha2 or dbias
};

struct GemmArgs {
  const int8_t* x;     // int8 activations [M,K], or
  const float* xf;     // fp32 activations quantized in the kernel (fused form; x unused)
  const float* s_x;
  const uint8_t* packed;
  const float* alpha;
  float* y;            // fp32 output, or
  int32_t* acc;        // int32 output (exactly one of y / acc is non-null)
  int M, N, K;
  int32_t* partials;   // workspace: zero-filled 64-bit accumulators [M,N] for K-splits
};

// What a product's epilogue does with the exact sums.
enum Epilogue {
  kEpNone = 0,       // y = (acc s_x) alpha, or the int32 sums
  kEpFused = 1,      // out = act((acc s_x) alpha + bias) + residual
  kEpGlu = 2,        // out = act((acc s_x) alpha) * ((acc2 s_x) alpha2), two weight matrices
  kEpFusedBack = 3,  // the gradients of kEpFused's pre-activation, for the input-gradient product
  kEpGluBack = 4     // those of kEpGlu's two
};
constexpr bool ep_glu(int ep) { return ep == kEpGlu || ep == kEpGluBack; }
constexpr bool ep_back(int ep) { return ep == kEpFusedBack || ep == kEpGluBack; }

// Arguments of the epilogues other than kEpNone (whose kernels take an empty struct).
struct EpilogueArgs {
  const uint8_t* packed2;   // GLU: the up matrix; packed / alpha are the gate's
  const float* alpha2;
  const float* bias;        // fused: nullptr = none
  const void* residual;     // fused: nullptr = none
  void* out;                // forward: [M,N] of type dtype
  int act, dtype;           // SHERRY_ACT_*, SHERRY_F32 / F16 / BF16
  GradArgs grad;            // backward
};
struct NoEpilogueArgs {};
template <int EP>
using EpilogueOf = std::conditional_t<EP == kEpNone, NoEpilogueArgs, EpilogueArgs>;

// The product kernels take their arguments as pointers and scalars, not as
// a GemmArgs struct, with the ones their first instructions need in front:
// packed, x, xf, M, N, K, two plan integers (the GEMVs: splits and k-tiles
// per split; the prefill GEMM: n tiles and 0), then s_x, alpha, y, acc,
// partials, and last the epilogue's (the matrix-core kernels).  The build
// has the leading ones preloaded into SGPRs at dispatch (gfx950
// kernel-argument preload), which removes a memory round trip from the start
// of every launch; a struct argument cannot be preloaded.
template <typename Kernel, typename... E>
inline void launch_product_kernel(Kernel kernel, dim3 grid, dim3 block, size_t lds_bytes,
                                  hipStream_t stream, const GemmArgs& a, int plan0, int plan1, E... e) {
  hipLaunchKernelGGL(kernel, grid, block, lds_bytes, stream, a.packed, a.x, a.xf, a.M, a.N, a.K, plan0,
                     plan1, a.s_x, a.alpha, a.y, a.acc, a.partials, e...);
}

// The GemmArgs a product kernel rebuilds from its arguments.
__device__ __forceinline__ GemmArgs product_args(const uint8_t* packed, const int8_t* x, const float* xf,
                                                 int M, int N, int K, const float* s_x, const float* alpha,
                                                 float* y, int32_t* acc, int32_t* partials) {
  GemmArgs a{};
  a.packed = packed;
  a.x = x;
  a.xf = xf;
  a.M = M;
  a.N = N;
  a.K = K;
  a.s_x = s_x;
  a.alpha = alpha;
  a.y = y;
  a.acc = acc;
  a.partials = partials;
  return a;
}

hipError_t launch_quantize_pack(const float* W, int N, int K, uint8_t* packed, float* alpha,
                                hipStream_t stream);
hipError_t launch_quantize_pack2(const float* W, int N, int K, uint8_t* packed, float* alpha,
                                 hipStream_t stream);
hipError_t launch_quantize_act(const float* x, int M, int K, int8_t* q, float* s_x,
                               hipStream_t stream);
hipError_t launch_lut_gemv(const GemmPlan& plan, const GemmArgs& args, hipStream_t stream);
hipError_t launch_mfma_gemv(const GemmPlan& plan, const GemmArgs& args, hipStream_t stream);
bool mfma_gemv_fusable(const GemmPlan& plan, int M, int K);
bool lut_gemv_fusable(const GemmPlan& plan, int M, int K);
// The same GEMV on the 2-bit baseline format (packed = kTile2Bytes tiles).
hipError_t launch_mfma_gemv2(const GemmPlan& plan, const GemmArgs& args, hipStream_t stream);
// The prefill GEMM's grid and LDS for tiles of bm (64 or 128) activation rows.
int mfma_gemm_grid(int M, int N, int bm, int kp);
int mfma_gemm_lds_bytes(int bm, int kp);
int mfma_gemm_threads();
hipError_t launch_mfma_gemm(const GemmPlan& plan, const GemmArgs& args, hipStream_t stream);
// The product (x int8) on the plan's path, in launches of plan.chunk tokens
// when the plan asks for it.  On a failed launch, *partial (if given) tells
// whether earlier launches of the same call were already enqueued.
hipError_t launch_product(const GemmPlan& plan, const GemmArgs& args, hipStream_t stream,
                          bool* partial = nullptr);
// The same kernels with another epilogue (paths 1 and 2; ep != kEpNone).
hipError_t launch_mfma_gemv_epilogue(const GemmPlan& plan, const GemmArgs& args, int ep,
                                     const EpilogueArgs& e, hipStream_t stream);
hipError_t launch_mfma_gemm_epilogue(const GemmPlan& plan, const GemmArgs& args, int ep,
                                     const EpilogueArgs& e, hipStream_t stream);

// The backward product once more for the tokens whose gradients do not fit
// their scale (writes z, and `back` of every token; `largest` is complete).
hipError_t launch_gradients_again(const GemmArgs& args, int ep, const EpilogueArgs& e, hipStream_t stream);

// Plan of a backward pass: the input-gradient product's tiles and splits and
// where each array lies in the scratch memory (input_grad.hip).
struct GradPlan {
  int terms;          // fp16 terms per gradient
  int R;              // row tiles of all matrices
  int mt;             // tokens per workgroup tile / 32
  int splits, r_per_split;
  int token_tiles;    // of the recomputing product: rows of partial column sums
  size_t tops, rows, largest, back, codes, z, cols, dx_part, bytes;
};
GradPlan plan_grad(const GemmPlan& product, int M, int N, int K, int parts, int dtype);
// `product` is the recomputing product's plan (path 1), ep its epilogue; d0 =
// dalpha, d1 = dalpha2 or dbias, either may be nullptr.
hipError_t launch_backward(const GemmPlan& product, const GradPlan& plan, const GemmArgs& args, int ep,
                           EpilogueArgs e, void* dx, float* d0, float* d1, void* scratch, hipStream_t stream,
                           bool* partial);

// Layer norm (norm.hip): y in x's type, or q and s (int8 tokens).
hipError_t launch_layernorm(const void* x, const float* w, const float* b, float eps, void* y, int8_t* q,
                            float* s, float* mean, float* rstd, int dtype, int M, int K, hipStream_t stream);
int layernorm_backward_rows(int M, int K);   // rows of 2 K partial sums the backward needs
hipError_t launch_layernorm_backward(const void* dy, const void* x, const float* mean, const float* rstd,
                                     const float* w, void* dx, float* dw, float* db, int dtype, int M, int K,
                                     float* part, hipStream_t stream, bool* partial);

// Norm and rotation of each head (head_norm.hip).  Forward: q, k are written;
// backward: q, k hold dz and dx is written (its first (Hq + Hk) D columns).
struct HeadNormArgs {
  const void* x;            // [T, x_stride]: Hq heads of queries, then Hk of keys
  int64_t x_stride, dx_stride;
  const float *wq, *wk;     // nullptr: ones
  float eps;
  const double* freqs;      // [R / 2]
  const int32_t* positions;
  int T, Hq, Hk, D, R;
  bool interleaved, norm;
  int dtype;
  void *q, *k, *dx;
  float* part;              // backward: rows of 2 D partial weight gradients
};
hipError_t launch_head_norm(const HeadNormArgs& g, hipStream_t stream);
int head_norm_backward_rows(int T, int heads, int D);
hipError_t launch_head_norm_backward(const HeadNormArgs& g, float* dwq, float* dwk, hipStream_t stream,
                                     bool* partial);

// The 8-bit cache (sherry_cache.h) and what a call brings to it.
struct CacheArgs {
  uint8_t *k, *v;
  float *k_scale, *v_scale;
  int pages, block_shift;   // a page is 2^block_shift blocks of 16 tokens
  int H, D;
  const int32_t* table;     // [S, table_width]
  int table_width;
  const int32_t *starts, *lens;
  int S, T;
  int dtype;                // of rows
  const void *x_k, *x_v;    // cache_write's rows
  int64_t k_stride, v_stride;
};
hipError_t launch_cache_write(const CacheArgs& c, hipStream_t stream);
hipError_t launch_cache_read(const CacheArgs& c, void* k, void* v, hipStream_t stream);

// Attention over it (cache_attention.hip).
struct AttentionArgs {
  CacheArgs c;
  const void* q;
  int64_t q_stride;
  int Hq;
  float scale;
  int window, sinks;        // window 0: none
  void* y;                  // [T, Hq, D] of type c.dtype
  float* lse;               // [T, Hq], or nullptr
  float* scratch;
  int* counters;            // zero, and left zero
};
size_t cache_attention_workspace_bytes();
size_t cache_attention_scratch_bytes(int T, int S, int Hq, int H, int D);
size_t attention_tiles_scratch_bytes(int S, int D);      // cache_attention_tiles.hip: many queries a sequence
hipError_t launch_attention_tiles(const AttentionArgs& a, hipStream_t stream, bool* partial);
hipError_t launch_cache_attention(const AttentionArgs& a, hipStream_t stream, bool* partial);

}  // namespace sherry
