/*
 * sherry.h -- C ABI of the Sherry 3:4-sparse ternary matmul library for
 * AMD MI355X (gfx950).
 *
 * Method: the page "Sherry框架：三元量化与3:4稀疏优化LLM推理"
 * (pnsm.cn/news/1195499.html).  Weights are ternary {-1,0,+1} with exactly
 * three nonzeros in every block of four consecutive weights of a row
 * (§1.1).  A block is stored in 5 bits: a 4-bit index into the 16 canonical
 * patterns plus one sign bit, 1.25 bit/weight (§2.1).  Inference cuts the
 * int8 activations into 4-element segments, builds one table of the 16
 * pattern dot products per segment, looks each weight block up, applies its
 * sign, sums in integers and rescales once in float (§2.2).  The ternary
 * block is the solution of min ||W - a*T||^2 with ||T||_0 = 3: keep the three
 * largest |w| with their signs (§3.1).
 *
 * Conventions shared by every entry point
 *   - W is [N,K] row-major fp32 (N outputs, K inputs); x and y are [M,K] and
 *     [M,N] row-major.  y[m,n] = sum_k x[m,k] * W[n,k] in the quantized
 *     domain: y = ((float)acc[m,n] * s_x[m]) * alpha[n],
 *     acc[m,n] = sum_k q[m,k] * T[n,k] exactly in int32.
 *   - Every pointer argument is a DEVICE pointer unless stated otherwise.
 *     The caller allocates and frees every buffer; the library allocates no
 *     device memory.
 *   - `stream` is a hipStream_t passed as void* (NULL = the null stream).
 *     Every call only enqueues work on `stream` and returns; results are
 *     visible after the caller synchronizes the stream.
 *   - Argument errors are found on the host before any HIP call; such a call
 *     enqueues nothing and returns a negative status.  A failed launch
 *     returns SHERRY_ERR_HIP, or SHERRY_ERR_PARTIAL when launches of the
 *     same call were enqueued before it.  A fault inside a kernel is
 *     reported by the caller's next synchronizing HIP call, not by this
 *     library.
 *   - Shapes supported: K % 16 == 0, N % 4 == 0, 1 <= M,N,K <= 2^20
 *     (whole 4-weight blocks, 16-byte aligned int8 activation rows and
 *     whole 16-byte output stores).
 *   - Code 5-bit layout ("packed"): code c = 2*p + s per block; p = 4*z +
 *     2*r1 + r2 where z is the zero position and r1 (r2) says the 2nd (3rd)
 *     nonzero's sign differs from the 1st's; s = 1 iff the 1st nonzero is -1.
 *     Rows are grouped in tiles of 64 rows x 128 columns (1280 bytes),
 *     row-tile-major and column-tile-minor.  Tile row r = 16t + i
 *     (t = 0..3, i = 0..15) keeps its 32 codes as four groups of 8: group g
 *     (blocks 8g..8g+7) is a 40-bit little-endian string with block 8g+jj at
 *     bits [5jj, 5jj+5).  It belongs to slot L = 16g + i: group bits 0..31
 *     are the 4 bytes at tile byte 16*L + 4*t, bits 32..39 the byte at tile
 *     byte 1024 + 4*L + t.  (Slot L is what lane L of a 64-wide wave loads;
 *     it holds that lane's matrix-core operands.)  The matrix is padded to
 *     whole tiles (N up to a
 *     multiple of 64, K up to a multiple of 128); padding blocks hold code 0
 *     and no product uses them.  Total sherry_packed_bytes(N,K) =
 *     ceil(N/64) * ceil(K/128) * 1280 bytes (N*K*5/32 when no padding).
 */
#ifndef SHERRY_H
#define SHERRY_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  SHERRY_OK = 0,
  SHERRY_ERR_NULL = -1,      /* a required pointer is NULL */
  SHERRY_ERR_SHAPE = -2,     /* M, N or K out of range or not a multiple */
  SHERRY_ERR_ALIGN = -3,     /* a pointer is not aligned as required */
  SHERRY_ERR_WORKSPACE = -4, /* workspace missing or smaller than required */
  SHERRY_ERR_HIP = -5,       /* a HIP runtime call or launch failed */
  SHERRY_ERR_DEVICE = -6,    /* the current device is not a gfx950 GPU */
  SHERRY_ERR_PARTIAL = -7,   /* a launch failed after earlier launches of the
                                same call were enqueued (sherry_linear's
                                quantizer, the 64-token launches of
                                64 < M <= 128, or an earlier step of a
                                backward pass): those complete, so the output
                                is partly written; a launch that fails runs
                                nothing and every launch that runs leaves the
                                split-K workspace zero, so the workspace needs
                                no re-zeroing */
  SHERRY_ERR_ARG = -8        /* an activation, element type or eps that is
                                none of the listed ones */
} sherry_status;

/* Human-readable name of a status code (static string; never NULL). */
const char* sherry_status_string(int status);

/* Bytes of the packed 5-bit weight format for an [N,K] matrix: N*K*5/32.
 * Host-only, pure; returns 0 for an unsupported shape. */
size_t sherry_packed_bytes(int64_t N, int64_t K);

/* Bytes of scratch that sherry_gemm / sherry_gemm_i32 need for this shape
 * (0 when the chosen kernel needs none).  Host-only, pure.
 * The workspace holds one 64-bit accumulator per output when the product is
 * split along K.  It must be zero-filled once before its first use; every
 * completed call leaves it zero-filled again, so one buffer of the largest
 * size needed can serve any sequence of calls on one stream.  Calls that run
 * concurrently must not share a workspace. */
size_t sherry_workspace_bytes(int64_t M, int64_t N, int64_t K);

/* Offline compression (kernel 1), §3.1 and §2.1.
 *   W      [N,K] fp32, finite values, 16-byte aligned (read only).
 *   packed sherry_packed_bytes(N,K) bytes, 16-byte aligned (written).
 *   alpha  [N] fp32 (written): alpha[n] = (sum of the kept |W[n,k]|,
 *          accumulated in double in ascending k) / (3*K/4), rounded once.
 * Per block the smallest |w| is dropped (the lowest index on ties) and the
 * other three keep their signs (w < 0 -> -1, otherwise +1, so -0.0 -> +1). */
sherry_status sherry_quantize_pack(const float* W, int64_t N, int64_t K,
                                   void* packed, float* alpha, void* stream);

/* Per-token symmetric int8 quantization of activations (the input stage of
 * the product; the page's lookup works on int8 segments, §2.2).
 *   x    [M,K] fp32, finite, 16-byte aligned.  K % 4 == 0 is enough here.
 *   q    [M,K] int8 (written), 4-byte aligned.
 *   s_x  [M] fp32 (written): s = max_k |x[m,k]| / 127 (float division);
 *        q = clamp(rint(x / s), -127, 127) rounding half to even.
 *        An all-zero row gives s = 1 and q = 0. */
sherry_status sherry_quantize_act(const float* x, int64_t M, int64_t K,
                                  int8_t* q, float* s_x, void* stream);

/* The product, §2.2: y[m,n] = ((float)acc[m,n] * s_x[m]) * alpha[n] with
 * acc[m,n] = sum_k x[m,k] * T[n,k] in int32 (exact; any int8 value of x is
 * accepted, -128 included).
 *   x        [M,K] int8, 16-byte aligned.
 *   s_x      [M] fp32.            alpha  [N] fp32 (from sherry_quantize_pack).
 *   packed   packed weights, 16-byte aligned.
 *   y        [M,N] fp32 (written), 16-byte aligned (with N % 4 == 0 every
 *            row then starts on a 16-byte boundary; the prefill GEMM stores
 *            16 bytes per lane).
 *   workspace / workspace_bytes: scratch of at least
 *            sherry_workspace_bytes(M,N,K) bytes, 256-byte aligned, zero
 *            filled before first use (may be NULL when that size is 0).
 * Every path decodes the codes or looks them up; which one runs depends on
 * M (sherry_gemm_plan reports it), and every path returns identical results:
 *   M <= 16: the matrix-core GEMV (codes decoded to int8 {-1,0,+1}, tokens
 *            padded to 16, one 64-row weight tile per workgroup), or the
 *            lookup-table GEMV (per-segment tables of the 16 pattern dot
 *            products and their negations in LDS, one lookup per weight
 *            block and token pair);
 *   16 < M <= 64: the matrix-core GEMV with the tokens in two or four
 *            blocks of 16;
 *   64 < M <= 128: the prefill GEMM below, except when its grid is at
 *            most 64 workgroups and its waves take long shares of K (more
 *            than 12 k-tiles each up to M = 80, more than 18 up to 96,
 *            more than 24 up to 128): then that GEMV in launches of 64
 *            tokens on the same stream (sherry_workspace_bytes covers one
 *            launch);
 *   M > 128: the prefill GEMM on the int8 matrix cores, in the first
 *            workgroup tile whose grid fits the GPU in one round (at most
 *            256 tiles): 64 tokens x 128 weight rows, 128 x 128, 64 x 256,
 *            else 128 x 256; tiles 128 rows wide split each workgroup's K
 *            over 4 wave phases, 256 rows wide over 2. */
sherry_status sherry_gemm(const int8_t* x, const float* s_x, const void* packed,
                          const float* alpha, float* y, int64_t M, int64_t N,
                          int64_t K, void* workspace, size_t workspace_bytes,
                          void* stream);

/* The same product as sherry_gemm for callers that cannot allocate device
 * memory (code under HIP graph capture, tight serving loops, harnesses that
 * forbid hipMalloc): no workspace argument.  When the plan splits K, the
 * split-K cells live in a static device array of the library, 8 MiB per
 * GPU (held until the process ends), so shapes whose
 * sherry_workspace_bytes(M,N,K) exceeds 8 MiB (8388608) are rejected with
 * SHERRY_ERR_WORKSPACE before anything is enqueued.  The call allocates
 * nothing and calls no allocating routine.
 *   Arguments, alignment, shapes and results: as sherry_gemm (identical y).
 *   The first call on a device resolves the array's device address; until
 *   one call has run outside graph capture, each call first enqueues a
 *   zero fill of the array (one extra small kernel) on its stream.  Every
 *   completed call leaves the array zero again.
 *   Every call on one GPU shares that GPU's array: calls that can overlap
 *   on one GPU (different streams, or different threads without ordering)
 *   race and may return wrong sums; serialize them on one stream. */
sherry_status sherry_gemm_noalloc(const int8_t* x, const float* s_x, const void* packed,
                                  const float* alpha, float* y, int64_t M, int64_t N,
                                  int64_t K, void* stream);

/* Same product, stopping at the int32 accumulators: acc [M,N] int32
 * (written, 16-byte aligned).  Same kernels and workspace rules. */
sherry_status sherry_gemm_i32(const int8_t* x, const void* packed, int32_t* acc,
                              int64_t M, int64_t N, int64_t K, void* workspace,
                              size_t workspace_bytes, void* stream);

/* Bytes of scratch (beyond the workspace) that sherry_linear needs for this
 * shape: q [M,K] and s_x [M] when the quantization is not fused into the
 * product, else 0.  Host-only, pure; 0 for an unsupported shape. */
size_t sherry_linear_scratch_bytes(int64_t M, int64_t N, int64_t K);

/* The whole decode step from fp32 activations: per-token int8 quantization
 * (as sherry_quantize_act) followed by the product (as sherry_gemm), with
 * identical results: y is bit-identical to calling the two.  Small token
 * counts (M <= 4, M*K <= 16384) on the matrix-core GEMV path quantize inside
 * the product kernel (one launch, no round trip of q through memory);
 * otherwise q and s_x are first written to `scratch`.
 *   x        [M,K] fp32, finite, 16-byte aligned.
 *   packed, alpha, y, M, N, K: as sherry_gemm.
 *   workspace / workspace_bytes: as sherry_gemm (sherry_workspace_bytes,
 *            zero filled before first use, left zero by every call).
 *   scratch / scratch_bytes: at least sherry_linear_scratch_bytes(M,N,K)
 *            bytes, 256-byte aligned, any content (may be NULL when 0);
 *            must not overlap the workspace. */
sherry_status sherry_linear(const float* x, const void* packed, const float* alpha,
                            float* y, int64_t M, int64_t N, int64_t K,
                            void* workspace, size_t workspace_bytes,
                            void* scratch, size_t scratch_bytes, void* stream);

/* --- 2-bit baseline -------------------------------------------------------
 * The plain ternary packing the Sherry page measures its 5-bit code against
 * (§2.1: the 5-bit code cuts bit-operation overhead relative to 2-bit
 * packing): the SAME ternary weights and alpha as sherry_quantize_pack,
 * written 2 bits per weight (0 -> 00, +1 -> 01, -1 -> 11), so every product
 * is identical to sherry_gemm's and only the format (2 vs 1.25 bit/weight)
 * and its decode differ.  Layout: tiles of 64 rows x 128 columns (2048
 * bytes), row-tile-major; weight j of tile row r at bits [2j, 2j+2) of the
 * row's 256-bit little-endian string, bits 0..127 at tile byte 16*r and bits
 * 128..255 at tile byte 1024 + 16*r.  Same shape rules as the 5-bit format. */

/* ceil(N/64) * ceil(K/128) * 2048 (N*K/4 when no padding; padding is 00);
 * host-only, pure; 0 for an unsupported shape. */
size_t sherry_packed2_bytes(int64_t N, int64_t K);

/* As sherry_quantize_pack, output in the 2-bit format (packed: 16-byte
 * aligned, sherry_packed2_bytes(N,K) bytes). */
sherry_status sherry_quantize_pack2(const float* W, int64_t N, int64_t K,
                                    void* packed, float* alpha, void* stream);

/* Scratch bytes of sherry_gemm2 (same zero-fill rule as
 * sherry_workspace_bytes); 0 when M > 16 or the shape is unsupported. */
size_t sherry_gemm2_workspace_bytes(int64_t M, int64_t N, int64_t K);

/* The product on the 2-bit format, decode shapes only (1 <= M <= 16, else
 * SHERRY_ERR_SHAPE): the matrix-core GEMV with the codes decoded through a
 * 256-entry table (one lookup per 4 weights).  Arguments as sherry_gemm. */
sherry_status sherry_gemm2(const int8_t* x, const float* s_x, const void* packed,
                           const float* alpha, float* y, int64_t M, int64_t N,
                           int64_t K, void* workspace, size_t workspace_bytes,
                           void* stream);

/* --- Feed-forward operators ------------------------------------------------
 * What surrounds the product in a decoder layer: bias, activation and
 * residual in the product's epilogue, the gated block whose two products
 * share one kernel, and the layer norm that makes the int8 tokens.
 *
 * Element types of x / y / residuals / gradients (dtype): arithmetic is fp32
 * (64-bit where stated), and each output is rounded once, to nearest even. */
#define SHERRY_F32 0
#define SHERRY_F16 1
#define SHERRY_BF16 2

/* Activations (act), Phi = the normal distribution function:
 *   NONE z;  RELU max(z, 0);  RELU2 max(z, 0)^2;  SILU z / (1 + e^-z);
 *   GELU z Phi(z);
 *   GELU_TANH z (1 + tanh(sqrt(2/pi) (z + 0.044715 z^3))) / 2. */
#define SHERRY_ACT_NONE 0
#define SHERRY_ACT_RELU 1
#define SHERRY_ACT_RELU2 2
#define SHERRY_ACT_SILU 3
#define SHERRY_ACT_GELU 4
#define SHERRY_ACT_GELU_TANH 5

/* The product with a bias, an activation and a residual in its epilogue:
 *   y[m,n] = act((acc[m,n] * s_x[m]) * alpha[n] + bias[n]) + residual[m,n].
 *   x, s_x, packed, alpha, M, N, K: as sherry_gemm.
 *   bias     [N] fp32, or NULL.       act: SHERRY_ACT_*.
 *   residual [M,N] of type dtype, 16-byte aligned, or NULL.  It may be y
 *            itself (each element is read before it is written, by the same
 *            thread); it must not overlap y otherwise.
 *   y        [M,N] of type dtype (written), 16-byte aligned.
 *   workspace: at least sherry_gemm_fused_workspace_bytes(M,N,K) bytes, by
 *            the rules of sherry_workspace_bytes (zero before its first use,
 *            left zero); the two operators' calls may share one buffer on
 *            one stream with each other and with sherry_gemm.
 * Runs on sherry_gemm's matrix-core kernels and plan (the lookup-table path,
 * which only sherry_gemm_plan_override selects, is taken as path 2 here). */
sherry_status sherry_gemm_fused(const int8_t* x, const float* s_x, const void* packed,
                                const float* alpha, const float* bias, int act,
                                const void* residual, void* y, int dtype, int64_t M, int64_t N,
                                int64_t K, void* workspace, size_t workspace_bytes, void* stream);
size_t sherry_gemm_fused_workspace_bytes(int64_t M, int64_t N, int64_t K);

/* The gated feed-forward block's first half, both products in one kernel:
 *   h[m,n] = act(g) * u,  g = (acc_gate * s_x[m]) * alpha_gate[n],
 *                         u = (acc_up * s_x[m]) * alpha_up[n].
 *   packed_gate, packed_up: two [N,K] matrices in the packed format; the
 *   other arguments as sherry_gemm_fused.  act(g) * u is formed in fp32. */
sherry_status sherry_glu(const int8_t* x, const float* s_x, const void* packed_gate,
                         const float* alpha_gate, const void* packed_up, const float* alpha_up,
                         int act, void* h, int dtype, int64_t M, int64_t N, int64_t K,
                         void* workspace, size_t workspace_bytes, void* stream);
size_t sherry_glu_workspace_bytes(int64_t M, int64_t N, int64_t K);

/* Gradients of the two, with the rounding of x to int8 taken as the identity:
 * dx is the gradient of the token x * s_x, dz that of the value the
 * activation is applied to.
 *   gemm_fused:  dz = dy * act'(z);
 *     dx[m,k] = sum_n dz[m,n] * alpha[n] * T[n,k],
 *     dalpha[n] = sum_m dz[m,n] * acc[m,n] * s_x[m],  dbias[n] = sum_m dz[m,n]
 *     (the residual's gradient is dy itself).
 *   glu:  dg = dh * u * act'(g), du = dh * act(g); dx sums both matrices'
 *     terms, dalpha_gate and dalpha_up are as dalpha.
 *   relu' and relu2' are 0 at 0.
 *   dy, dh   [M,N] of type dtype, 16-byte aligned.
 *   x, s_x, packed, alpha, bias, act: as the forward call had them; the sums
 *            are computed again, so the forward saves nothing.
 *   dx       [M,K] of type dtype (written), 16-byte aligned; overlaps no input.
 *   dalpha, dbias, ...  [N] fp32 (written), 4-byte aligned, each may be NULL.
 *   scratch  at least the queried bytes, any content, 256-byte aligned.
 * dx's terms dz * alpha are rounded to fp16 under one power-of-two scale per
 * token: one term for bf16 results, off by at most 2^-11 of itself or 2^-16 of
 * the token's largest, a high and a low one for fp16 and fp32 results (2^-22
 * or 2^-24), whatever the sizes of the scales and gradients they come from
 * (and 2^-145, where all of a token's are near fp32's least numbers).
 * The sums run in a fixed order: equal calls give equal bits. */
sherry_status sherry_gemm_fused_backward(const void* dy, const int8_t* x, const float* s_x,
                                         const void* packed, const float* alpha,
                                         const float* bias, int act, void* dx, float* dalpha,
                                         float* dbias, int dtype, int64_t M, int64_t N, int64_t K,
                                         void* scratch, size_t scratch_bytes, void* stream);
size_t sherry_gemm_fused_backward_scratch_bytes(int64_t M, int64_t N, int64_t K, int dtype);

sherry_status sherry_glu_backward(const void* dh, const int8_t* x, const float* s_x,
                                  const void* packed_gate, const float* alpha_gate,
                                  const void* packed_up, const float* alpha_up, int act, void* dx,
                                  float* dalpha_gate, float* dalpha_up, int dtype, int64_t M,
                                  int64_t N, int64_t K, void* scratch, size_t scratch_bytes,
                                  void* stream);
size_t sherry_glu_backward_scratch_bytes(int64_t M, int64_t N, int64_t K, int dtype);

/* Layer norm of each token:
 *   y = ((x - mean) * rstd) * weight + bias,  mean = sum x / K,
 *   rstd = 1 / sqrt(sum (x - mean)^2 / K + eps).
 *   x       [M,K] of type dtype, 16-byte aligned, 1 <= M <= 2^20,
 *           4 <= K <= 2^20, K % 4 == 0.
 *   weight, bias  [K] fp32, 16-byte aligned, or NULL (ones, zeros).
 *   eps     finite and positive.
 *   y       [M,K] of type dtype (written), 16-byte aligned; may be x.
 *   mean, rstd  [M] fp32 (written), for the backward pass; both or neither
 *           NULL. */
sherry_status sherry_layernorm(const void* x, const float* weight, const float* bias, float eps,
                               void* y, float* mean, float* rstd, int dtype, int64_t M, int64_t K,
                               void* stream);

/* The same token as the products take it: the norm's value v, computed in 64
 * bits, as int8 with one scale,
 *   s_x = max|v| / 127 rounded to fp32 (1 if that is 0),
 *   q = clamp(rint(v / s_x), -127, 127), half to even.
 *   q  [M,K] int8 (written), 4-byte aligned;  s_x [M] fp32 (written).
 *   A token with a value v that is not finite (one feature of it, or a weight
 *   or bias, is infinite or NaN) gets s_x = NaN, so that its products are NaN;
 *   its q then has no meaning.  The rest as sherry_layernorm. */
sherry_status sherry_layernorm_quantize(const void* x, const float* weight, const float* bias,
                                        float eps, int8_t* q, float* s_x, float* mean, float* rstd,
                                        int dtype, int64_t M, int64_t K, void* stream);

/* Gradients of sherry_layernorm, with xh = (x - mean) * rstd and
 * g = dy * weight:
 *   dx = rstd * (g - sum g / K - xh * sum(g * xh) / K),
 *   dweight = sum over tokens of dy * xh,  dbias = sum over tokens of dy.
 *   dy, x   [M,K] of type dtype;  mean, rstd [M] as the forward wrote them.
 *   weight  as the forward's.
 *   dx      [M,K] of type dtype (written); may be dy, must not be x.
 *   dweight, dbias  [K] fp32 (written), 4-byte aligned, each may be NULL.
 *   scratch at least sherry_layernorm_backward_scratch_bytes(M,K) bytes, any
 *           content, 256-byte aligned.
 * For sherry_layernorm_quantize it is the gradient with the rounding to int8
 * taken as the identity.  The sums run in a fixed order: equal calls give
 * equal bits. */
sherry_status sherry_layernorm_backward(const void* dy, const void* x, const float* mean,
                                        const float* rstd, const float* weight, void* dx,
                                        float* dweight, float* dbias, int dtype, int64_t M,
                                        int64_t K, void* scratch, size_t scratch_bytes,
                                        void* stream);
size_t sherry_layernorm_backward_scratch_bytes(int64_t M, int64_t K);

/* --- Attention operators ----------------------------------------------------
 * What lies between a layer's stacked q/k/v product and its output product:
 * the norm and rotation of each head, a paged cache of keys and values in 8
 * bits, and attention over it.  dim is a head's features: a multiple of 16
 * from 16 to 256.  At most 1024 query heads and 512 key heads, 2^20 rows T.
 * Rows are T rows of heads * dim values of type dtype (SHERRY_F32 ...), a
 * `stride` of values apart (a multiple of 8, so that slices of a stacked row
 * serve), 16-byte aligned. */

/* Norm of each query and key head and the rotation by its token's position:
 *   r = 1 / sqrt(sum x^2 / dim + eps),  y = x * r * weight (norm != 0) or x,
 *   z = y with the pairs (a, b) among its first rotary_dim features turned:
 *       (a cos t - b sin t, b cos t + a sin t),  t = positions[row] * freqs[i];
 *   pair i is features i and i + rotary_dim / 2, or 2 i and 2 i + 1 with
 *   `interleaved`.
 *   x        [T, x_stride]: q_heads heads of queries, then k_heads of keys
 *            (what follows them in a row, the values, is not looked at).
 *   q_weight, k_weight  [dim] fp32, 16-byte aligned, or NULL (ones); NULL
 *            without the norm.
 *   eps      finite and positive (not looked at without the norm).
 *   freqs    [rotary_dim / 2] in 64 bits, radians a position (NULL where
 *            rotary_dim is 0); rotary_dim a multiple of 8, at most dim.
 *            Angles are taken in 64 bits.
 *   positions [T] int32.
 *   q [T, q_heads, dim], k [T, k_heads, dim]  (written), 16-byte aligned; they
 *            overlap no input. */
sherry_status sherry_qk_norm_rope(const void* x, int64_t x_stride, const float* q_weight,
                                  const float* k_weight, float eps, int norm, const double* freqs,
                                  int64_t rotary_dim, int interleaved, const int32_t* positions,
                                  void* q, void* k, int dtype, int64_t T, int64_t q_heads,
                                  int64_t k_heads, int64_t dim, void* stream);

/* Its gradients, from those of q and k and the same x:
 *   dy = dz turned back,  dweight = sum over tokens and heads of dy * x * r,
 *   dx = r * (g - x * r * mean(g * x * r)),  g = dy * weight.
 *   dq [T, q_heads, dim], dk [T, k_heads, dim].
 *   dx       the first (q_heads + k_heads) * dim values of rows dx_stride
 *            apart (written; what follows them is left as it was); may be x
 *            with the same stride, overlaps no input otherwise (SHERRY_ERR_ARG).
 *   dq_weight, dk_weight  [dim] fp32 (written), each may be NULL; NULL without
 *            the norm (x and scratch may be NULL then too).
 *   scratch  at least the queried bytes, any content, 256-byte aligned.
 * The sums run in a fixed order: equal calls give equal bits. */
sherry_status sherry_qk_norm_rope_backward(const void* dq, const void* dk, const void* x,
                                           int64_t x_stride, const float* q_weight,
                                           const float* k_weight, float eps, int norm,
                                           const double* freqs, int64_t rotary_dim, int interleaved,
                                           const int32_t* positions, void* dx, int64_t dx_stride,
                                           float* dq_weight, float* dk_weight, int dtype, int64_t T,
                                           int64_t q_heads, int64_t k_heads, int64_t dim,
                                           void* scratch, size_t scratch_bytes, void* stream);
size_t sherry_qk_norm_rope_backward_scratch_bytes(int64_t T, int64_t q_heads, int64_t k_heads,
                                                  int64_t dim);

/* The cache: pages of page_size tokens (a power of two from 16 to 1024) of
 * every head, in blocks of 16 tokens of one head with one scale each:
 *   k  int8 [pages, heads, page_size / 16, dim / 16, 16 tokens, 16 features],
 *   v  int8 [pages, heads, page_size / 16, dim / 16, 16 features, 16 tokens],
 *   k_scale, v_scale  fp32 [pages, heads, page_size / 16]; value = int8 * scale.
 * k and v 16-byte aligned device pointers, fewer than 2^31 blocks; the struct
 * itself is host memory. */
typedef struct {
  void* k;
  void* v;
  float* k_scale;
  float* v_scale;
  int64_t pages, page_size, heads, dim;
} sherry_kv_cache;

/* The calls below take S sequences at once:
 *   table    [S, table_width] int32: position t of sequence i lies in page
 *            table[i][t / page_size] (table_width * page_size <= 2^30).
 *   starts   [S + 1] int32, ascending from 0 to at most T: rows starts[i] ..
 *            starts[i + 1] - 1 of the call are sequence i's (rows behind the
 *            last sequence's are neither read nor written).
 *   lens     [S] int32: tokens sequence i has; the call's rows are its last.
 * They are device memory and checked there: a position without a page (slot
 * past the table, page number out of range) is not written, reads as NaN, and
 * makes the queries that see it, or all of a sequence longer than its table,
 * NaN.  Entries past a sequence's last page are not looked at. */

/* Writes new tokens' keys and values: rows of k and v (heads * dim values) go
 * to the positions lens[i] - n .. lens[i] - 1.  A block's scale is the least
 * power of two 2^e, e >= -126, with max|x| <= 127 * 2^e over its tokens so far,
 * and q = rint(x / 2^e), half to even.  Where a block has earlier tokens (the
 * position of the first new one is no multiple of 16) its scale can only grow,
 * and the earlier values are rounded again, rint(q * old / new).  A value that
 * is not finite makes its block's scale NaN, and so the block's values.  One past
 * 127 * 2^121 (1.98 * 2^127) is 64 * 2^122, infinity in fp32.
 * A block is written by one sequence of a call only, and a block's first
 * position first; earlier positions may be written again (drafts that were
 * refused): values at later ones are then never looked at, but the block's scale
 * stays what they made it.  A large draft leaves the block's other tokens, and
 * those written after it, as coarse as its scale; one that is not finite leaves
 * them NaN.  Writing the block again from its first position makes the scale anew. */
sherry_status sherry_cache_write(const sherry_kv_cache* cache, const void* k, int64_t k_stride,
                                 const void* v, int64_t v_stride, int dtype, const int32_t* table,
                                 int64_t table_width, const int32_t* starts, const int32_t* lens,
                                 int64_t S, int64_t T, void* stream);

/* Reads the last starts[i + 1] - starts[i] tokens of each sequence back:
 *   k, v  [T, heads, dim] of type dtype (written), 16-byte aligned. */
sherry_status sherry_cache_read(const sherry_kv_cache* cache, void* k, void* v, int dtype,
                                const int32_t* table, int64_t table_width, const int32_t* starts,
                                const int32_t* lens, int64_t S, int64_t T, void* stream);

/* Causal attention of each sequence's newest tokens (which the cache holds
 * already) over the cache: query row j of n in sequence i is at position
 * p = lens[i] - n + j and sees positions t <= p, and with a window (> 0) only
 * those with p - t < window or t < sinks;
 *   s_t = scale * q . k_t,  y = sum e^(s_t - lse) v_t,  lse = log sum e^(s_t).
 * Query head h reads key head h / (q_heads / heads).  A query that sees nothing
 * gives y = 0 and lse = -infinity.
 *   q        rows of q_heads * dim values;  q_heads a multiple of heads.
 *   window   0: none.        sinks: looked at with a window only.
 *   y        [T, q_heads, dim] of type dtype (written), 16-byte aligned; it
 *            overlaps no input (over q: SHERRY_ERR_ARG).
 *   lse      [T, q_heads] fp32 (written), or NULL.
 *   workspace  at least sherry_cache_attention_workspace_bytes() bytes, by the
 *            rules of sherry_workspace_bytes (zero before its first use, left
 *            zero; one buffer may serve all calls on a stream).
 *   scratch  at least the queried bytes, any content, 256-byte aligned.
 * Products run in fp16 with fp32 sums: 16-bit queries are exact (bf16 down to
 * 2^-38 of the row's largest) and fp32 queries are rounded to 22 bits; the weights
 * e^(s - m) are rounded to 11 bits for bf16, to 22 for fp16 and fp32; weights times value scales below 2^-31 of
 * the largest weight times the largest scale that the query sees are lost (what it
 * does not see has no part in this).  Value scales are taken to be powers of two,
 * as cache_write leaves them.  The sums run in a fixed order: equal calls give equal
 * bits (a row's bits may differ with the other rows of a call, which decide how the
 * work is split).  One kernel takes all sequences of a call, chosen by T * q_heads /
 * (heads * S), the rows a key head has on average of a sequence, and table_width * page_size as the longest sequence's length: a
 * table no wider than needed helps short prompts, and a long prompt among very many
 * single tokens is faster in a call of its own. */
sherry_status sherry_cache_attention(const void* q, int64_t q_stride, int64_t q_heads,
                                     const sherry_kv_cache* cache, const int32_t* table,
                                     int64_t table_width, const int32_t* starts,
                                     const int32_t* lens, int64_t S, int64_t T, float scale,
                                     int64_t window, int64_t sinks, void* y, float* lse, int dtype,
                                     void* workspace, size_t workspace_bytes, void* scratch,
                                     size_t scratch_bytes, void* stream);
size_t sherry_cache_attention_workspace_bytes(void);
size_t sherry_cache_attention_scratch_bytes(int64_t T, int64_t S, int64_t q_heads, int64_t heads,
                                            int64_t dim);

/* Launch plan sherry_gemm uses for a shape (host-only, pure; for
 * diagnostics and benchmarks).  Any output pointer may be NULL.
 *   path: 0 = lookup-table GEMV (per-segment tables in LDS, §2.2; M <= 16),
 *         1 = decode + int8 matrix-core GEMM (M > 64, except where path 2
 *             runs in launches of 64 tokens),
 *         2 = decode + int8 matrix-core GEMV (M <= 128; grid is per launch
 *             of at most 64 tokens).
 *   grid: workgroups per launch; block: threads per workgroup;
 *   splits: K-splits per output row group (1 = none);
 *   lds_bytes: LDS per workgroup. */
sherry_status sherry_gemm_plan(int64_t M, int64_t N, int64_t K, int* path,
                               int* grid, int* block, int* splits,
                               int* lds_bytes);

/* Launch plan of sherry_linear's product for a shape, with the same outputs
 * as sherry_gemm_plan, plus fused = 1 when the quantization runs inside the
 * product kernel (one launch), else 0 (sherry_quantize_act first, then the
 * product on the plan above).  The fused form on path 2 with a K-split takes
 * twice the waves per row tile of sherry_gemm's plan and, from 8 K-splits on,
 * half the splits: its workgroups each read their tokens' whole fp32 rows
 * for the scales, so fewer, wider workgroups cost less.  Host-only, pure;
 * follows sherry_gemm_plan_override (with rw or splits set, the fused form
 * keeps that plan). */
sherry_status sherry_linear_plan(int64_t M, int64_t N, int64_t K, int* path,
                                 int* grid, int* block, int* splits,
                                 int* lds_bytes, int* fused);

/* Tuning knob for benchmark sweeps and tests (host-only).  Replaces the
 * built-in launch plan for shapes with M <= 128 for every later call in this
 * process (M > 128 always uses path 1):
 *   path   -1 = built-in choice, or 0, 1, 2 as in sherry_gemm_plan; for
 *          16 < M <= 128, 1 gives the prefill GEMM and 0 or 2 the GEMV.
 *   rw     path 0: row tiles per workgroup, 1, 2 or 4 (the workgroup's 4
 *          waves are rw row tiles x 4/rw waves sharing one), or 8: 4 row
 *          tiles x 2 waves (512 threads; needs K-splits of at least 2
 *          k-tiles, else 4 is taken);
 *          path 2: waves per workgroup sharing its one row tile, 4, 8 or
 *          16 (at most 8 when M > 16);
 *          path 1 (forced): 1 or 2 = tiles of 64 or 128 tokens;
 *          0 (or a value the path does not take) = built-in choice.
 *   ch     path 0: k-tiles (128 inputs) per LDS table stage: 1, 2, 4
 *          or 8, capped so one stage stays within 32 KB (with rw = 8 at
 *          least 2, one per wave, up to 64 KB);
 *          path 1 (forced): 2 or 4 k-phases (4: tiles 128 weight rows
 *          wide, each workgroup's K split four ways);
 *          0 = built-in.
 *   splits K-splits per output row group; 0 = built-in choice.
 * Results do not depend on the plan.  sherry_workspace_bytes reflects the
 * override, so query it after setting one.  Not thread-safe with respect to
 * concurrent calls.  Returns SHERRY_ERR_SHAPE for an invalid value. */
sherry_status sherry_gemm_plan_override(int path, int rw, int ch, int splits);

/* --- Diagnostics (not part of the product) -------------------------------
 * Ceilings for the benchmark, measured in the same process as the product:
 * the plain streaming-read rate of a device buffer, the cost of an empty
 * launch and the rate of the decode step alone. */

/* Reads `bytes` (a multiple of 16) of device memory at `src` (16-byte
 * aligned) with 16-byte loads: grid x block threads (block a multiple of 64,
 * at most 1024), each keeping `unroll` (1, 2, 4 or 8) loads in flight, the
 * grid walking the buffer front to back.  Nothing is written unless the XOR
 * of all the data equals one fixed constant; then one dword goes to `sink`
 * (device, 4-byte aligned).  Asynchronous on `stream`. */
sherry_status sherry_probe_read(const void* src, size_t bytes, void* sink, int grid, int block,
                                int unroll, void* stream);

/* Enqueues an empty kernel (one workgroup of 64 threads) on `stream`. */
sherry_status sherry_probe_empty(void* stream);

/* The decode step of the matrix-core kernels with nothing else in the loop:
 * grid x block threads (block a multiple of 64, at most 1024; iters and
 * grid in [1, 2^20]) each look up sherry_probe_decode_codes(iters, 1, 1)
 * codes as code pairs in a 1024-entry table of 8-byte entries in LDS
 * (two 8-byte lookups per 4 codes, the product's decode).  The looked-up
 * values are folded and written to `sink` (device, 4-byte aligned) only if
 * they equal one fixed constant.  Asynchronous on `stream`. */
sherry_status sherry_probe_decode(int iters, void* sink, int grid, int block, void* stream);

/* Codes one sherry_probe_decode launch looks up (0 for non-positive
 * arguments).  Host-only. */
int64_t sherry_probe_decode_codes(int iters, int grid, int block);

#ifdef __cplusplus
}
#endif

#endif /* SHERRY_H */
