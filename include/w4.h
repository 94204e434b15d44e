/*
 * w4.h -- C ABI of libw4.so: the group-wise INT4 weight-only quantized linear layer on MI355X
 * (gfx950), and the operators of a decoder layer around it (rotary positions, attention over a
 * paged key-value cache, cross attention, the cache's tables, the residual norm).
 *
 *   y = x . W_hat^T (+ b),   W_hat[j][k] = s[j][G] * (code[j][k] - z[j][G]),  G = k / group_size
 *
 * Pages cited (title, then section):
 *   [Lab5]  "Lab 5: Gemma4 端到端推理优化"
 *   [Orin]  "Jetson Orin AGX INT4 推理优化实践：super 分支从 9 tok/s 到 24 tok/s"
 *   [Infra] "【infra之路】12-投机解码、量化与推理引擎对比"
 *   [QAT]   "Yeniden paketlenmiş QAT Gemma 4 26B-A4B, tek bir TPU v6e'de FP8 işlemenin 1.9 katı
 *            verimle sunuluyor"
 *
 * Conventions shared by every entry point
 *   - Array arguments are DEVICE pointers owned by the caller.  The library never allocates,
 *     frees or retains device memory and keeps no state between calls (thread-safe; calls on one
 *     stream are ordered by that stream).  The linear layers and the codecs need no scratch
 *     memory (partial sums meet in LDS); GPTQ's factor and column loop take caller-owned work
 *     buffers.  The one exception is w4_gptq_quantize_noalloc, for callers that cannot
 *     allocate: it keeps its work buffer in a device array of the library (see there).
 *   - bf16 values travel as uint16_t bit patterns.  `stream` is a hipStream_t passed as void*
 *     (NULL = the default stream).  Calls enqueue kernels and return without synchronizing.
 *   - Arguments are validated on the host before anything is enqueued.  A failed check returns
 *     a nonzero w4_status and enqueues nothing; a failed launch returns W4_ERR_HIP and the HIP
 *     error text is kept in w4_last_hip_error() (per host thread).
 *   - Outputs are overwritten, never accumulated into.  Inputs and outputs must not overlap.
 *   - Identical inputs give bitwise-identical outputs (no floating-point atomics).
 *   - Inputs must be finite; NaN/Inf inputs are not checked and give unspecified results.
 *
 * Packed weight format [Lab5 INT4 线性量化], [Lab5 融合INT4反量化与矩阵乘]
 *   k_pad    = ceil(d_in / group_size) * group_size   (group_size in {32, 64, 128, 256})
 *            = ceil(d_in / 32) * 32 with one group per row   (group_size == 0)
 *   n_groups = k_pad / group_size   (1 when group_size == 0)
 *   qweight  uint8 [d_out][k_pad/2]: two 4-bit codes per byte, column 2i in the low nibble and
 *            column 2i+1 in the high nibble.  Rows are output channels.
 *   scales   bf16 [d_out][n_groups]
 *   zeros    bf16 [d_out][n_groups] for W4_ASYM; absent (NULL) for W4_SYM, whose zero point is
 *            the constant 8 (signed levels -8..7 stored as codes 0..15).
 *   Padded columns k >= d_in carry the zero code and decode to exactly 0.
 */
#ifndef W4_H
#define W4_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    W4_OK = 0,
    W4_ERR_NULL = 1,        /* a required pointer is NULL, or zeros given/missing for the mode */
    W4_ERR_SHAPE = 2,       /* a size is < 1, or a leading dimension is smaller than its row  */
    W4_ERR_GROUP = 3,       /* group_size not in {0, 32, 64, 128, 256}                        */
    W4_ERR_ALIGN = 4,       /* a pointer or leading dimension breaks the alignment rules       */
    W4_ERR_RANGE = 5,       /* a size beyond the limits stated for the entry point             */
    W4_ERR_UNSUPPORTED = 6, /* valid arguments this entry point does not serve (e.g. M > 64)   */
    W4_ERR_HIP = 7          /* a HIP launch or query failed; see w4_last_hip_error()           */
} w4_status;

enum { W4_SYM = 0, W4_ASYM = 1 };         /* quantization mode                      */
enum { W4_OUT_BF16 = 0, W4_OUT_F32 = 1 }; /* element type of y                      */

/* Upper bounds checked by every entry point (W4_ERR_RANGE beyond them). */
#define W4_MAX_DIM ((int64_t)1 << 24)  /* d_out, d_in, M, K                      */
#define W4_MAX_W4A8_D_IN ((int64_t)1 << 20) /* keeps sum(code * q) within int32: 2^20*15*127 < 2^31 */
#define W4_GEMV_MAX_M 64
#define W4_DECODE_MAX_D_IN ((int64_t)1 << 16) /* d_in of the decode (M <= 64) entry points     */
#define W4_MAX_GPTQ_D_IN 8192 /* the GPTQ factorization holds d_in x d_in fp32 matrices      */

/*
 * w4_packed_layout -- host-only size query (no GPU work).
 * [Lab5 INT4 线性量化]: the input dimension is padded to a whole number of groups.
 * Writes k_pad, n_groups and the byte size of qweight (d_out * k_pad / 2) for the given shape.
 * Any output pointer may be NULL.  Errors: W4_ERR_SHAPE, W4_ERR_GROUP, W4_ERR_RANGE.
 */
int w4_packed_layout(int64_t d_out, int64_t d_in, int group_size, int64_t *k_pad,
                     int64_t *n_groups, size_t *qweight_bytes);

/*
 * w4_pack -- round-to-nearest (RTN) quantization of an fp32 weight into the packed format.
 * [Lab5 INT4 线性量化]: per (output row, group):
 *   W4_SYM : s = bf16(max|r| / 7), z = 8
 *   W4_ASYM: s = bf16((max r - min r) / 15), z = bf16(round(-min r / s))
 *   code = clip(round(r / s + z), 0, 15), with the stored bf16 s and z; round = ties-to-even.
 * Statistics run over the padded group (pads are 0), so pads encode to z and decode to 0.
 * A group whose bf16 scale is 0 is stored as s = +0, z = +0 (ASYM) and all codes equal to z.
 * The fp32 steps are single IEEE operations in this order:  a/7 (or (mx-mn)/15), bf16 rounding,
 * (-mn)/s, rint, bf16 rounding, then per element  r/s, +z, rint, clamp.
 *   w        fp32 [d_out][ldw], ldw >= d_in, 4-byte aligned
 *   qweight  uint8 [d_out][k_pad/2], 16-byte aligned
 *   scales   bf16 [d_out][n_groups];  zeros bf16 [d_out][n_groups] iff mode == W4_ASYM, else NULL
 */
int w4_pack(const float *w, int64_t d_out, int64_t d_in, int64_t ldw, int group_size, int mode,
            uint8_t *qweight, uint16_t *scales, uint16_t *zeros, void *stream);

/*
 * GPTQ -- quantization that compensates each column's rounding error in the columns after it,
 * producing the packed format of w4_pack.  [Lab5 从 RTN 到 GPTQ]:
 *   objective  min_Q ||X W^T - X Q^T||_F^2 over calibration activations X [N][d_in];
 *   H = (2/N) X^T X; dead columns (H_ii = 0) get H_ii = 1 and zero weights; H += alpha mean(diag H) I;
 *   H^-1 = U^T U (U upper triangular); columns in order: q_i = the code of w_i (the group's scale
 *   and zero by w4_pack's rule from the current, already updated weights of the group at its first
 *   column), e_i = (w_i - q_i) / U_ii, W[:, i:] -= e_i U[i, i:];
 *   L_pred = 1/2 sum_i ||w_i - q_i||^2 / U_ii^2.
 * Everything runs in fp32, as on the page.  Three calls, each enqueued on `stream`:
 *
 * w4_gptq_hessian -- h = (2/N) X^T X.
 *   x  bf16 [N][ldx], ldx >= d_in, only k < d_in read;  h  fp32 [d_in][d_in] (written in full)
 *
 * w4_gptq_factor -- dead columns, damping, and U with (H + lambda I)^-1 = U^T U.
 *   h     fp32 [d_in][d_in], in: the Hessian; destroyed (its lower triangle is worked in place)
 *   alpha the damping factor (the reference uses 0.01), >= 0; with alpha = 0 the Hessian must be
 *         positive definite (N >= d_in calibration rows in general position), else U holds NaN
 *   u     fp32 [d_in][d_in], out: U (zeros below the diagonal)
 *   work  fp32 [d_in][d_in], scratch (the reverse Cholesky factor V, H = V V^T, U = V^-1)
 *   dead  uint8 [d_in], out: 1 for dead columns
 *   The factorization launches about 2 d_in small kernels (an offline step).
 *
 * w4_gptq_quantize -- the column loop.
 *   w        fp32 [d_out][ldw], in: the weights; destroyed (the error-updated working copy)
 *   u, dead  from w4_gptq_factor (dead may be NULL: no dead columns)
 *   group_size, mode, qweight, scales, zeros: as for w4_pack
 *   work     fp32 [d_out][32], scratch (a block's errors)
 *   row_loss fp32 [d_out] or NULL: each row's share of L_pred
 * Limits: d_in <= W4_MAX_GPTQ_D_IN (W4_ERR_RANGE).
 */
int w4_gptq_hessian(const uint16_t *x, int64_t N, int64_t d_in, int64_t ldx, float *h,
                    void *stream);
int w4_gptq_factor(float *h, int64_t d_in, float alpha, float *u, float *work, uint8_t *dead,
                   void *stream);
int w4_gptq_quantize(float *w, int64_t d_out, int64_t d_in, int64_t ldw, const float *u,
                     const uint8_t *dead, int group_size, int mode, uint8_t *qweight,
                     uint16_t *scales, uint16_t *zeros, float *work, float *row_loss,
                     void *stream);

/*
 * w4_gptq_quantize_noalloc -- w4_gptq_quantize without the `work` argument, for callers that
 * cannot allocate device memory (code under HIP graph capture, tight serving loops, harnesses
 * that forbid hipMalloc). The block errors live in a device array of the library,
 * W4_GPTQ_NOALLOC_MAX_ROWS rows of 32 floats (8 MiB), which each GPU holds from the first call on
 * it until the process ends. Every call on one GPU shares that array: calls that overlap on one
 * GPU (other streams, other host threads) race and give unspecified results; serialize them.
 * The call allocates nothing. d_out > W4_GPTQ_NOALLOC_MAX_ROWS returns W4_ERR_RANGE; every other
 * argument and result is that of w4_gptq_quantize.
 */
#define W4_GPTQ_NOALLOC_MAX_ROWS ((int64_t)1 << 16)
int w4_gptq_quantize_noalloc(float *w, int64_t d_out, int64_t d_in, int64_t ldw, const float *u,
                             const uint8_t *dead, int group_size, int mode, uint8_t *qweight,
                             uint16_t *scales, uint16_t *zeros, float *row_loss, void *stream);

/*
 * w4_qat_repack -- pack a weight trained on the 4-bit grid (a QAT export stored in bf16) without
 * re-quantizing it: the g32 symmetric format of w4_pack (group_size = 32, W4_SYM).
 * [QAT "Yeniden nicelendirme değil, yeniden paketleme"]: per row and group of 32 columns,
 *   a = max|r|; for m = 1 .. 8 the step a / m is kept if it reproduces the whole group, i.e.
 *   every v = r / (a / m) (fp32) is within 1/16 of a level l = rint(v) in [-8, 7];
 *   the kept levels give the codes l + 8 and the least-squares step s = sum r l / sum l^2
 *   (fp64 sums and quotient, rounded to fp32, stored as bf16).
 * A group no m reproduces is off the grid: it is packed by w4_pack's symmetric rule and m = 0 is
 * reported for it. An all-zero group has m = 1 and scale +0. Padded columns decode to 0.
 *   w        bf16 [d_out][ldw], ldw >= d_in, ldw % 8 == 0, 16-byte aligned; only k < d_in is read
 *   qweight  uint8 [d_out][k_pad/2], k_pad = ceil(d_in/32)*32, 16-byte aligned
 *   scales   bf16 [d_out][k_pad/32]
 *   m_out    uint8 [d_out][k_pad/32] or NULL: the m kept per group, 0 for groups off the grid
 * The result is bit-identical to the CPU reference of the same rule.
 */
int w4_qat_repack(const uint16_t *w, int64_t d_out, int64_t d_in, int64_t ldw, uint8_t *qweight,
                  uint16_t *scales, uint8_t *m_out, void *stream);

/*
 * w4_gemv -- W4A16 decode linear for 1 <= M <= 64 token rows, weights read once per call.
 * [Lab5 Prefill和Decode分流] (the small-M decode path), [Lab5 融合INT4反量化与矩阵乘]
 * (dequantize in registers inside the product, never a dense weight in memory),
 * [Orin 模型尺寸和 decode 的真实瓶颈] (y_j = sum_i W_ji x_i + b_j).
 *   x        bf16 [M][ldx], ldx >= d_in, ldx % 8 == 0, 16-byte aligned; only k < d_in is used
 *   qweight, scales, zeros, group_size: the packed format above (zeros NULL iff symmetric)
 *   bias     bf16 [d_out] or NULL
 *   y        [M][ldy], ldy >= d_out, element type out_dtype (W4_OUT_BF16 / W4_OUT_F32),
 *            naturally aligned.  Accumulation is fp32; the bf16 output is the round-to-nearest-
 *            even image of the fp32 result of the same call.
 * M > 64 returns W4_ERR_UNSUPPORTED (use w4_gemm); d_in <= W4_DECODE_MAX_D_IN = 65536 (else
 * W4_ERR_RANGE; w4_gemm serves any d_in up to W4_MAX_DIM).
 */
int w4_gemv(const uint16_t *x, int64_t M, int64_t ldx, const uint8_t *qweight,
            const uint16_t *scales, const uint16_t *zeros, const uint16_t *bias, int64_t d_out,
            int64_t d_in, int group_size, void *y, int64_t ldy, int out_dtype, void *stream);

/*
 * w4_gemv_ws -- w4_gemv with a caller-provided workspace, for 2 <= M <= 64 token rows.
 * [Lab5 Prefill和Decode分流] (the small-M path reads every weight once per step),
 * [Lab5 Linear形状采样] (the projections of a decoder layer: q/k/v and o have few rows, down has
 * few rows and long ones).
 * On matrices with fewer than four 16-row tiles per compute unit (d_out < 64 * CUs) and long
 * rows (at least 64 KiB of codes per compute unit; groups of 128 or 256 columns or one per row),
 * the reduction over d_in is split over column slices that run on different compute units: each
 * slice converts only its own columns of the activations and stores fp32 partial sums in `work`,
 * and a second kernel adds the slices in slice order (so the result is deterministic).  Other
 * shapes run the w4_gemv path.
 *   work        device memory of at least w4_gemv_work_bytes(M, d_out, d_in, group_size) bytes,
 *               16-byte aligned, owned by the caller; its contents on entry do not matter and
 *               are left undefined.  Calls that share a workspace must be ordered (one stream,
 *               or events).  May be NULL when that size is 0.
 *   work_bytes  its size in bytes
 *   the other arguments as for w4_gemv, with the same result within the tolerance.
 * Returns W4_ERR_NULL for a missing workspace, W4_ERR_RANGE for one that is too small,
 * W4_ERR_ALIGN for a misaligned one, and otherwise the codes of w4_gemv.
 */
int w4_gemv_ws(const uint16_t *x, int64_t M, int64_t ldx, const uint8_t *qweight,
               const uint16_t *scales, const uint16_t *zeros, const uint16_t *bias, int64_t d_out,
               int64_t d_in, int group_size, void *y, int64_t ldy, int out_dtype, void *work,
               size_t work_bytes, void *stream);

/*
 * w4_gemv_work_bytes -- the workspace w4_gemv_ws needs for these sizes (0: none; also 0 for
 * arguments w4_gemv_ws rejects): S * M * d_out * 4 bytes of partial sums for S column slices
 * (S <= d_in / 128 + 1).  It depends only on its arguments and the device's compute-unit count.
 */
size_t w4_gemv_work_bytes(int64_t M, int64_t d_out, int64_t d_in, int group_size);

/*
 * w4_gemv_glu -- the gate/up half of the MLP with its gate fused into the epilogue:
 *   h[m][j] = SiLU(g[m][j]) * u[m][j],  SiLU(v) = v / (1 + exp(-v)),
 *   g = x W_gate^T (+ b_gate),  u = x W_up^T (+ b_up),
 * [Lab5 基础] (FFN(x) = W_down [SiLU(W_gate x) (.) (W_up x)]), [Orin 后续还能继续优化什么] (the
 * SwiGLU kernel boundary). One launch reads the fused weight once and writes only h.
 *   qweight, scales, zeros: a packed weight of 2 d_ff rows, the gate rows [0, d_ff) then the
 *            up rows [d_ff, 2 d_ff) (w4_pack of the stacked gate and up weights)
 *   bias     bf16 [2 d_ff] (gate biases, then up biases) or NULL
 *   y        [M][ldy], ldy >= d_ff: h, as fp32 or its round-to-nearest-even bf16 image
 *   the other arguments as for w4_gemv.
 * Served by the int8 matrix-core decode kernel: 1 <= M <= 4 tokens, group_size 128 or 256, or
 * 0 with k_pad a multiple of 128, and k_pad <= 32768 / M (its activation stage); other arguments
 * return W4_ERR_UNSUPPORTED (use w4_gemv on the fused weight and apply the gate separately).
 * d_in <= W4_DECODE_MAX_D_IN (W4_ERR_RANGE beyond).
 */
int w4_gemv_glu(const uint16_t *x, int64_t M, int64_t ldx, const uint8_t *qweight,
                const uint16_t *scales, const uint16_t *zeros, const uint16_t *bias, int64_t d_ff,
                int64_t d_in, int group_size, void *y, int64_t ldy, int out_dtype, void *stream);

/*
 * w4_gemm -- W4A16 prefill linear for any M >= 1 (the arguments of w4_gemv, and the same
 * result within the tolerance).
 * [Lab5 Prefill和Decode分流] (large M: dequantize once per tile and run a dense matrix product).
 * Weight tiles are dequantized on chip to the fp32 values s (code - z), split into two bf16
 * halves whose sum is exact, and multiplied on the bf16 matrix cores with fp32 accumulation.
 * No dense weight is written to memory.
 */
int w4_gemm(const uint16_t *x, int64_t M, int64_t ldx, const uint8_t *qweight,
            const uint16_t *scales, const uint16_t *zeros, const uint16_t *bias, int64_t d_out,
            int64_t d_in, int group_size, void *y, int64_t ldy, int out_dtype, void *stream);

/*
 * act_quant_int8 -- per-token dynamic symmetric int8 quantization of activations.
 * [Orin 从 FP 线性层到 INT4 DP4A 的数学推导], [Infra 2.2 量化的基本概念]:
 *   s_x[m] = max_k |x[m][k]| / 127 (fp32),  q[m][k] = clip(round(x[m][k] / s_x[m]), -127, 127)
 * round = ties-to-even, the division is one correctly rounded fp32 division.  A token whose
 * values are all zero gets s_x = 0 and q = 0.
 *   x      bf16 [M][ldx], ldx >= K, ldx % 8 == 0, 16-byte aligned
 *   q      int8 [M][ldq], ldq >= K, ldq % 16 == 0, 16-byte aligned; q[m][k] for k < K only
 *   s_x    fp32 [M]
 *   q_sum  int32 [M] = sum_k q[m][k], or NULL
 */
int act_quant_int8(const uint16_t *x, int64_t M, int64_t K, int64_t ldx, int8_t *q, int64_t ldq,
                   float *s_x, int32_t *q_sum, void *stream);

/*
 * w4a8_gemv -- W4A8 decode linear: int4 weights x int8 activations into an int32 accumulator.
 * [Orin 从 FP 线性层到 INT4 DP4A 的数学推导], [Orin INT32 accumulator 是否安全]:
 *   acc[m][j] = sum_{k < d_in} (code[j][k] - 8) * q[m][k]          (exact, int32)
 *   y[m][j]   = s_w[j] * s_x[m] * acc[m][j] + b[j]                  (fp32)
 * Weights are a per-row symmetric pack (w4_pack with group_size = 0, W4_SYM); s_w is that pack's
 * scales array.  1 <= M <= 64 (W4_ERR_UNSUPPORTED beyond: use w4a8_gemm) and
 * d_in <= W4_DECODE_MAX_D_IN = 65536, the decode kernels' limit (W4_ERR_RANGE beyond: w4a8_gemm
 * serves d_in up to W4_MAX_W4A8_D_IN = 2^20, the bound that keeps every partial sum in int32).
 *   q        int8 [M][ldq], ldq >= d_in, ldq % 16 == 0, 16-byte aligned (from act_quant_int8)
 *   s_x      fp32 [M]
 *   qweight  uint8 [d_out][k_pad/2], k_pad = ceil(d_in/32)*32, 16-byte aligned
 *   s_w      bf16 [d_out];  bias bf16 [d_out] or NULL
 *   y        [M][ldy], ldy >= d_out, out_dtype as for w4_gemv
 *   acc      int32 [M][d_out] (dense), or NULL: the exact accumulators, for bit-exact checks
 */
int w4a8_gemv(const int8_t *q, const float *s_x, int64_t M, int64_t ldq, const uint8_t *qweight,
              const uint16_t *s_w, const uint16_t *bias, int64_t d_out, int64_t d_in, void *y,
              int64_t ldy, int out_dtype, int32_t *acc, void *stream);

/*
 * w4a8_linear -- the W4A8 decode linear with the activation quantization folded in: the result
 * of act_quant_int8 followed by w4a8_gemv, in one launch, without q in memory.
 * [Orin 从 FP 线性层到 INT4 DP4A 的数学推导] (s_x = max|x|/127, q = clamp(rint(x/s_x), +-127)),
 * [Orin INT32 accumulator 是否安全], and the kernel boundary between quantization and linear that
 * [Orin 后续还能继续优化什么] names for further fusion.
 *   x        bf16 [M][ldx], ldx >= d_in, ldx % 8 == 0, 16-byte aligned; only k < d_in is used
 *   qweight, s_w, bias, y, out_dtype, acc: as for w4a8_gemv
 *   s_x      fp32 [M] or NULL: receives the token scales
 * The codes, s_x and acc are bit-identical to those of act_quant_int8 + w4a8_gemv on the same x.
 * Limits: those of w4a8_gemv (1 <= M <= 64, d_in <= W4_DECODE_MAX_D_IN, W4_ERR_RANGE beyond).
 * Every workgroup quantizes the whole activation row it needs; rows longer than the kernel's
 * activation stage (k_pad > 32768) return W4_ERR_UNSUPPORTED: use the two calls.
 */
int w4a8_linear(const uint16_t *x, int64_t M, int64_t ldx, const uint8_t *qweight,
                const uint16_t *s_w, const uint16_t *bias, int64_t d_out, int64_t d_in, void *y,
                int64_t ldy, int out_dtype, float *s_x, int32_t *acc, void *stream);

/*
 * w4a8_gemm -- W4A8 prefill linear for any M >= 1: the arguments and the result of w4a8_gemv
 * (acc bit-identical, y within the same rounding), for token counts where the weight tile is
 * reused across many tokens.
 * [Orin 从 FP 线性层到 INT4 DP4A 的数学推导] (the integer form of the linear layer),
 * [Infra 2.3] (int8 products with int32 accumulation for the compute-bound large-batch case).
 * The codes (0..15) and the int8 activations are multiplied on the int8 matrix cores as they
 * are; sum_k 8 q[m][k] is subtracted per token from the int32 sums, so acc is exact.
 *   q, s_x, qweight, s_w, bias, y, out_dtype, acc: as for w4a8_gemv, with any M >= 1
 * Limits (W4_ERR_RANGE beyond them): M <= W4_MAX_DIM, d_in <= W4_MAX_W4A8_D_IN, M * ldq < 2^31
 * and d_out * k_pad / 2 < 2^31 (32-bit buffer offsets), ceil(M / 128) * ceil(d_out / 256) < 2^23
 * (the launch grid).
 */
int w4a8_gemm(const int8_t *q, const float *s_x, int64_t M, int64_t ldq, const uint8_t *qweight,
              const uint16_t *s_w, const uint16_t *bias, int64_t d_out, int64_t d_in, void *y,
              int64_t ldy, int out_dtype, int32_t *acc, void *stream);

/*
 * The operators of a decoder layer that stand between its linears: rotary positions and the append
 * to a paged key-value cache, attention of one new token and of prompts over that cache, of sequences
 * that share prefixes and over an encoder's states, the tables of a step, and the residual norm.
 * (Lab5 基础: the layer's attention with its sliding window; Infra 第四部分: the paged cache of a
 * serving batch.)
 *
 * w4_kv_cache -- a paged key-value cache and the sequences in it.  The struct is read on the host
 * during the call; its arrays are device memory.
 *   k, v        bf16, 16-byte aligned; element d of key-value head h in slot s of page p is
 *               k[p * page_stride + s * slot_stride + h * head_stride + d]  (v likewise), so both
 *               [page][slot][head][d] and [page][head][slot][d] fit.  Strides are in elements and
 *               multiples of 8; what lies between two rows is never touched.
 *   n_pages     pages in k and v (1 .. 2^31 - 1); page offsets may pass 32 bits, while the
 *               elements spanned inside one page must be fewer than 2^31
 *   page_size   slots of a page, a power of two, 1 .. 32768
 *   n_kv_heads  1 .. 1024;   head_dim  a multiple of 8, 8 .. 256
 *   page_table  int32 [n_seqs][ld_table], table_cols entries used (table_cols * page_size up to
 *               2^30 positions): position p of sequence b lives
 *               in slot p % page_size of page page_table[b][p / page_size].  Only entries of
 *               positions that an operator reads or writes matter; the others may hold anything.
 *               An entry outside [0, n_pages) never makes an access leave the cache (reads see
 *               another page's values, appends are dropped).
 *   kv_len      int32 [n_seqs]: keys of each sequence, the tokens of this call included.  Values
 *               below 0 count as 0, values above table_cols * page_size as that.
 * Slots that hold no visible key are never used, whatever bits they hold (NaN included).  Nor does a
 * token that another one sees reach the rows of those that do not see it, infinite or NaN as its key
 * and value may be.  A score that is NaN makes y and lse of its row NaN; a visible value that is NaN
 * or infinite makes its dimension of y what such a sum is (that infinity; NaN for both, and where
 * the weight is too small for fp32).  An infinite element of a visible key may make its score NaN,
 * and so may scores of 2^127 and more in magnitude.
 *
 * Token rows: sequence b has the rows q_start[b] <= t < q_start[b + 1] (q_start int32
 * [n_seqs + 1], nondecreasing, q_start[0] = 0, q_start[n_seqs] = T), which are its LAST tokens: row
 * q_start[b] + i stands at position kv_len[b] - (q_start[b + 1] - q_start[b]) + i.  A row whose
 * position is negative sees no key and is not appended.
 *
 * Visible keys of a token at position p:  j <= p, and with window > 0 also
 *   j > p - window  or  j < sinks    (the window counts the token itself; sinks are the first
 *   tokens of a sequence that stay visible).  window = 0 means no window; sinks are then ignored.
 */
typedef struct w4_kv_cache {
    uint16_t *k, *v;
    int64_t n_pages, page_stride, slot_stride, head_stride;
    int32_t page_size, n_kv_heads, head_dim;
    const int32_t *page_table;
    int64_t n_seqs, table_cols, ld_table;
    const int32_t *kv_len;
} w4_kv_cache;

#define W4_MAX_HEAD_DIM 256
#define W4_MAX_HEADS 1024           /* n_heads, n_kv_heads                                  */
#define W4_NORM_MAX_D ((int64_t)1 << 15) /* the residual norm keeps a row in registers      */

enum { W4_ROPE_HALF = 0, W4_ROPE_INTERLEAVED = 1 }; /* pairs (i, i + R/2), or (2i, 2i + 1)   */
enum { W4_ROPE_PLAIN = 0, W4_ROPE_LINEAR = 1, W4_ROPE_NTK = 2, W4_ROPE_YARN = 3 };

/*
 * w4_rope_frequencies -- host-only: the angle per position of each rotated pair, and the amplitude,
 * for the usual ways of reaching contexts longer than a model was trained on.  R = rot_dim (even,
 * 2 .. 256), i < R / 2, plain frequencies f_i = base^(-2 i / R):
 *   W4_ROPE_PLAIN   f_i                                       (factor and context are ignored)
 *   W4_ROPE_LINEAR  f_i / factor                              (position interpolation)
 *   W4_ROPE_NTK     f_i with base * factor^(R / (R - 2)): the lowest frequency is divided by
 *                   factor, the highest kept                  (R >= 4)
 *   W4_ROPE_YARN    f_i (1 - g_i) + f_i / factor * g_i; pairs that turn 32 times or more over the
 *                   original `context` positions keep f_i (g = 0), pairs that turn once or less
 *                   are divided (g = 1), linear in i between those two dimensions; the amplitude
 *                   is 0.1 ln(factor) + 1.  ("YaRN: Efficient Context Window Extension of Large
 *                   Language Models", arXiv 2309.00071, sections 3.2 - 3.4)
 * Computed in 64 bits and rounded once.
 *   inv_freq   HOST fp32 [R / 2], out;   amplitude  HOST fp32, out, may be NULL (1 but for YARN)
 * Errors: W4_ERR_NULL, W4_ERR_SHAPE (rot_dim), W4_ERR_RANGE (base <= 1, factor < 1, context < 1 or
 * any of them not finite), W4_ERR_UNSUPPORTED (an unknown scaling).
 */
int w4_rope_frequencies(int rot_dim, int scaling, double base, double factor, double context,
                        float *inv_freq, float *amplitude);

/*
 * w4_rope_append -- rotary positions on the fused q/k/v projection of T tokens, the rotated keys
 * and the values appended to the cache.  Per token at position p, per q and k head, for the first
 * rot_dim dimensions in pairs (a, b):
 *   t = p * inv_freq[i];   a' = factor (a cos t - b sin t),   b' = factor (a sin t + b cos t)
 * the other dimensions of q and k, and v, are copied bit for bit.  The angle keeps full precision
 * at any position: it is reduced modulo one turn in 64 bits.
 *   qkv       bf16 [T][ldqkv], the n_heads query heads, then the key heads, then the value heads,
 *             each of head_dim; ldqkv % 8 == 0, 16-byte aligned (the output of a w4 linear)
 *   q_start   int32 [n_seqs + 1], or NULL: one token per sequence (T = n_seqs)
 *   inv_freq  fp32 [rot_dim / 2], rot_dim even, 2 .. head_dim;  factor  finite
 *   q         bf16 [T][ldq], ldq >= n_heads * head_dim, ldq % 8 == 0, 16-byte aligned.  It must not
 *             overlap the rows of qkv (W4_ERR_SHAPE; columns of one buffer beside them are fine),
 *             nor may the cache: one thread's output is another one's input.
 * Tokens at negative positions, or whose page table entry lies outside the cache, are not
 * appended; their q row is written all the same.
 */
int w4_rope_append(const uint16_t *qkv, int64_t T, int64_t ldqkv, int n_heads,
                   const int32_t *q_start, const float *inv_freq, int rot_dim, int layout,
                   float factor, const w4_kv_cache *cache, uint16_t *q, int64_t ldq,
                   void *stream);

/*
 * w4_attn_decode -- attention of one new token per sequence over the cache, the token at position
 * kv_len[b] - 1:
 *   s_j = scale * q . k_j,   y = sum_j exp(s_j) v_j / sum_j exp(s_j),   lse = ln sum_j exp(s_j)
 * over the visible keys j; query head h reads key-value head h / (n_heads / n_kv_heads).  A token
 * that sees no key gets y = 0 and lse = -inf.
 *   q      bf16 [n_seqs][ldq], head h at element h * head_dim; ldq % 8 == 0, 16-byte aligned
 *   scale  finite, >= 0
 *   y      [n_seqs][ldy], ldy >= n_heads * head_dim, element type out_dtype, naturally aligned
 *   lse    fp32 [n_seqs][n_heads] or NULL
 *   y, lse and work must overlap neither what the call reads nor each other (not checked)
 *   work   device memory of at least w4_attn_decode_work_bytes bytes, 16-byte aligned, as for
 *          w4_gemv_ws; may be NULL when that size is 0
 * Long caches are split over several compute units and joined in order (deterministic).
 * w4_attn_decode_work_bytes reads only sizes, no array; 0 for arguments the call rejects.
 * Limits (W4_ERR_RANGE beyond them): n_seqs * n_heads times one more than the number of 32-key tiles
 * that table_cols pages can hold < 2^31 - 2^16; and the 2^24 - 1 workgroups of a launch, enough for
 * n_seqs * n_heads up to 2^24 - 2^16 at any length.
 */
int w4_attn_decode(const uint16_t *q, int64_t ldq, int n_heads, const w4_kv_cache *cache,
                   float scale, int64_t window, int64_t sinks, void *y, int64_t ldy,
                   int out_dtype, float *lse, void *work, size_t work_bytes, void *stream);
size_t w4_attn_decode_work_bytes(int n_heads, const w4_kv_cache *cache, int64_t window,
                                 int64_t sinks);

/*
 * w4_attn_prefill -- the same attention for T tokens of n_seqs sequences (token rows as above),
 * each at its own position: prompts, chunks of prompts, or several new tokens per sequence.
 *   q      bf16 [T][ldq];  q_start int32 [n_seqs + 1];  y [T][ldy];  lse fp32 [T][n_heads] or NULL
 *   the other arguments as for w4_attn_decode.
 * Limits (W4_ERR_RANGE): T * n_heads and n_seqs * n_heads below 2^31, and T * n_heads / 128 +
 * n_seqs * n_kv_heads below 2^24, the workgroups of a launch.  The softmax weights enter
 * the second product as bf16, their sum in fp32.
 */
int w4_attn_prefill(const uint16_t *q, int64_t T, int64_t ldq, int n_heads,
                    const int32_t *q_start, const w4_kv_cache *cache, float scale,
                    int64_t window, int64_t sinks, void *y, int64_t ldy, int out_dtype,
                    float *lse, void *work, size_t work_bytes, void *stream);
size_t w4_attn_prefill_work_bytes(int64_t T, int n_heads, const w4_kv_cache *cache,
                                  int64_t window, int64_t sinks);

/*
 * w4_attn_shared -- the same attention for sequences that share prefixes (a system prompt, a document,
 * the question of several samples): the keys of a prefix are read and multiplied once for all rows of
 * the sequences that share it, not once for each.  The visible keys and the result are those of
 * w4_attn_decode (q_start NULL: T = n_seqs, one row each) and w4_attn_prefill; only the place of a key
 * differs: position j of sequence b with prefix g = prefix_of[b] is
 *   j < prefix length of g:  position j of the prefix, by row g of the prefixes' table
 *   else:                    position j of the sequence, by its own row of the page table
 * so that entries of a sequence's row below its prefix are not read, and a prefix may end inside a
 * page.  kv_len counts the prefix.  A row that stands inside the prefix sees it up to itself.
 *
 * w4_prefixes -- the prefixes of a batch; a struct on the host, arrays on the device.
 *   prefix_of   int32 [n_seqs]: the prefix of each sequence, in any order; a value outside
 *               [0, n_prefixes) for none
 *   table       int32 [n_prefixes][ld_table], table_cols entries used: pages of the same cache.  (Rows
 *               of the page table itself serve as well.)  Entries outside the cache as there.
 *   len         int32 [n_prefixes]: keys of each prefix; below 0 as 0, above table_cols * page_size
 *               as that
 *   n_prefixes  1 .. W4_MAX_PREFIXES;  table_cols * page_size up to 2^30
 * The other arguments are those of w4_attn_prefill.  Limits (W4_ERR_RANGE): T <= 2^21, n_seqs
 * <= 2^16, T * n_heads < 2^26, table_cols * page_size of either table up to 2^26, and n_kv_heads (T G / 64
 * + n_seqs + n_prefixes) times the 32-key tiles that either table's pages can hold below 2^29, for G =
 * n_heads / n_kv_heads.  The softmax weights enter the second product as bf16, or as two bf16 values where
 * head_dim is up to 128 and a key-value head has up to 16 rows (tokens times G) over the same prefix or of
 * one sequence; their sum in fp32.  (So above 128 dims single tokens have weights within 2^-8 of
 * themselves here, 2^-16 in w4_attn_decode.)  Partial results are fp32 in `work`, joined in a fixed order.
 * work: 8 (head_dim + 4) bytes for each row and query head, and 1024 (head_dim + 2) for each compute unit.
 */
typedef struct w4_prefixes {
    const int32_t *prefix_of, *table, *len;
    int64_t n_prefixes, table_cols, ld_table;
} w4_prefixes;

#define W4_MAX_PREFIXES 256

int w4_attn_shared(const uint16_t *q, int64_t T, int64_t ldq, int n_heads, const int32_t *q_start,
                   const w4_kv_cache *cache, const w4_prefixes *prefixes, float scale,
                   int64_t window, int64_t sinks, void *y, int64_t ldy, int out_dtype, float *lse,
                   void *work, size_t work_bytes, void *stream);
size_t w4_attn_shared_work_bytes(int64_t T, int n_heads, const w4_kv_cache *cache,
                                 const w4_prefixes *prefixes, int64_t window, int64_t sinks);

/*
 * w4_attn_cross -- cross attention: every row sees all kv_len[b] keys of its sequence, which are an
 * encoder's states (of another length than the rows, and without positions).
 *   q        bf16 [T][ldq]; the rows q_start[b] .. q_start[b + 1] - 1 belong to sequence b: prompt
 *            tokens, or the newest tokens of the beams of a request.  q_start NULL: T = n_seqs, one
 *            row each
 *   cache    keys and values of the encoder's states; a dense [n_seqs][length][n_kv_heads][head_dim]
 *            is a cache of pages in ascending order
 *   the other arguments as for w4_attn_prefill.  A sequence without states gives y = 0, lse = -inf.
 * The weights of the second product are within 2^-16 of themselves without q_start; with it they are those
 * of w4_attn_shared where T n_heads / n_kv_heads <= 16 n_seqs, else those of w4_attn_prefill.
 * Limits (W4_ERR_RANGE): those of w4_attn_decode without q_start, else those of w4_attn_prefill.
 */
int w4_attn_cross(const uint16_t *q, int64_t T, int64_t ldq, int n_heads, const int32_t *q_start,
                  const w4_kv_cache *cache, float scale, void *y, int64_t ldy, int out_dtype,
                  float *lse, void *work, size_t work_bytes, void *stream);
size_t w4_attn_cross_work_bytes(int64_t T, int n_heads, const w4_kv_cache *cache);

/*
 * w4_batch_tables -- the tables of a step, made on the device from the lengths of its requests: pages
 * for the new tokens, the token rows of each sequence, and the slot of each row.  The results are what
 * the operators above take, so that a step recorded once replays as sequences begin, grow and end.
 *   L = kv_len[b],  m = n_new[b],  [begin, end) = spans[b]: the entries of row b of the page table that
 *   name pages of its own.  (Entries below `begin` are those of a shared prefix, or not used.)
 *   m >= 0  entries end .. ceil((L + m) / page_size) - 1 get free pages, in the order of the sequences
 *           and of the entries; kv_len_out[b] = L + m;  spans_out[b] = [begin, end + pages it got)
 *   m < 0   the sequence ends: its pages are free from the next call on; kv_len_out[b] = 0,
 *           spans_out[b] = [0, 0).  A sequence that begins sets kv_len and spans itself: 0 and [0, 0),
 *           or P and [P / page_size, P / page_size) after a prefix of P keys.
 *   q_start[b + 1] = sum of max(m, 0) up to b;  row t = q_start[b] + i stands at position L + i:
 *   seqs[t] = b,  positions[t] = L + i,  slots[t] = page * page_size + (L + i) % page_size.
 * Free pages lie in a ring: ring_state = {head, count, missing}, number k of `count` at place
 * (head + k) % ring_size.  Pages are taken from its head; pages that come back follow its last one, in
 * the order of the sequences and of the entries.  Where no page is left the entry becomes -1 (an
 * append there is dropped), the row's slot -1, and missing_out counts those entries.  The step can then be
 * made again from the kv_len, spans and ring_state that it had (all three: pages taken and returned are
 * taken and returned again), after a call in which a sequence ended, or with pages put into the ring
 * behind its last one and `count` raised.  So a caller that may run out keeps them: an output in place
 * overwrites them.  Entries past the table's last column are neither written nor counted; rows there get
 * slot -1, while lengths and positions count on, up to 2^31 - 1.
 *   kv_len       int32 [n_seqs], values below 0 count as 0;  kv_len_out  int32 [n_seqs]
 *   n_new        int32 [n_seqs], values up to 2^30 - 1;  spans, spans_out  int32 [n_seqs][2]
 *   ring_state, ring_state_out  int32 [3]
 *   page_table   int32 [n_seqs][ld_table], table_cols entries used, in and out
 *   page_size    a power of two, 1 .. 32768;  table_cols * page_size and n_seqs * table_cols up to 2^30
 *   ring         int32 [ring_size], in and out.  Pages beyond its size are dropped
 *   q_start      int32 [n_seqs + 1];  sums beyond T count as T
 *   slots int64 [T], seqs and positions int32 [T], each may be NULL; rows behind the last sequence's
 *                get -1 in all three.  T  0 .. W4_MAX_DIM
 *   An output may be the input of its kind (kv_len_out = kv_len, ...); no other overlap (not checked).
 */
int w4_batch_tables(const int32_t *kv_len, const int32_t *n_new, const int32_t *spans,
                    int64_t n_seqs, int32_t *page_table, int64_t table_cols, int64_t ld_table,
                    int page_size, int32_t *ring, int64_t ring_size, const int32_t *ring_state,
                    int64_t T, int32_t *q_start, int64_t *slots, int32_t *seqs,
                    int32_t *positions, int32_t *kv_len_out, int32_t *spans_out,
                    int32_t *ring_state_out, void *stream);

/*
 * w4_residual_norm -- the seam between two blocks of a layer: the norm after a block, its gate and
 * residual scale, the residual add, and the norm before the next block, in one pass:
 *   n = x,  or  rms(x, w_post) where w_post is given
 *   r' = r + alpha * g * n         (g = 1 without a gate)
 *   y = rms(r', w_pre),            rms(u, w) = u / sqrt(mean(u^2) + eps) * (w + weight_offset)
 * All in fp32; r' is rounded once to its own type, y once to bf16 (from the unrounded r').
 *   x         bf16 [T][ldx], or NULL: y = rms(r, w_pre) alone (w_post, gate, r_out then NULL too)
 *   r         [T][ldr], r_dtype W4_OUT_BF16 or W4_OUT_F32
 *   w_post    bf16 [d] or NULL;  w_pre bf16 [d]
 *   gate      bf16 [T][ldg], or one vector [d] for all tokens with ldg = 0, or NULL
 *   alpha, weight_offset  finite;  eps  finite, >= 0
 *   r_out     as r, [T][ldr_out]; may be r itself (with ldr_out = ldr), else no overlap
 *   y         bf16 [T][ldy]; no overlap with the other arrays (not checked)
 * d <= W4_NORM_MAX_D (W4_ERR_RANGE beyond).  Leading dimensions are >= d and otherwise free;
 * pointers are naturally aligned.  (Rows that start at 16-byte boundaries are read faster.)
 */
int w4_residual_norm(const uint16_t *x, int64_t ldx, const void *r, int64_t ldr, int r_dtype,
                     int64_t T, int64_t d, const uint16_t *w_post, const uint16_t *w_pre,
                     float weight_offset, const uint16_t *gate, int64_t ldg, float alpha,
                     float eps, void *r_out, int64_t ldr_out, uint16_t *y, int64_t ldy,
                     void *stream);

/* Text for a w4_status value (static storage). */
const char *w4_status_string(int status);

/* Text of the last HIP error seen by this host thread ("" if none). */
const char *w4_last_hip_error(void);

#ifdef __cplusplus
}
#endif

#endif /* W4_H */
