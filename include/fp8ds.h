/*
 * fp8ds.h -- C ABI of the FP8 delayed-scaling Linear for AMD MI355X (gfx950).
 *
 * The library computes the hot path of an FP8 training Linear with delayed
 * per-tensor scaling:
 *
 *   amax of a BF16/FP32 tensor  ->  scale from an amax-history window
 *   ->  saturating round-to-nearest-even cast to OCP E4M3 / E5M2
 *   ->  FP8 x FP8 GEMM with FP32 accumulation (NN, NT, TN)
 *   ->  dequant by 1/(s_a * s_b) into BF16, with the output amax fused.
 *
 * Sources (cited by page title and section):
 *   [P1] "算子与编译器：FP8 训练与优化器 Kernel" (charles2530.github.io)
 *   [P2] "FP8 混合精度训练工程实践：从 H100 到大模型训练的范式跃迁" (ybb.press)
 *   [P3] "LLM FP8 微调上线生产实战：用 Amax Scaling、层级白名单与 BF16 回退守住收敛"
 *        (oh-bug.com)
 *   [OCP] the OCP 8-bit floating point formats (Micikevicius et al., "FP8 Formats
 *        for Deep Learning", in [P3]'s reference list) for special values.
 *
 * Conventions for every entry point:
 *   - Pointers are DEVICE pointers unless a parameter says "host".  The caller
 *     owns every buffer; the library keeps no pointer after the call returns and
 *     allocates no device memory.
 *   - Every call is asynchronous on `stream` (0 = the null stream): it validates
 *     its arguments on the host, enqueues kernels and returns.  Device-side
 *     results are ready after the stream is synchronised.
 *   - Return value: FP8DS_OK (0) or a negative fp8ds_status.  On failure nothing
 *     has been enqueued (validation) or a launch failed (FP8DS_ERR_HIP), and
 *     fp8ds_last_error() returns a thread-local message.  No C++ exception,
 *     abort or exit crosses the ABI.  A device fault (e.g. a pointer that does
 *     not span the stated size) surfaces at the caller's next synchronisation.
 *   - Zero-size inputs are legal no-ops that still write their scalar outputs
 *     (amax = 0, saturation count = 0, scale_used = *scale).
 *   - Row-major layouts; `ld*` are leading dimensions in elements.
 *   - Calls that write the same output buffers must not overlap (the fused
 *     amax / counters are reset by the call that writes them).  The `_acc`
 *     variants (fp8ds_cast_acc, fp8ds_gemm_acc) combine into their amax and
 *     counters instead; fp8ds_scale_update_clear zeroes such accumulators for
 *     the next step, so a training step needs no reset launches.
 */
#ifndef FP8DS_H
#define FP8DS_H

#include <stdint.h>

#include <hip/hip_runtime_api.h>

#ifdef __cplusplus
extern "C" {
#endif

#define FP8DS_ABI_VERSION 8

typedef enum {
  FP8DS_OK = 0,
  FP8DS_ERR_NULL = -1,        /* a required pointer is NULL */
  FP8DS_ERR_SHAPE = -2,       /* negative / overflowing size, or ld too small */
  FP8DS_ERR_ENUM = -3,        /* a format, dtype, op or algo value out of range */
  FP8DS_ERR_ALIGN = -4,       /* pointer or leading dimension not 16-byte aligned */
  FP8DS_ERR_HIP = -5,         /* a HIP runtime call or kernel launch failed */
  FP8DS_ERR_UNSUPPORTED = -6, /* valid but unsupported combination (e.g. TT) */
  FP8DS_ERR_VALUE = -7        /* a scalar argument out of its range (fp8ds_adamw) */
} fp8ds_status;

/* FP8 formats ([P2] §一 "FP8 格式设计"; [P3] §核心原理 "E4M3 与 E5M2 承担不同职责"):
 * E4M3: bias 7, largest finite 448, no infinity (OCP "fn" variant, [OCP]).
 * E5M2: bias 15, largest finite 57344, with +-inf ([OCP]).
 * E2M1: the 4-bit element of MXFP4 (OCP Microscaling Formats): 0, 0.5, 1, 1.5, 2, 3, 4, 6
 * and their negatives; accepted only where a call says so. */
typedef enum { FP8DS_E4M3 = 0, FP8DS_E5M2 = 1, FP8DS_E2M1 = 2 } fp8ds_format;

/* High-precision element types of inputs and GEMM outputs. */
typedef enum { FP8DS_F32 = 0, FP8DS_BF16 = 1 } fp8ds_dtype;

/* Window reductions of the amax history ([P3] §核心原理 "Delayed Scaling
 * 用历史换取稳定性", the table of strategies: max over the window, or the most
 * recent value). */
typedef enum { FP8DS_ALGO_MAX = 0, FP8DS_ALGO_MOST_RECENT = 1 } fp8ds_algo;

/* GEMM operand layout: N = used as stored, T = the stored array is transposed. */
typedef enum { FP8DS_OP_N = 0, FP8DS_OP_T = 1 } fp8ds_op;

/* GEMM datapath.
 * FP8DS_MMA_EXACT: the FP8 operands are widened exactly to F16 inside the kernel
 *   and multiplied on the F16 matrix cores; products are exact and every sum is an
 *   FP32 addition, so |acc - exact| stays at FP32 rounding level.  Default.
 * FP8DS_MMA_FP8: the FP8 matrix instructions of gfx950 on the FP8 bytes, at twice
 *   the F16 rate.  These instructions add each group of 8 products at a fixed
 *   point about 13 bits below the group's largest product, so a product 2^14 or
 *   more smaller than its largest neighbour is lost.  Measured worst case about
 *   2^-11 of the largest product per instruction; on Gaussian-like operands the
 *   error is FP32-like, on heavy-tailed gradients (outliers next to small values)
 *   it exceeds 1e-5 * sum|a*b| for most elements.  Opt-in only. */
typedef enum { FP8DS_MMA_EXACT = 0, FP8DS_MMA_FP8 = 1 } fp8ds_mma;

/* ABI version (FP8DS_ABI_VERSION of the built library). */
int fp8ds_abi_version(void);

/* Static description of a status code (never NULL). */
const char* fp8ds_status_string(int status);

/* Thread-local detail of the last failing call on this thread ("" if none). */
const char* fp8ds_last_error(void);

/*
 * fp8ds_amax -- amax = max_i |x_i| of the unscaled tensor.
 * [P2] §四 "动态缩放" (the quantize step takes the maximum absolute value of the
 * high-precision tensor); [P3] §核心原理 "Scale 决定数值是否进入可表示区间".
 *
 *   x      device, n elements of `xt` (BF16 or FP32), 16-byte aligned.
 *   n      element count, n >= 0.
 *   amax   device, 1 float: overwritten with the result.  Exact (the maximum is
 *          one of the inputs).  NaN anywhere gives the canonical qNaN 0x7FC00000;
 *          otherwise +inf if any element is infinite; 0 for n == 0; |-0| = +0.
 */
int fp8ds_amax(const void* x, fp8ds_dtype xt, int64_t n, float* amax, hipStream_t stream);

/*
 * fp8ds_cast -- scaled saturating cast of a [rows x cols] tensor to FP8, with the
 * input amax fused into the same pass.
 * [P2] §四 "动态缩放" (quantize: multiply by the scale, clamp to the format's
 * range, convert); [P2] §五 (the fp8 linear op casts input and weight with their
 * scales before the product).
 *
 *   q[i] = encode_fmt( fl32(x[i] * (*scale)) )
 * where fl32 is one IEEE fp32 multiply (round to nearest even) and encode is the
 * saturating round-to-nearest-even conversion: |v| > max (infinities included)
 * gives the largest finite code of v's sign, NaN gives 0x7F | sign << 7, and the
 * sign is kept on underflow to zero.
 *
 *   x          device, rows*cols elements of `xt`, row-major, contiguous, 16-byte aligned.
 *   rows,cols  >= 0.
 *   fmt        target format.
 *   scale      device, 1 float: the delayed scale of this step (read once).  Finite and
 *              not 0, as fp8ds_scale_update makes it: NaN products that another scale
 *              makes of inputs other than NaN may be coded as +-max.
 *   q          device, rows*cols bytes, row-major, 16-byte aligned.
 *   q_t        device or NULL: if non-NULL also receives the transposed copy,
 *              [cols x rows] row-major (q_t[c*rows + r] == q[r*cols + c]), for GEMM
 *              operands the caller wants K-contiguous.  16-byte aligned; rows at
 *              most 65535 * 128, cols at most 2^31 - 128 (else FP8DS_ERR_SHAPE).
 *   scale_used device or NULL: receives a copy of *scale -- the snapshot the FP8
 *              bytes were made with.  GEMMs must be given this snapshot, because
 *              fp8ds_scale_update overwrites *scale for the next step.
 *   amax       device or NULL: receives max|x| of the UNSCALED input (as fp8ds_amax).
 *   sat_count  device or NULL: receives #{i : |fl32(x[i]*scale)| > max}
 *              (infinities counted, NaN not).
 */
int fp8ds_cast(const void* x, fp8ds_dtype xt, int64_t rows, int64_t cols, fp8ds_format fmt,
               const float* scale, uint8_t* q, uint8_t* q_t, float* scale_used, float* amax,
               uint64_t* sat_count, hipStream_t stream);

/*
 * fp8ds_cast_acc -- fp8ds_cast that accumulates its reductions instead of
 * resetting them (same arguments, same bytes q / q_t):
 *   amax       device or NULL: on return max(previous amax, max|x|) (fp32 bits of
 *              non-negative values compared as integers; NaN as fp8ds_amax).
 *   sat_count  device or NULL: the saturation count of this call added to it.
 *   scale_used device or NULL: written by the cast kernel itself.
 * With amax and sat_count zeroed before a step (fp8ds_scale_update_clear of the
 * previous step does it), the results equal fp8ds_cast's, with no reset kernel
 * launched before the cast.
 */
int fp8ds_cast_acc(const void* x, fp8ds_dtype xt, int64_t rows, int64_t cols, fp8ds_format fmt,
                   const float* scale, uint8_t* q, uint8_t* q_t, float* scale_used, float* amax,
                   uint64_t* sat_count, hipStream_t stream);

/*
 * fp8ds_cast_health -- fp8ds_cast plus quantization-health counts of the same pass.
 * [P3] "第四步：建立 Amax 与低精度异常画像" (per-module metrics: the share of values
 * near the FP8 upper limit, the share of zeros after quantization, NaN / Inf /
 * overflow counts); [P2] §七 "陷阱 1：NaN/Inf 难以定位" (NaN and Inf checks).
 *
 * Arguments as fp8ds_cast, with sat_count replaced by
 *   counts     device, FP8DS_HEALTH_COUNTS uint64 (required), reset by the call:
 *              [0] saturated: #{|fl32(x*scale)| > max} (infinities counted, NaN not)
 *              [1] NaN inputs
 *              [2] infinite inputs
 *              [3] zero codes: q[i] is +-0 (underflow to zero and exact zeros)
 *              [4] near-max codes: q[i] finite with magnitude in the format's top
 *                  binade [2^emax, max] ([256, 448] E4M3, [32768, 57344] E5M2).
 */
#define FP8DS_HEALTH_COUNTS 5
int fp8ds_cast_health(const void* x, fp8ds_dtype xt, int64_t rows, int64_t cols, fp8ds_format fmt,
                      const float* scale, uint8_t* q, uint8_t* q_t, float* scale_used, float* amax,
                      uint64_t* counts, hipStream_t stream);

/*
 * fp8ds_cast_batched -- `batch` independent casts of equal size n, each with its
 * own scale (the per-problem scales of a batch of small Linears).
 * [P3] §适用场景 (among the cases to treat with care: many small matrices) and
 * §常见误区 误区一 (small matrices, frequent casts and scale kernels can eat the FP8
 * gain): one launch casts every tensor of the batch, so a small matrix's cast
 * costs no launch of its own.  Each tensor's cast is the scaled saturating cast
 * of fp8ds_cast ([P2] §四 "动态缩放", the quantize step).
 *
 *   x          device, batch tensors of n elements, tensor b at x + b*stride_x elements
 *              (stride_x >= n, stride_x*elem_size a multiple of 16).
 *   scale      device [batch].
 *   q          device, tensor b at q + b*stride_q bytes (stride_q >= n, multiple of 16).
 *   scale_used, amax: device [batch] or NULL.   sat_count: device [batch] or NULL.
 * Semantics per tensor as fp8ds_cast without the transposed copy.
 */
int fp8ds_cast_batched(const void* x, fp8ds_dtype xt, int64_t batch, int64_t n, int64_t stride_x,
                       fp8ds_format fmt, const float* scale, uint8_t* q, int64_t stride_q,
                       float* scale_used, float* amax, uint64_t* sat_count, hipStream_t stream);

/*
 * fp8ds_scale_update -- push this step's amax into each tensor's history ring and
 * compute the scale of the next step.
 * [P3] §核心原理 "Scale 决定数值是否进入可表示区间" (scale = (FP8_MAX/amax)/2^margin);
 * [P3] §核心原理 "Delayed Scaling 用历史换取稳定性" (history window, max or
 * most_recent); [P2] §四 "Delayed Scaling 的工程细节" (ring buffer with a cursor
 * advanced modulo the history length; scale 1.0 when the history maximum is not
 * positive).
 *
 * For each tensor t in [0, n_tensors):
 *   history[t*hist_len + cursor[t]] = amax[t];  cursor[t] = (cursor[t] + 1) % hist_len;
 *   w = max over history[t*hist_len .. +hist_len)  (ALGO_MAX; NaN propagates)
 *     | amax[t]                                       (ALGO_MOST_RECENT);
 *   scale[t] = ldexp(fl32(FP8_MAX(fmt[t]) / w), -margin)   if w is finite and > 0 and
 *              the result is finite and > 0;   1.0 otherwise.
 * The quotient is one correctly rounded fp32 division.
 *
 *   n_tensors  1 .. 4096.          hist_len  1 .. 65536.
 *   history    device [n_tensors][hist_len] fp32, in/out (initially zeros).
 *   cursor     device [n_tensors] int32, in/out (initially 0; must be in [0, hist_len)).
 *   amax       device [n_tensors] fp32 (e.g. the amax outputs of fp8ds_cast).
 *   fmt        HOST [n_tensors] fp8ds_format, read during the call only.
 *   algo       window reduction.       margin  integer exponent, -126..126.
 *   scale      device [n_tensors] fp32, overwritten with the next step's scale.
 *   scale_inv  device [n_tensors] or NULL: receives fl32(1 / scale).
 */
int fp8ds_scale_update(int n_tensors, int hist_len, float* history, int32_t* cursor,
                       const float* amax, const fp8ds_format* fmt, fp8ds_algo algo, int margin,
                       float* scale, float* scale_inv, hipStream_t stream);

/*
 * fp8ds_scale_update_clear -- fp8ds_scale_update that also zeroes `clear_bytes`
 * bytes at `clear` (device, 4-byte aligned, a multiple of 4 bytes up to 2^30)
 * in the same launch: the accumulators that the next step's fp8ds_cast_acc and
 * fp8ds_gemm_acc calls combine into.  The cleared bytes must not overlap the
 * other arguments (an overlap with amax returns FP8DS_ERR_VALUE); clear may be
 * NULL when clear_bytes is 0.
 */
int fp8ds_scale_update_clear(int n_tensors, int hist_len, float* history, int32_t* cursor,
                             const float* amax, const fp8ds_format* fmt, fp8ds_algo algo,
                             int margin, float* scale, float* scale_inv, void* clear,
                             int64_t clear_bytes, hipStream_t stream);

/*
 * fp8ds_gemm -- C = dequant( op(A) . op(B) ), FP8 x FP8 with FP32 accumulation.
 * [P2] §五 (the fp8 linear op: FP8 product divided by the product of the two
 * scales; the per-tensor FP8 GEMM: FP8 inputs, FP32 accumulate, BF16 output);
 * [P2] §三 (the three products of a training step: Y = X W, dX = dY W^T,
 * dW = X^T dY; HYBRID formats per [P3] §核心原理: E4M3 forward, E5M2 gradients).
 *
 *   acc[i][j] = sum_k a(i,k) * b(k,j)   over decoded FP8 values, FP32 accumulation
 *   C[i][j]   = convert_ct( acc[i][j] * d ),  d = fl32(1 / fl32((*scale_a) * (*scale_b)))
 * with round-to-nearest-even to BF16 (ct = BF16) or no rounding (ct = F32).
 *
 *   opa, opb   (N,N), (N,T) or (T,N); (T,T) returns FP8DS_ERR_UNSUPPORTED.
 *   M, N, K    >= 0 and < 2^31, with ceil(M/128) * ceil(N/128) < 2^31 (else
 *              FP8DS_ERR_SHAPE).  op(A) is M x K, op(B) is K x N, C is M x N.
 *   A          device: opa == N: [M x K] with lda >= K;  opa == T: [K x M] with lda >= M.
 *   B          device: opb == N: [K x N] with ldb >= N;  opb == T: [N x K] with ldb >= K.
 *   fa, fb     formats of A and B, independently E4M3 or E5M2.
 *   lda, ldb   multiples of 16 bytes; A and B 16-byte aligned.
 *   scale_a/b  device, 1 float each: the scale snapshots the operands were cast with.
 *   C          device [M x N] of `ct` with ldc >= N; C and ldc*elem_size 16-byte aligned.
 *   amax_c     device or NULL: receives max |C[i][j]| of the stored output (NaN as
 *              fp8ds_amax).
 *   mma        datapath (FP8DS_MMA_EXACT unless the caller accepts the FP8 matrix
 *              instructions' summation precision, see fp8ds_mma).
 */
int fp8ds_gemm(fp8ds_op opa, fp8ds_op opb, int64_t M, int64_t N, int64_t K,
               const uint8_t* A, fp8ds_format fa, int64_t lda, const float* scale_a,
               const uint8_t* B, fp8ds_format fb, int64_t ldb, const float* scale_b,
               void* C, fp8ds_dtype ct, int64_t ldc, float* amax_c, fp8ds_mma mma,
               hipStream_t stream);

/*
 * fp8ds_gemm_acc -- fp8ds_gemm whose output amax is combined into amax_c
 * (max(previous, max|C|)) instead of reset; otherwise identical.
 */
int fp8ds_gemm_acc(fp8ds_op opa, fp8ds_op opb, int64_t M, int64_t N, int64_t K,
                   const uint8_t* A, fp8ds_format fa, int64_t lda, const float* scale_a,
                   const uint8_t* B, fp8ds_format fb, int64_t ldb, const float* scale_b,
                   void* C, fp8ds_dtype ct, int64_t ldc, float* amax_c, fp8ds_mma mma,
                   hipStream_t stream);

/*
 * fp8ds_gemm_batched -- `batch` independent GEMMs of one shape, each with its own
 * scales and output amax (many small Linears in one launch).
 * [P3] §适用场景 (many small matrices among the cases to treat with care) and
 * §常见误区 误区一 (small matrices can cancel the FP8 gain): the products of a
 * batch of small Linears share one launch, one workgroup per output tile of any
 * problem.  Each product is fp8ds_gemm's ([P2] §五).
 * Problem b uses A + b*stride_a, B + b*stride_b (bytes), C + b*stride_c (elements),
 * scale_a[b], scale_b[b], amax_c[b]; otherwise as fp8ds_gemm.  Strides must keep
 * every operand 16-byte aligned.
 */
int fp8ds_gemm_batched(fp8ds_op opa, fp8ds_op opb, int64_t M, int64_t N, int64_t K, int64_t batch,
                       const uint8_t* A, fp8ds_format fa, int64_t lda, int64_t stride_a,
                       const float* scale_a, const uint8_t* B, fp8ds_format fb, int64_t ldb,
                       int64_t stride_b, const float* scale_b, void* C, fp8ds_dtype ct,
                       int64_t ldc, int64_t stride_c, float* amax_c, fp8ds_mma mma,
                       hipStream_t stream);

/*
 * fp8ds_linear_batched -- the whole forward step of `batch` independent small
 * Linears Y_i = X_i W_i, each with its own delayed scaling of X_i and W_i, in one
 * launch.  [P3] §适用场景 (many small matrices among the cases to treat with care)
 * and §常见误区 误区一 (with small matrices the conversion work can cancel the
 * FP8 gain): one workgroup per problem reads X_i and W_i once, casts them, keeps
 * the codes on chip for the product and updates both tensors' scaling state, so
 * the codes are never read back and no other launch is needed.
 *
 * Per problem i (tensor t = i is X_i, tensor t = batch + i is W_i):
 *   xq_i = cast(X_i, scale[i]), wq_i = cast(W_i, scale[batch + i])   (fp8ds_cast)
 *   y_i  = fp8ds_gemm(N, N) of xq_i and wq_i with those scales, BF16, amax_y[i]
 *   then for both tensors, with this step's amax: fp8ds_scale_update
 * The results equal those of fp8ds_cast_batched (X, then W), fp8ds_gemm_batched
 * (exact datapath) and fp8ds_scale_update over the 2 * batch tensors, in that
 * order; the outputs amax, sat_count, amax_y are stored, not combined into.
 *
 *   batch            1 .. 65535 problems
 *   M, N, K          multiples of 16 in [16, 256]
 *   x                [batch][M][K] BF16 (problem i at x + i*stride_x elements)
 *   w                [batch][K][N] BF16 (at w + i*stride_w elements)
 *   fx, fw           formats of the X and W codes
 *   hist_len, history, cursor, algo, margin: as fp8ds_scale_update, over the
 *                    2 * batch tensors ([2 batch][hist_len], [2 batch])
 *   scale            [2 batch] in: this step's scales; out: the next step's
 *   scale_used       [2 batch] (nullable): this step's scales
 *   amax             [2 batch] out: max |X_i|, then max |W_i| (NaN canonical)
 *   sat_count        [2 batch] (nullable) out: saturated values of each cast
 *   xq, wq           (nullable) codes: [batch][M][K] at stride_xq bytes,
 *                    [batch][K][N] at stride_wq bytes
 *   y                [batch][M][N] BF16 at stride_y elements
 *   amax_y           [batch] (nullable) out: max |y_i|
 * Every pointer 16-byte aligned, every stride a multiple of 16 bytes, strides at
 * least the problem's size.  Only the BF16 input dtype is supported
 * (FP8DS_ERR_UNSUPPORTED otherwise); the products run on the exact datapath.
 */
int fp8ds_linear_batched(int64_t batch, int64_t M, int64_t N, int64_t K, fp8ds_dtype xt,
                         const void* x, int64_t stride_x, fp8ds_format fx, const void* w,
                         int64_t stride_w, fp8ds_format fw, int hist_len, float* history,
                         int32_t* cursor, fp8ds_algo algo, int margin, float* scale,
                         float* scale_used, float* amax, uint64_t* sat_count, uint8_t* xq,
                         int64_t stride_xq, uint8_t* wq, int64_t stride_wq, void* y,
                         int64_t stride_y, float* amax_y, hipStream_t stream);

/*
 * fp8ds_adamw -- fused AdamW step on FP32 master weights that also writes the
 * FP8 copy of the updated weights for the next forward.
 * "算子与编译器：FP8 训练与优化器 Kernel" (charles2530.github.io): §"FP8 训练主路径图"
 * (unscale/clip -> fused optimizer -> master weight -> cast/scale to FP8) and
 * §"Fused Optimizer 的意义" (one kernel reads the gradient, updates both moments,
 * applies the bias corrections and the weight decay, updates the parameter);
 * [P2] §"自动混合精度与 FP8 的协同" (gradient un-scaling, FP32 AdamW, the updated
 * weights cast to FP8 with scaling for the next forward).
 *
 * The pages name AdamW without its formula; this is AdamW with decoupled weight
 * decay (Loshchilov & Hutter) and bias-corrected moments (Kingma & Ba).  Per
 * element, each operation one correctly rounded fp32 operation in this order,
 * no fused multiply-add:
 *   g' = g * grad_scale
 *   m  = beta1 * m + (1 - beta1) * g'
 *   v  = beta2 * v + ((1 - beta2) * g') * g'
 *   w  = decay * w - step_size * (m / (sqrt(v) * inv_sqrt_bc2 + eps))
 * with the fp32 constants decay = 1 - lr*weight_decay, 1 - beta1, 1 - beta2,
 * step_size = lr / (1 - beta1^step), inv_sqrt_bc2 = 1 / sqrt(1 - beta2^step),
 * each evaluated in float64 (C library pow and sqrt) and rounded once.
 * If scale != NULL, the updated weights are then cast exactly as fp8ds_cast
 * casts them (q, q_t, scale_used, amax, sat_count with fp8ds_cast's meaning, amax
 * and saturation of the NEW weights), so the next forward needs no weight cast.
 *
 *   w          device [rows x cols] fp32 master weights, row-major, updated in place.
 *   g          device [rows x cols] gradient of dtype gt (BF16 or FP32), read only.
 *   m, v       device [rows x cols] fp32 first and second moments, updated in
 *              place (zeros before the first step).  w, g, m, v must not overlap.
 *   rows,cols  >= 0.  All of w, g, m, v, q, q_t 16-byte aligned.
 *   lr, weight_decay  finite.   beta1, beta2  in [0, 1).   eps  finite, > 0.
 *   grad_scale finite, > 0: multiplies the gradient first (1/K for a loss
 *              scaled by K, times any clipping factor the caller computed).
 *   step       the step count t >= 1 of this update (bias corrections).
 *   grad_amax  device or NULL: if it holds an infinity or NaN (e.g. the amax_c of
 *              the fp8ds_gemm that produced g), the update is skipped -- w, m, v
 *              are left unchanged -- and the FP8 copy is made of the unchanged w.
 *   scale      device or NULL: the delayed scale of the weights.  NULL = no FP8
 *              copy (then q, q_t, scale_used, amax and sat_count must be NULL).
 *   fmt        FP8 format of the copy (checked when scale != NULL).
 *   q          device, rows*cols bytes (required with scale when rows*cols > 0): the
 *              FP8 copy of the new weights.
 *   q_t        device or NULL: the transposed copy [cols x rows]; rows at most
 *              65535 * 128 (cols at most 2^31 - 128).
 *   scale_used, amax, sat_count  device or NULL: as fp8ds_cast (written also when
 *              rows*cols == 0).
 * Out-of-range scalars return FP8DS_ERR_VALUE.
 */
int fp8ds_adamw(float* w, const void* g, fp8ds_dtype gt, float* m, float* v, int64_t rows,
                int64_t cols, float lr, float beta1, float beta2, float eps, float weight_decay,
                float grad_scale, int64_t step, const float* grad_amax, fp8ds_format fmt,
                const float* scale, uint8_t* q, uint8_t* q_t, float* scale_used, float* amax,
                uint64_t* sat_count, hipStream_t stream);

/*
 * Finer-grained scaling: current (just-in-time) scales and one scale per row.
 * [P2] §"FBGEMM_GPU 底层优化" (per-tensor, per-channel and per-token FP8 GEMM modes:
 * FP8 operands, FP32 accumulation, BF16 output); the scale formula of [P3]
 * §核心原理 "Scale 决定数值是否进入可表示区间" applied to the amax of what is being
 * cast, with no history ([P3]'s reference list names current scaling beside
 * delayed scaling).  In every case
 *   s = ldexp(fl32(FP8_MAX(fmt) / a), -margin)  if a and the result are finite and
 *       > 0, else 1.0;        scale_inv = fl32(1 / s)
 * with a the amax of the tensor (current) or of the row (per row).
 */

/*
 * fp8ds_cast_rowwise -- per-row current scaling of a [rows x cols] matrix:
 *   a_r = max_c |x[r][c]|,  s_r from a_r as above,  q[r][c] = encode(fl32(x[r][c] * s_r)).
 * Per-token scaling of activations X [M x K] is this call on X; per-channel
 * scaling of a weight W [K x N] (a scale per output channel) is this call on
 * W^T [N x K], the K-contiguous layout the forward GEMM reads with op T.
 *
 *   x          device, rows*cols elements of `xt`, row-major, 16-byte aligned.
 *   rows       0 .. 2^31 - 1.   cols >= 0.
 *   margin     integer exponent, -126..126.
 *   q          device, rows*cols bytes, 16-byte aligned.
 *   scale      device [rows] fp32 (required when rows > 0).
 *   scale_inv  device [rows] or NULL: fl32(1 / scale[r]) -- the GEMM's row/column factors.
 *   amax       device [rows] or NULL: a_r (NaN as fp8ds_amax).
 */
int fp8ds_cast_rowwise(const void* x, fp8ds_dtype xt, int64_t rows, int64_t cols, fp8ds_format fmt,
                       int margin, uint8_t* q, float* scale, float* scale_inv, float* amax,
                       hipStream_t stream);

/*
 * fp8ds_cast_current -- per-tensor current scaling: the amax of x, the scale from
 * it, then fp8ds_cast with that scale (three passes: amax, scale, cast).
 *
 *   x, xt, rows, cols, fmt, q, q_t  as fp8ds_cast.    margin  -126..126.
 *   scale      device, 1 float (required): receives s.
 *   scale_inv  device or NULL: receives fl32(1 / s).
 *   amax       device, 1 float (required): receives the amax of x.
 *   sat_count  device or NULL: as fp8ds_cast (non-zero only for margin < 0).
 */
int fp8ds_cast_current(const void* x, fp8ds_dtype xt, int64_t rows, int64_t cols,
                       fp8ds_format fmt, int margin, uint8_t* q, uint8_t* q_t, float* scale,
                       float* scale_inv, float* amax, uint64_t* sat_count, hipStream_t stream);

/*
 * fp8ds_gemm_rowcol -- fp8ds_gemm with one scale per row of op(A) and per column
 * of op(B) (per-token x per-channel), exact datapath:
 *   C[i][j] = convert_ct( fl32( fl32(acc[i][j] * scale_inv_a[i]) * scale_inv_b[j] ) )
 * with acc as fp8ds_gemm (FP32 accumulation of the decoded FP8 products).
 *
 *   scale_inv_a  device [M] fp32: inverse scale of each row of op(A) (e.g. the
 *                scale_inv of fp8ds_cast_rowwise on X).
 *   scale_inv_b  device [N] fp32, 16-byte aligned: inverse scale of each column of
 *                op(B) (e.g. fp8ds_cast_rowwise on W^T).  A per-tensor scale is
 *                passed as a vector of equal values.
 *   Other arguments as fp8ds_gemm (no batch, no datapath choice).
 * A scale that varies along K cannot be taken out of the sum: the products whose
 * contraction runs along the scaled dimension need operands cast in the other
 * orientation.
 */
int fp8ds_gemm_rowcol(fp8ds_op opa, fp8ds_op opb, int64_t M, int64_t N, int64_t K,
                      const uint8_t* A, fp8ds_format fa, int64_t lda, const float* scale_inv_a,
                      const uint8_t* B, fp8ds_format fb, int64_t ldb, const float* scale_inv_b,
                      void* C, fp8ds_dtype ct, int64_t ldc, float* amax_c, hipStream_t stream);

/*
 * MXFP8: FP8 elements in blocks of 32 consecutive elements along a row (the
 * contraction dimension of the GEMM below), each block with one E8M0 scale.
 * [P2] §九 "展望：Blackwell 的 Microscaling 与未来" (32 FP8 values share an 8-bit
 * E8M0 scale, scaled block by block); the block rule, which that figure leaves
 * garbled, is the OCP Microscaling Formats (MX) specification's:
 *   a = max |x_i| over the block;   E8M0 code = floor(log2 a) - emax + 127,
 *   clamped to [0, 254] (emax = 8 for E4M3, 15 for E5M2; a zero block has code 0);
 *   q_i = encode(x_i / 2^(code - 127)), saturating round-to-nearest-even.
 * A block holding a NaN or an infinity gets code 255 (NaN) and the element code
 * 0x7F (NaN) throughout.  The value of element i is 2^(code - 127) * decode(q_i).
 */

/*
 * fp8ds_cast_mx -- MXFP8 quantization of a [rows x cols] matrix along its rows,
 * optionally also of its transpose, from one read of x.
 *
 *   x          device, rows*cols elements of `xt`, row-major, 16-byte aligned.
 *   cols       a multiple of 32 (else FP8DS_ERR_SHAPE).
 *   q          device, rows*cols bytes, 16-byte aligned: the element codes.
 *   scales     device, rows*cols/32 bytes: the E8M0 code of block b of row r at
 *              [r * cols/32 + b].
 *   q_t        device or NULL: [cols x rows] codes of x^T quantized along its rows
 *              (blocks of 32 consecutive rows of a column of x), 16-byte aligned;
 *              requires rows and cols to be multiples of 128 (else FP8DS_ERR_SHAPE).
 *   scales_t   device [cols x rows/32] E8M0 codes of q_t; NULL exactly when q_t is.
 * The GEMMs of a training step all run as fp8ds_gemm_mx (A B^T, both blocked
 * along K): Y = X W takes (q of X, q_t of W); dX = dY W^T takes (q of dY, q of W);
 * dW = X^T dY takes (q_t of X, q_t of dY).  No amax, scale state or history is
 * involved.
 */
int fp8ds_cast_mx(const void* x, fp8ds_dtype xt, int64_t rows, int64_t cols, fp8ds_format fmt,
                  uint8_t* q, uint8_t* scales, uint8_t* q_t, uint8_t* scales_t,
                  hipStream_t stream);

/*
 * fp8ds_gemm_mx -- MXFP8 GEMM  C = A B^T  with FP32 accumulation:
 *   C[i][j] = convert_ct( sum_k X_a(i, k/32) a(i,k) X_b(j, k/32) b(j,k) )
 * with a, b the decoded element codes and X the block scales.  Exact datapath:
 * every element is widened to BF16 times its block scale (exact while the scaled
 * value is a normal BF16 number, i.e. |X * decode| >= 2^-126, or zero: blocks whose
 * scale code is above about 17) and multiplied on the BF16 matrix cores with
 * FP32 sums; a NaN block makes every output it touches NaN.
 *
 *   A          device [M x K] codes (K-contiguous, leading dimension lda), format fa.
 *   scales_a   device [M x ld_scales_a] E8M0 codes; block b of row i at
 *              [i * ld_scales_a + b] (fp8ds_cast_mx of A writes ld = K/32).
 *   B          device [N x K] codes (leading dimension ldb), format fb; for a
 *              Linear Y = X W with W [K x N], B is the MX cast of W^T.
 *   scales_b   device [N x ld_scales_b] E8M0 codes.
 *   C          device [M x ldc], BF16 or FP32 (ct).   amax_c  device or NULL: max |C|.
 *   K          a multiple of 128 (four blocks per pipeline stage), else FP8DS_ERR_SHAPE.
 *   A, B, C, lda, ldb, ldc * element size: 16-byte aligned; the scale arrays and
 *   ld_scales_a / ld_scales_b: 4-byte aligned (FP8DS_ERR_ALIGN otherwise).
 *   mma        FP8DS_MMA_EXACT (the BF16 widening above, default) or FP8DS_MMA_FP8:
 *              gfx950's block-scaled FP8 matrix instruction, each lane passing the
 *              E8M0 scale of its 32 K values, at twice the rate and with the FP8
 *              instructions' summation precision (see fp8ds_mma).
 */
int fp8ds_gemm_mx(int64_t M, int64_t N, int64_t K, const uint8_t* A, fp8ds_format fa, int64_t lda,
                  const uint8_t* scales_a, int64_t ld_scales_a, const uint8_t* B, fp8ds_format fb,
                  int64_t ldb, const uint8_t* scales_b, int64_t ld_scales_b, void* C,
                  fp8ds_dtype ct, int64_t ldc, float* amax_c, fp8ds_mma mma, hipStream_t stream);

/*
 * RMSNorm with the residual's addition and a quantised output.  Per row:
 *   h = x + residual   rounded to ht (the residual stream's type); h = x without residual
 *   r = 1 / sqrt(sum_c h[c]^2 / cols + eps)          fp32 sums
 *   y[c] = (h[c] * r) * gamma[c]                     fp32, from the rounded h
 * and y, in fp32, is cast as the call says: the operand of the next product, with no
 * 16-bit copy of y in between.  (Squares are fp32: |h| above 1e18 overflows them.)
 *
 * Arguments of the three calls:
 *   x          device [rows x cols] of xt, rows ldx elements apart.
 *   residual   device or NULL: [rows x cols] of ht, ldr apart.
 *   gamma      device [cols] of gt.
 *   eps        finite, >= 0.
 *   h          device or NULL: [rows x cols] of ht, ldh apart: the new residual stream.
 *              May be residual or x itself (same type, same leading dimension).
 *   y          device or NULL: [rows x cols] of yt, ldy apart.
 *   rstd       device or NULL: [rows], r (for the backward pass).
 *   rows, cols >= 0 and < 2^31; any cols (fp8ds_rmsnorm_mx: a multiple of 32).  Leading
 *              dimensions at least cols.  Matrices aligned to their elements; fastest
 *              with 16-byte aligned rows (8 bytes for q) and cols a multiple of 8.
 *   (xt, ht)   (BF16, BF16), (BF16, F32) or (F32, F32); (F32, BF16) is
 *              FP8DS_ERR_UNSUPPORTED.
 * No rows or no columns: nothing but *scale_used is written.
 */

/*
 * fp8ds_rmsnorm -- y and / or its FP8 copy with a given per-tensor scale, as
 * fp8ds_cast_acc casts: q = encode(y * (*scale)), amax and sat_count are COMBINED INTO
 * (max / add; zero them first, fp8ds_scale_update_clear does), scale_used is written.
 * scale NULL: no FP8 copy, then q, scale_used, amax and sat_count must be NULL.
 *   q          device [rows x cols] bytes, rows ldq apart.
 */
int fp8ds_rmsnorm(const void* x, fp8ds_dtype xt, int64_t ldx, const void* residual, int64_t ldr,
                  fp8ds_dtype ht, const void* gamma, fp8ds_dtype gt, int64_t rows, int64_t cols,
                  float eps, void* h, int64_t ldh, void* y, fp8ds_dtype yt, int64_t ldy,
                  float* rstd, fp8ds_format fmt, const float* scale, uint8_t* q, int64_t ldq,
                  float* scale_used, float* amax, uint64_t* sat_count, hipStream_t stream);

/*
 * fp8ds_rmsnorm_rowwise -- the FP8 copy with a scale per row, as fp8ds_cast_rowwise
 * casts: scale, scale_inv (or NULL) and amax (or NULL) are [rows], overwritten.
 */
int fp8ds_rmsnorm_rowwise(const void* x, fp8ds_dtype xt, int64_t ldx, const void* residual,
                          int64_t ldr, fp8ds_dtype ht, const void* gamma, fp8ds_dtype gt,
                          int64_t rows, int64_t cols, float eps, void* h, int64_t ldh, void* y,
                          fp8ds_dtype yt, int64_t ldy, float* rstd, fp8ds_format fmt, int margin,
                          uint8_t* q, int64_t ldq, float* scale, float* scale_inv, float* amax,
                          hipStream_t stream);

/*
 * fp8ds_rmsnorm_mx -- the copy in blocks of 32 with E8M0 scales, as fp8ds_cast_mx (E4M3,
 * E5M2) or fp8ds_cast_mxfp4 (E2M1: two elements per byte) casts.
 *   q          device [rows], ldq bytes apart (at least cols, E2M1: cols / 2).
 *   scales     device [rows x cols / 32], rows ld_scales apart.
 * Every row of x, residual, h, y 16-byte aligned, gamma too, rows of q 8-byte aligned
 * (FP8DS_ERR_ALIGN otherwise).
 */
int fp8ds_rmsnorm_mx(const void* x, fp8ds_dtype xt, int64_t ldx, const void* residual, int64_t ldr,
                     fp8ds_dtype ht, const void* gamma, fp8ds_dtype gt, int64_t rows, int64_t cols,
                     float eps, void* h, int64_t ldh, void* y, fp8ds_dtype yt, int64_t ldy,
                     float* rstd, fp8ds_format fmt, uint8_t* q, int64_t ldq, uint8_t* scales,
                     int64_t ld_scales, hipStream_t stream);

/*
 * fp8ds_rmsnorm_bwd -- backward of the norm.  With xhat = h r and g = dy gamma, per row
 *   dx     = r (g - xhat * (sum_c g xhat) / cols) + dres
 *   dgamma = sum over rows of dy xhat
 * dx is the gradient of x and of residual; dres is the gradient that reaches h from above.
 *   dy         device [rows x cols] of dt, lddy apart.
 *   h          device [rows x cols] of ht, ldh apart: what the forward stored (or its x).
 *   rstd       device [rows]: what the forward stored.
 *   gamma      device [cols] of gt.
 *   dres       device or NULL: [rows x cols] of ht, lddr apart.
 *   dx         device [rows x cols] of ht, lddx apart.  May be dres, or dy (same type and
 *              leading dimension).
 *   dgamma     device [cols] fp32, overwritten (zeros for rows == 0).
 *   workspace  device, at least fp8ds_rmsnorm_bwd_workspace(rows, cols) bytes, 16-byte
 *              aligned; its contents need no preparation and do not matter afterwards.
 *   scale      device or NULL: with it dx, in fp32, is also cast to FP8 as fp8ds_rmsnorm
 *              casts y (fmt, q, ldq, scale_used, amax, sat_count): the dY operand of the
 *              products below.
 * (dt, ht) as (xt, ht) above.  Sums are fp32, in an order fixed by the shape.
 */
int64_t fp8ds_rmsnorm_bwd_workspace(int64_t rows, int64_t cols);
int fp8ds_rmsnorm_bwd(const void* dy, fp8ds_dtype dt, int64_t lddy, const void* h, fp8ds_dtype ht,
                      int64_t ldh, const float* rstd, const void* gamma, fp8ds_dtype gt,
                      const void* dres, int64_t lddr, int64_t rows, int64_t cols, void* dx,
                      int64_t lddx, float* dgamma, void* workspace, int64_t workspace_bytes,
                      fp8ds_format fmt, const float* scale, uint8_t* q, int64_t ldq,
                      float* scale_used, float* amax, uint64_t* sat_count, hipStream_t stream);

/*
 * fp8ds_grad_norm -- global norm of n_tensors gradients and the clipping coefficient:
 *   norm = grad_scale * sqrt(sum over all elements of g^2)     sums in 64 bits
 *   coef = min(1, max_norm / (norm + 1e-6))
 * An infinite norm gives coef 0, NaN gives NaN: hand `norm` to fp8ds_adamw_clip as
 * grad_amax and such a step is skipped.
 *   grads      HOST array of device addresses (each aligned to its elements), types and
 *              counts HOST arrays; read during the call only.  0 to 4096 tensors, of any
 *              size (0 included; its address may be NULL), 2^40 elements at most.
 *   grad_scale finite, > 0: the un-scaling that the optimizer applies (its grad_scale).
 *   max_norm   > 0 (may be infinite); unused if coef is NULL.
 *   norm, coef device, 1 float each (coef or NULL).
 *   workspace  device, fp8ds_grad_norm_workspace() bytes, 16-byte aligned, needing no
 *              preparation; may be NULL for up to 65536 elements in up to 128 tensors.
 */
int64_t fp8ds_grad_norm_workspace(void);
int fp8ds_grad_norm(int n_tensors, const void* const* grads, const fp8ds_dtype* types,
                    const int64_t* counts, float grad_scale, float max_norm, float* norm,
                    float* coef, void* workspace, int64_t workspace_bytes, hipStream_t stream);

/*
 * fp8ds_grad_clip -- out_t[i] = grads_t[i] * (*coef), an fp32 product rounded to out's
 * type.  out NULL: in place (nothing is touched if *coef is 1).  out_t may be grads_t
 * (same type) and must not overlap it otherwise.  Arrays as fp8ds_grad_norm.
 */
int fp8ds_grad_clip(int n_tensors, const void* const* grads, const fp8ds_dtype* types,
                    const int64_t* counts, void* const* out, const fp8ds_dtype* out_types,
                    const float* coef, hipStream_t stream);

/*
 * fp8ds_adamw_clip -- fp8ds_adamw whose gradient is also multiplied by a device factor
 * (fp8ds_grad_norm's coef): g' = g * fl32(grad_scale * (*grad_coef)); otherwise identical.
 * Clipping then costs no pass over the gradients and no synchronisation.
 */
int fp8ds_adamw_clip(float* w, const void* g, fp8ds_dtype gt, float* m, float* v, int64_t rows,
                     int64_t cols, float lr, float beta1, float beta2, float eps,
                     float weight_decay, float grad_scale, const float* grad_coef, int64_t step,
                     const float* grad_amax, fp8ds_format fmt, const float* scale, uint8_t* q,
                     uint8_t* q_t, float* scale_used, float* amax, uint64_t* sat_count,
                     hipStream_t stream);

/*
 * fp8ds_cast_mxfp4 -- MXFP4 cast of a [rows x cols] matrix along its rows: blocks of 32
 * consecutive elements, E8M0 code floor(log2 amax) - 2 + 127 clamped to [0, 254] (0 for a
 * zero block, 255 for one that holds a NaN or infinity, whose elements are stored as 6),
 * elements round to nearest (ties to the even code), saturating at 6, sign kept.
 *   x          device [rows x cols] of xt, contiguous, 16-byte aligned; cols a multiple of 32.
 *   q          device [rows x cols / 2] bytes, 16-byte aligned: element 2 i in the low half.
 *   scales     device [rows x cols / 32].
 *   q_t, scales_t  device or both NULL: the transpose [cols x rows / 2], [cols x rows / 32],
 *              blocked along its own rows, from the same read; rows a multiple of 32, at
 *              most 128 * 65535, cols at most 2^31 - 128 (FP8DS_ERR_SHAPE otherwise).
 */
int fp8ds_cast_mxfp4(const void* x, fp8ds_dtype xt, int64_t rows, int64_t cols, uint8_t* q,
                     uint8_t* scales, uint8_t* q_t, uint8_t* scales_t, hipStream_t stream);

/*
 * fp8ds_dequant_mxfp4 -- the values y [rows x cols] of yt that MXFP4 codes stand for
 * (exact; NaN for a block with code 255).  q and y contiguous, 16-byte aligned.
 */
int fp8ds_dequant_mxfp4(const uint8_t* q, const uint8_t* scales, int64_t rows, int64_t cols,
                        void* y, fp8ds_dtype yt, hipStream_t stream);

/*
 * fp8ds_gemm_mxfp4 -- C = A B^T with B [N x K] in MXFP4 and A [M x K] in MXFP4 or MXFP8:
 *   C[i][j] = convert_ct( sum_k X_a(i, k/32) a(i,k) X_b(j, k/32) b(j,k) )
 * with exact products and FP32 sums.  MXFP4 x MXFP4 runs on gfx950's block-scaled matrix
 * instruction.  An FP8 A, whose products that instruction adds in fewer bits, is by default
 * widened with B to BF16 times the block scales, as fp8ds_gemm_mx widens its operands: exact
 * where the scaled values are normal BF16 numbers (or zero), i.e. for scale codes from 10 (A
 * E4M3) or 17 (E5M2) up to 246 or 239, and to 252 of B.  A NaN block makes every output that it
 * touches NaN.
 *   A, fa      E2M1 (two per byte), E4M3 or E5M2; rows lda ELEMENTS apart.
 *   scales_a   [M x ld_scales_a] E8M0 codes; scales_b [N x ld_scales_b].
 *   B          E2M1; rows ldb ELEMENTS apart.
 *   C          [M x ldc] of ct, aligned to its elements.   amax_c  device or NULL: max |C|.
 *   M, N       >= 0, any size (M <= 65535 * 64).   K  >= 0, a multiple of 32.
 *   Rows of A and B 16-byte aligned (lda a multiple of 32, of 16 for FP8; ldb of 32).
 */
int fp8ds_gemm_mxfp4(int64_t M, int64_t N, int64_t K, const uint8_t* A, fp8ds_format fa,
                     int64_t lda, const uint8_t* scales_a, int64_t ld_scales_a, const uint8_t* B,
                     int64_t ldb, const uint8_t* scales_b, int64_t ld_scales_b, void* C,
                     fp8ds_dtype ct, int64_t ldc, float* amax_c, hipStream_t stream);

/*
 * fp8ds_gemm_mxfp4_mma -- fp8ds_gemm_mxfp4 with the datapath of an FP8 A named:
 * FP8DS_MMA_EXACT (what fp8ds_gemm_mxfp4 takes), or FP8DS_MMA_FP8: the block-scaled FP8
 * instruction at up to twice the rate, with its summation precision (see fp8ds_mma).  An
 * MXFP4 A takes the same path for both.
 */
int fp8ds_gemm_mxfp4_mma(int64_t M, int64_t N, int64_t K, const uint8_t* A, fp8ds_format fa,
                         int64_t lda, const uint8_t* scales_a, int64_t ld_scales_a,
                         const uint8_t* B, int64_t ldb, const uint8_t* scales_b,
                         int64_t ld_scales_b, void* C, fp8ds_dtype ct, int64_t ldc, float* amax_c,
                         fp8ds_mma mma, hipStream_t stream);

/* Activations of a gated feed-forward block: SiLU g / (1 + e^-g), GELU in its tanh form
 * g (1 + tanh(sqrt(2 / pi) (g + 0.044715 g^3))) / 2. */
typedef enum { FP8DS_ACT_SILU = 0, FP8DS_ACT_GELU = 1 } fp8ds_act;

/*
 * fp8ds_gated_gemm -- gate and up projections of a feed-forward block, its activation and their
 * product in one kernel:
 *   g[i][j] = d sum_k a(i,k) b(j,k),  u[i][j] = d sum_k a(i,k) b(F+j,k),  d as fp8ds_gemm's
 *   y[i][j] = act(g[i][j]) u[i][j]                    fp32, from the fp32 sums
 * with y stored in 16 or 32 bits and / or cast to FP8 as fp8ds_cast_acc casts (q = encode(y *
 * (*scale)); amax, of |y|, and sat_count are COMBINED INTO): the operand of the down projection.
 *   A          device [M x K] codes, rows lda apart.   fa  E4M3.
 *   B          device [2F x K] codes, rows ldb apart: the gate's rows, then the up projection's
 *              (for weights stored [K x 2F] the transposed copy of their cast).   fb  E4M3.
 *   scale_a/b  device, 1 float each: the scale snapshots of the operands.
 *   gu         device or NULL: [M x 2F] BF16, rows ldgu apart: g, then u (for the backward pass).
 *   y          device or NULL: [M x F] of yt, rows ldy apart.
 *   scale      device or NULL (then q, scale_used and sat_count must be NULL): the delayed scale.
 *   q          device [M x F] codes of fmt, rows ldq apart.
 *   amax       device or NULL: of y, with or without a scale.
 *   mma        as fp8ds_gemm; up to 16 rows run exact either way.
 *   M, F, K    >= 0, any size (ceil(M/128) ceil(F/64) < 2^23).  Rows of A and B 16-byte aligned; gu
 *              and y aligned to their elements (fastest with rows at 16 bytes, F a multiple of 16).
 * At least one of gu, y and q.  Outputs must not overlap each other or the operands.  M or F of 0:
 * nothing but *scale_used is written.  Up to 16 rows read every weight once.
 */
int fp8ds_gated_gemm(int64_t M, int64_t F, int64_t K, const uint8_t* A, fp8ds_format fa, int64_t lda,
                     const float* scale_a, const uint8_t* B, fp8ds_format fb, int64_t ldb,
                     const float* scale_b, fp8ds_act act, void* gu, int64_t ldgu, void* y,
                     fp8ds_dtype yt, int64_t ldy, fp8ds_format fmt, const float* scale, uint8_t* q,
                     int64_t ldq, float* scale_used, float* amax, uint64_t* sat_count, fp8ds_mma mma,
                     hipStream_t stream);

/*
 * fp8ds_gated_gemm_bwd -- backward of the block through the down projection and the activation:
 *   da[i][j] = d sum_h a(i,h) b(j,h)
 *   dg = da u act'(g),   du = da act(g)               fp32, from the stored g and u
 *   A          device [M x H] codes of dY, E5M2 or E4M3.
 *   B          device [F x H] codes of the down projection as stored ([in, out]), E4M3.
 *   gu         device [M x 2F] BF16: what fp8ds_gated_gemm stored.
 *   dgu        device or NULL: [M x 2F] of dt, rows lddgu apart: dg, then du.
 *   q          device or NULL: the same in FP8 (E5M2 as a rule), rows ldq apart, with scale,
 *              scale_used, amax and sat_count as fp8ds_gated_gemm.  One scale for both halves, so
 *              dX = [dg du] W^T and dW = X^T [dg du] are single fp8ds_gemm calls.
 * Other arguments, sizes, alignment and mma as fp8ds_gated_gemm.  At least one of dgu and q; neither
 * may overlap gu.
 */
int fp8ds_gated_gemm_bwd(int64_t M, int64_t F, int64_t H, const uint8_t* A, fp8ds_format fa,
                         int64_t lda, const float* scale_a, const uint8_t* B, fp8ds_format fb,
                         int64_t ldb, const float* scale_b, fp8ds_act act, const void* gu,
                         int64_t ldgu, void* dgu, fp8ds_dtype dt, int64_t lddgu, fp8ds_format fmt,
                         const float* scale, uint8_t* q, int64_t ldq, float* scale_used, float* amax,
                         uint64_t* sat_count, fp8ds_mma mma, hipStream_t stream);

/*
 * The norms around a residual addition: the branch's output x is normalised, gated and added, the
 * new stream is normalised for the next block, and that is cast.  Per row
 *   r1 = 1 / sqrt(sum_c x[c]^2 / cols + post_eps)
 *   h[c] = residual[c] + t (x[c] r1) (alpha gate[c] post_gamma[c])    rounded to ht
 *   r2 = 1 / sqrt(sum_c h[c]^2 / cols + eps),   y[c] = (h[c] r2) gamma[c]
 * with h in 64 bits, rounded to fp32 and then to ht (rows of 8 to 16384 columns; others in fp32), the
 * rest in fp32, and y cast as fp8ds_rmsnorm, _rowwise and _mx cast theirs.
 *   x, residual, h, y, gamma, eps, rstd (r2) and the cast's arguments: as those calls; residual and
 *              h are required here.  h may be residual itself.
 *   post_gamma device [cols] of pt.          post_eps  finite, >= 0.
 *   gate       device or NULL: [cols] of gate_t, a factor per channel.
 *   row_gate   device or NULL: [rows], t, a factor per token (1 without it).
 *   alpha      finite: the residual scale.
 *   post_rstd  device or NULL: [rows], r1 (for the backward pass).
 * fp8ds_rmsnorm_sandwich_mx needs post_gamma and gate 16-byte aligned too.
 */
int fp8ds_rmsnorm_sandwich(const void* x, fp8ds_dtype xt, int64_t ldx, const void* post_gamma,
                           fp8ds_dtype pt, float post_eps, const void* gate, fp8ds_dtype gate_t,
                           const float* row_gate, float alpha, const void* residual, int64_t ldr,
                           fp8ds_dtype ht, const void* gamma, fp8ds_dtype gt, int64_t rows,
                           int64_t cols, float eps, void* h, int64_t ldh, void* y, fp8ds_dtype yt,
                           int64_t ldy, float* post_rstd, float* rstd, fp8ds_format fmt,
                           const float* scale, uint8_t* q, int64_t ldq, float* scale_used, float* amax,
                           uint64_t* sat_count, hipStream_t stream);
int fp8ds_rmsnorm_sandwich_rowwise(const void* x, fp8ds_dtype xt, int64_t ldx, const void* post_gamma,
                                   fp8ds_dtype pt, float post_eps, const void* gate,
                                   fp8ds_dtype gate_t, const float* row_gate, float alpha,
                                   const void* residual, int64_t ldr, fp8ds_dtype ht,
                                   const void* gamma, fp8ds_dtype gt, int64_t rows, int64_t cols,
                                   float eps, void* h, int64_t ldh, void* y, fp8ds_dtype yt,
                                   int64_t ldy, float* post_rstd, float* rstd, fp8ds_format fmt,
                                   int margin, uint8_t* q, int64_t ldq, float* scale, float* scale_inv,
                                   float* amax, hipStream_t stream);
int fp8ds_rmsnorm_sandwich_mx(const void* x, fp8ds_dtype xt, int64_t ldx, const void* post_gamma,
                              fp8ds_dtype pt, float post_eps, const void* gate, fp8ds_dtype gate_t,
                              const float* row_gate, float alpha, const void* residual, int64_t ldr,
                              fp8ds_dtype ht, const void* gamma, fp8ds_dtype gt, int64_t rows,
                              int64_t cols, float eps, void* h, int64_t ldh, void* y, fp8ds_dtype yt,
                              int64_t ldy, float* post_rstd, float* rstd, fp8ds_format fmt, uint8_t* q,
                              int64_t ldq, uint8_t* scales, int64_t ld_scales, hipStream_t stream);

/*
 * fp8ds_rmsnorm_sandwich_bwd -- backward of those.  With xh2 = h r2, g2 = dy gamma, xh1 = x r1,
 * k = alpha gate post_gamma, per row
 *   dh = r2 (g2 - xh2 (sum_c g2 xh2) / cols) + dres        the gradient of residual
 *   g1 = t k dh,   dx = r1 (g1 - xh1 (sum_c g1 xh1) / cols)     from the fp32 dh
 *   drow_gate = sum_c k dh xh1
 * and over the rows, with S = sum alpha t dh xh1:
 *   dgamma = sum dy xh2,   dpost_gamma = gate S,   dgate = post_gamma S
 *   dy         device [rows x cols] of xt.      h   device [rows x cols] of ht: what was stored.
 *   x          device [rows x cols] of xt.      rstd, post_rstd  device [rows]: what was stored.
 *   dres       device or NULL: [rows x cols] of ht, the gradient that reaches h from above.
 *   dh         device [rows x cols] of ht.  May be dres (same leading dimension).
 *   dx         device or NULL: [rows x cols] of xt.  May be dy (same leading dimension).
 *   dgamma, dpost_gamma  device [cols] fp32.    dgate  device or NULL: [cols] fp32.
 *   drow_gate  device or NULL: [rows] fp32.
 *   workspace  device, at least fp8ds_rmsnorm_sandwich_bwd_workspace(rows, cols) bytes, 16-byte
 *              aligned; its contents need no preparation and do not matter afterwards.
 *   scale      device or NULL: with it dx, in fp32, is also cast to FP8 (fmt, q, ldq, scale_used,
 *              amax, sat_count as fp8ds_rmsnorm_bwd).
 * (xt, ht) as fp8ds_rmsnorm.  Sums are fp32, in an order fixed by the shape.
 */
int64_t fp8ds_rmsnorm_sandwich_bwd_workspace(int64_t rows, int64_t cols);
int fp8ds_rmsnorm_sandwich_bwd(const void* dy, fp8ds_dtype xt, int64_t lddy, const void* h,
                               fp8ds_dtype ht, int64_t ldh, const float* rstd, const void* gamma,
                               fp8ds_dtype gt, const void* x, int64_t ldx, const float* post_rstd,
                               const void* post_gamma, fp8ds_dtype pt, const void* gate,
                               fp8ds_dtype gate_t, const float* row_gate, float alpha,
                               const void* dres, int64_t lddr, int64_t rows, int64_t cols, void* dh,
                               int64_t lddh, void* dx, int64_t lddx, float* dgamma, float* dpost_gamma,
                               float* dgate, float* drow_gate, void* workspace,
                               int64_t workspace_bytes, fp8ds_format fmt, const float* scale, uint8_t* q,
                               int64_t ldq, float* scale_used, float* amax, uint64_t* sat_count,
                               hipStream_t stream);

/*
 * fp8ds_muon_direction -- Muon's update of one matrix: momentum, then Newton-Schulz steps that bring
 * the update's singular values near 1.
 *   g' = g * fl32(grad_scale * (*grad_coef)),   m = mu m + g'
 *   U = g' + mu m (nesterov) or m;  U = g' without a momentum
 *   X = U / (|U|_F + eps)                 in 64 bits, rounded to fp32 once
 *   per step, with its own a, b, c:  A = X X^T,  X = a X + (b A + c A A) X
 *   o = X                                 (on the transpose where rows > cols)
 * m and U: each operation one fp32 rounding.  The products take their operands as pairs of F16 (22
 * significant bits; what is below 2^-39 of |U|_F is lost), three products of each, with fp32 sums: o
 * is up to 1e-5 (relative, of the whole matrix) from the iteration in 64 bits for Gaussian g, up to
 * 1e-4 where a few directions are far stronger than the rest or the singular values fall by orders of
 * magnitude, as the iteration in fp32 is.
 *   g          device [rows x cols] of gt, rows ldg apart (a part of a stacked gradient, say).
 *   momentum   device or NULL: [rows x cols] fp32, contiguous, updated in place (zeros before the
 *              first step).
 *   rows,cols  0 .. 2^19 each, 2^34 elements at most.    mu  in [0, 1).
 *   grad_scale finite, > 0.    grad_coef  device or NULL: a further factor (fp8ds_grad_norm's coef).
 *   grad_amax  device or NULL: if it holds an infinity or NaN (fp8ds_grad_norm's norm), momentum and o
 *              are left as they are.
 *   steps      1 .. FP8DS_MUON_MAX_STEPS (5 as a rule).
 *   coefs      HOST [steps][3] or NULL: a, b, c of each step, finite; NULL: 3.4445, -4.7750, 2.0315.
 *   eps        finite, > 0 (1e-7 as a rule).  A zero U gives a zero o.
 *   o          device [rows x cols] of ot, rows ldo apart; must not overlap the others.
 *   workspace  device, at least fp8ds_muon_workspace(rows, cols) bytes; its contents need no
 *              preparation and do not matter afterwards.  With either side rounded up to 64, 128 or 256
 *              (64 at least, no side to twice itself): 12 bytes for each element, 8 for each of
 *              min(rows, cols)^2, 20 where one side is 1.5 times the other or more, and up to
 *              4 MB of partial sums.
 * g and o aligned to their elements, momentum and workspace to 16 bytes.  No atomics: the same
 * inputs give the same bits.
 */
#define FP8DS_MUON_MAX_STEPS 16
int64_t fp8ds_muon_workspace(int64_t rows, int64_t cols);
int fp8ds_muon_direction(const void* g, fp8ds_dtype gt, int64_t ldg, float* momentum, int64_t rows,
                         int64_t cols, float mu, int nesterov, float grad_scale,
                         const float* grad_coef, const float* grad_amax, int steps,
                         const float* coefs, float eps, void* o, fp8ds_dtype ot, int64_t ldo,
                         void* workspace, int64_t workspace_bytes, hipStream_t stream);

/*
 * fp8ds_muon_apply -- the weights' step along a direction, and the FP8 copy of the new weights:
 *   w = decay w - step o,   decay = 1 - lr weight_decay,  step = lr adjust
 * each operation one fp32 rounding, decay and step in float64 and rounded once.  adjust is the
 * update's size for lr 1, e.g. 0.2 sqrt(max(rows, cols)) for updates of AdamW's size.  With a scale
 * the new weights are cast as fp8ds_adamw casts them, except that amax and sat_count are COMBINED
 * INTO, as fp8ds_cast_acc does.
 *   w          device [rows x cols] fp32, updated in place.     o  device [rows x cols] of ot.
 *   lr, weight_decay, adjust  finite.
 *   grad_amax  device or NULL: if not finite, w stays; the FP8 copy is made all the same.
 *   fmt, scale, q, q_t, scale_used, amax, sat_count  as fp8ds_adamw.
 * At most 2^35 elements; w, o, q and q_t contiguous and 16-byte aligned.
 */
int fp8ds_muon_apply(float* w, const void* o, fp8ds_dtype ot, int64_t rows, int64_t cols, float lr,
                     float weight_decay, float adjust, const float* grad_amax, fp8ds_format fmt,
                     const float* scale, uint8_t* q, uint8_t* q_t, float* scale_used, float* amax,
                     uint64_t* sat_count, hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* FP8DS_H */
