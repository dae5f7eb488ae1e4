/*
 * q8.h -- C ABI of libq8, the 8-bit quantized linear layer Y = X . W^T on one
 * AMD Instinct MI355X (gfx950).
 *
 * Pages cited (by title and section):
 *   [LF]   "8-Bit LLM Quantization with Lightning Fabric"
 *   [OV]   "大模型量化技术概述" (LLM quantization overview, devpress)
 *   [FB]   "Transformers FP8 (W8A8) 量化实战：基于 FBGEMM 的模型压缩与加载"
 *   [BNB]  "Transformers 单 GPU 高效推理：bitsandbytes LLM.int8 8-bit 混合精度量化的原理与实操"
 *   [NOTE] Xilyfe, "大模型量化" (lecture notes)
 *
 * Conventions shared by every call
 * --------------------------------
 * - Every tensor pointer is DEVICE memory owned by the caller.  The library
 *   never allocates, frees or keeps a pointer after a call returns.  Scratch
 *   space comes from a caller-provided workspace sized by q8_workspace_bytes
 *   (q8_linear_noalloc: from a fixed device array of the library).
 * - Tensors are dense, row-major, 2-D.  X is [M, K] (tokens x input features),
 *   W is [N, K] (output features x input features, K contiguous), Y is [M, N].
 *   A caller with batch dimensions flattens them into M first ([FB] §5.2: the
 *   input is viewed as 2-D) and reshapes Y back afterwards.
 * - `stream` is a hipStream_t passed as void* (NULL = the default stream).
 *   Calls only enqueue work on that stream and return; no call ever waits for
 *   the device, so results are valid once the stream has reached this point.
 *   The library keeps no state between calls apart from a per-device cache of
 *   the device check (and the scratch array of q8_linear_noalloc); calls on
 *   different streams may run concurrently (q8_linear_noalloc excepted).
 * - Every argument is checked on the host BEFORE anything is enqueued.  On a
 *   non-Q8_OK status nothing has been written.  Q8_ERR_LAUNCH reports a
 *   failed kernel launch (hipGetLastError) after validation passed.
 * - Empty batches: every call that takes activations accepts M = 0 (T = 0
 *   for q8_linear_fp8_grouped).  It checks its other arguments as usual; the
 *   pointers to M-sized arrays (x, codes, scales, code sums, y, acc_out) may
 *   then be NULL, no workspace is needed (q8_workspace_bytes returns 0), and
 *   nothing is enqueued or written, except that q8_linear_int8_decomp writes
 *   0 to n_outliers when it is given (the outlier set of no rows is empty).
 * - Preconditions checked for every call: M >= 0 and N, K >= 1 (weight
 *   quantization: N, K >= 1); K % 16 == 0;
 *   K <= 65536 (keeps the zero-point-corrected INT32 sums in range); every
 *   matrix (X, W, Y) has fewer than 2^31 elements; all pointers 16-byte
 *   aligned; the device running `stream` is gfx950.
 *   Inputs must be finite: NaN/Inf inputs give unspecified codes and outputs.
 * - Floating point follows IEEE binary32 with round-to-nearest-even; scales
 *   are computed with correctly rounded division, codes with x / S (not
 *   x * (1/S)); nothing is flushed to zero.
 */
#ifndef Q8_H
#define Q8_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum q8_status {
  Q8_OK = 0,
  Q8_ERR_NULL_PTR = 1,   /* a required pointer is NULL */
  Q8_ERR_BAD_SHAPE = 2,  /* M < 0, N or K < 1, K % 16 != 0, or a size overflows */
  Q8_ERR_BAD_DTYPE = 3,  /* unsupported element type for this argument */
  Q8_ERR_BAD_FORMAT = 4, /* unsupported quantization format for this call */
  Q8_ERR_BAD_ARG = 5,    /* NaN threshold/bound, or a pointer that must be NULL is not */
  Q8_ERR_ALIGN = 6,      /* a pointer is not 16-byte aligned */
  Q8_ERR_WORKSPACE = 7,  /* workspace NULL or smaller than q8_workspace_bytes */
  Q8_ERR_DEVICE = 8,     /* no HIP device, or the device is not gfx950 */
  Q8_ERR_LAUNCH = 9      /* a kernel launch failed */
} q8_status;

typedef enum q8_dtype { Q8_F32 = 0, Q8_F16 = 1, Q8_BF16 = 2 } q8_dtype;

typedef enum q8_format {
  Q8_INT8_ASYM = 0, /* weights: per-row asymmetric int8, r = S (q - Z)         */
  Q8_INT8_SYM = 1,  /* activations: per-row symmetric int8, r = S q           */
  Q8_FP8_E4M3 = 2   /* weights or activations: per-row OCP e4m3fn, r = S q    */
} q8_format;

typedef enum q8_op {
  Q8_OP_LINEAR = 0, Q8_OP_DECOMP = 1, Q8_OP_FP8 = 2, Q8_OP_STATIC = 3, Q8_OP_GROUPED = 4,
  Q8_OP_FP8_BLOCK = 5
} q8_op;

/*
 * q8_quantize_weight -- per-output-channel weight quantization (done once,
 * off the per-token path).
 *
 * Q8_INT8_ASYM  ([LF] §2.1 per-channel asymmetric scale and zero-point, §3.3
 *   quantizer; [OV] §2.3 min-max S = (R_max - R_min)/(Q_max - Q_min),
 *   Z = Q_min - round(R_min/S); [NOTE] "量化是什么" r = S (q - Z)).  Per row n:
 *     lo = min(0, min_k w), hi = max(0, max_k w)
 *     S  = max((hi - lo) / 255, 1e-8)
 *     Z  = -128 - rne(lo / S)                         (integer in [-128, 127])
 *     q  = clamp(rne(w / S) + Z, -128, 127)
 *   wq: int8 [N, K]; w_scale: float [N]; w_zp: float [N] holding the integer Z.
 * Q8_FP8_E4M3  ([FB] §5.1: e4m3fn weight, one fp32 weight_scale per output
 *   channel).  Per row n: S = max(max_k |w| / 448, 1e-8),
 *   q = e4m3_rne(clamp(w / S, -448, 448)).  wq: uint8 e4m3fn codes [N, K];
 *   w_scale: float [N]; w_zp must be NULL (else Q8_ERR_BAD_ARG).
 * w: [N, K] of type w_dtype (F32, F16 or BF16).
 * Errors: Q8_ERR_BAD_FORMAT for fmt == Q8_INT8_SYM.
 */
q8_status q8_quantize_weight(q8_format fmt, const void* w, q8_dtype w_dtype,
                             int64_t N, int64_t K, void* wq, float* w_scale,
                             float* w_zp, void* stream);

/*
 * q8_quantize_act -- dynamic per-token activation quantization (recomputed at
 * every forward: [NOTE] dynamic quantization section; [FB] §5.2).
 *
 * Q8_INT8_SYM  ([NOTE] symmetric section and QuantInt8 code).  Per row m:
 *     S = max(max_k |x| / 127, 1e-8);  q = clamp(rne(x / S), -127, 127)
 *   xq: int8 [M, K]; x_scale: float [M]; x_rowsum: int32 [M] = sum_k q (the
 *   term the weight zero-point correction needs), may be NULL.  scale_ub is
 *   ignored.
 * Q8_FP8_E4M3  ([FB] §1, §4, §6: per-row e4m3 with the activation scale upper
 *   bound, default 1200).  Per row m:
 *     a = min(max_k |x|, scale_ub);  S = max(a / 448, 1e-8)
 *     q = e4m3_rne(clamp(x / S, -448, 448))
 *   scale_ub = +INFINITY means no bound; NaN or <= 0 is Q8_ERR_BAD_ARG.
 *   xq: uint8 e4m3fn codes [M, K]; x_scale: float [M]; x_rowsum must be NULL.
 * x: [M, K] of type x_dtype (F32, F16 or BF16).
 * Errors: Q8_ERR_BAD_FORMAT for fmt == Q8_INT8_ASYM.
 */
q8_status q8_quantize_act(q8_format fmt, const void* x, q8_dtype x_dtype,
                          int64_t M, int64_t K, float scale_ub, void* xq,
                          float* x_scale, int32_t* x_rowsum, void* stream);

/*
 * q8_linear -- W8A8 linear layer: dynamic per-token INT8 X, per-channel
 * asymmetric INT8 W, INT8 x INT8 products with INT32 accumulation ([NOTE]
 * "INT8 这么小的范围不会导致溢出吗？"), then the dequantization epilogue
 * ([OV] §2.1 quantized matmul, read as Y = S_x X_q . (S_w (W_q - Z_w))^T):
 *     acc[m,n] = sum_k xq[m,k] wq[n,k]                      (exact int32)
 *     y[m,n]   = S_x[m] S_w[n] (acc[m,n] - Z_w[n] sum_k xq[m,k]) (+ bias[n])
 * The activation quantization is the Q8_INT8_SYM rule above.  For M <= 10 it
 * is fused into the one kernel; for larger M the codes, scales and code sums
 * pass through the workspace (for M <= 16 into a streaming GEMV, above into
 * the MFMA GEMM).
 * x: [M, K] of x_dtype (F32, F16, BF16); wq/w_scale/w_zp: from
 * q8_quantize_weight(Q8_INT8_ASYM); bias: float [N] or NULL; y: [M, N] of
 * y_dtype (F32, F16, BF16).  acc_out: int32 [M, N] debug copy of acc, or NULL.
 * workspace: q8_workspace_bytes(Q8_OP_LINEAR, M, N, K) bytes (0 for M <= 10).
 */
q8_status q8_linear(const void* x, q8_dtype x_dtype, int64_t M, int64_t K,
                    const int8_t* wq, const float* w_scale, const float* w_zp,
                    int64_t N, const float* bias, void* y, q8_dtype y_dtype,
                    void* workspace, size_t workspace_bytes, int32_t* acc_out,
                    void* stream);

/*
 * q8_linear_int8_decomp -- LLM.int8() mixed-precision decomposition ([BNB]
 * core idea: outlier feature columns go through a 16-bit product, the regular
 * ~99.9% of values through int8; BitsAndBytesConfig table: threshold 6.0,
 * 0.0 maximizes the int8 share).
 *     O = { k : max_m |x[m,k]| >= threshold }  (ascending; empty if threshold <= 0)
 *     X_R = X with the columns O set to 0, quantized as Q8_INT8_SYM (so the
 *           per-token scale is taken over the regular columns only)
 *     W_O[n,j] = fp16(S_w[n] (wq[n,O_j] - Z_w[n]))    (no fp16 weight copy kept)
 *     y = [int8 path of q8_linear on X_R] + X[:,O] . W_O^T (+ bias)
 * x: fp16 [M, K]; y: fp16 [M, N]; weights as for q8_linear.
 * outlier_idx: int32 [K] receives O in ascending order (entries past the
 * count are unspecified), or NULL; n_outliers: int32 [1] receives |O|, or
 * NULL.  Both stay on the device: the call never synchronizes.
 * acc_out: int32 [M, N] debug copy of the int8-path accumulator, or NULL.
 * threshold NaN is Q8_ERR_BAD_ARG.
 * workspace: q8_workspace_bytes(Q8_OP_DECOMP, M, N, K) bytes: the activation
 * codes, scales and row sums, the column flags, the outlier list and count,
 * and the first 16 outlier columns of X and of W_O in compact fp16 form
 * ((M + N) x 32 bytes), which the product reads instead of gathering them.
 */
q8_status q8_linear_int8_decomp(const void* x, int64_t M, int64_t K,
                                const int8_t* wq, const float* w_scale,
                                const float* w_zp, int64_t N, float threshold,
                                const float* bias, void* y, void* workspace,
                                size_t workspace_bytes, int32_t* outlier_idx,
                                int32_t* n_outliers, int32_t* acc_out,
                                void* stream);

/*
 * q8_linear_fp8 -- FP8 e4m3 W8A8 rowwise linear ([FB] §5.2 per-row dynamic
 * activation quantization with the scale upper bound; §5.3 fp8 x fp8 product
 * with row scales on both sides, bf16 output, fp32 bias added after):
 *     xq, S_x = Q8_FP8_E4M3 activation rule with scale_ub
 *     y[m,n]  = (sum_k e4m3(xq[m,k]) e4m3(wq[n,k]))  S_x[m] S_w[n] (+ bias[n])
 * Products are exact; the sum is accumulated in fp32.
 * x: bf16 [M, K] (other dtypes are Q8_ERR_BAD_DTYPE: the page's forward is
 * bf16 only); wq: e4m3fn codes [N, K] and w_scale float [N] from
 * q8_quantize_weight(Q8_FP8_E4M3); bias: float [N] or NULL; y: bf16 [M, N].
 * scale_ub as for q8_quantize_act.  workspace: q8_workspace_bytes(Q8_OP_FP8).
 */
q8_status q8_linear_fp8(const void* x, int64_t M, int64_t K, const uint8_t* wq,
                        const float* w_scale, int64_t N, float scale_ub,
                        const float* bias, void* y, void* workspace,
                        size_t workspace_bytes, void* stream);

/*
 * q8_gemm_int8 -- the INT8 GEMM and dequantization epilogue of q8_linear on
 * activations that are already quantized (by q8_quantize_act(Q8_INT8_SYM), or
 * shared by several projections of the same X):
 *     acc[m,n] = sum_k xq[m,k] wq[n,k];  y = S_x[m] S_w[n] (acc - Z_w[n] x_rowsum[m]) (+ bias)
 * ([NOTE] "INT8 这么小的范围不会导致溢出吗？": INT32 accumulation; [OV] §2.1
 * quantized matmul with r = S (q - Z)).  xq: int8 [M, K]; x_scale: float [M];
 * x_rowsum: int32 [M] (= sum_k xq, required); weights, bias, y, y_dtype and
 * acc_out as for q8_linear.  No workspace.  q8_linear with M > 10 is exactly
 * q8_quantize_act followed by this call.
 */
q8_status q8_gemm_int8(const int8_t* xq, const float* x_scale, const int32_t* x_rowsum,
                       int64_t M, int64_t K, const int8_t* wq, const float* w_scale,
                       const float* w_zp, int64_t N, const float* bias, void* y,
                       q8_dtype y_dtype, int32_t* acc_out, void* stream);

/*
 * q8_gemm_fp8 -- the rowwise FP8 product on quantized operands, the shape of
 * the page's f8f8bf16_rowwise(xq, w, x_scale, w_scale) ([FB] §5.3):
 *     y[m,n] = (sum_k e4m3(xq[m,k]) e4m3(wq[n,k])) S_x[m] S_w[n] (+ bias[n])
 * xq: e4m3fn codes [M, K] with x_scale float [M] (from q8_quantize_act
 * (Q8_FP8_E4M3)); wq, w_scale, bias as for q8_linear_fp8; y: bf16 [M, N].
 * No workspace.  q8_linear_fp8 is q8_quantize_act followed by this call.
 */
q8_status q8_gemm_fp8(const uint8_t* xq, const float* x_scale, int64_t M, int64_t K,
                      const uint8_t* wq, const float* w_scale, int64_t N, const float* bias,
                      void* y, void* stream);

/*
 * q8_linear_fp8_grouped -- FP8 expert projection of a mixture-of-experts layer
 * on routed tokens ([FB] §5.4, Llama4 experts: per-expert FP8 weights with
 * per-row scales; each expert's tokens get per-token FP8 quantization and the
 * rowwise FP8 product with that expert's weights).  Rows
 * expert_offsets[e] .. expert_offsets[e+1]-1 of x belong to expert e:
 *     y[t,n] = S_x[t] S_w[e,n] sum_k e4m3(xq[t,k]) e4m3(wq[e,n,k])   (fp32 acc)
 * with the activation quantization of q8_quantize_act(Q8_FP8_E4M3, scale_ub).
 * x: bf16 [T, K] grouped by expert; expert_offsets: int32 [E+1] in DEVICE
 * memory, non-decreasing from 0 to T (the offsets are read on the device and
 * never copied to the host; values outside [0, T] or decreasing are clamped,
 * which may leave rows of y unwritten but never reads or writes outside the
 * arrays); wq: e4m3 [E, N, K] and w_scale: float [E, N] from
 * q8_quantize_weight(Q8_FP8_E4M3) on the [E*N, K] view; y: bf16 [T, N].
 * workspace: q8_workspace_bytes(Q8_OP_FP8, T, N, K).  Errors: Q8_ERR_BAD_SHAPE
 * unless 1 <= E <= 1024; Q8_ERR_BAD_ARG for a NaN or non-positive scale_ub.
 */
q8_status q8_linear_fp8_grouped(const void* x_bf16, int64_t T, int64_t K,
                                const int32_t* expert_offsets, int64_t E,
                                const uint8_t* wq, const float* w_scale, int64_t N,
                                float scale_ub, void* y_bf16, void* workspace,
                                size_t workspace_bytes, void* stream);

/*
 * q8_quantize_act_static -- static INT8 activation quantization ("lecture
 * notes on LLM quantization", static quantization: the scale is calibrated
 * beforehand and applied unchanged at inference): one float scale S for the
 * tensor, xq = clamp(rne(x / S), -127, 127) with the binary32 division,
 * x_rowsum[m] = sum_k xq[m,k] (nullable).  x: [M, K] of x_dtype; xq: int8
 * [M, K].  Errors: Q8_ERR_BAD_ARG unless 0 < x_scale < inf.
 */
q8_status q8_quantize_act_static(const void* x, q8_dtype x_dtype, int64_t M, int64_t K,
                                 float x_scale, int8_t* xq, int32_t* x_rowsum, void* stream);

/*
 * q8_linear_static -- W8A8 linear with a static activation scale and an INT8
 * output for the next layer (same notes, "INT8 这么小的范围不会导致溢出吗？", step 4:
 * the INT32 result is scaled back into INT8):
 *     xq = q8_quantize_act_static(x, x_scale);  acc = sum_k xq wq  (exact int32)
 *     v  = (x_scale S_w[n]) (acc - Z_w[n] sum_k xq) (+ bias[n])       (float64)
 *     yq = clamp(rne(v * (1 / y_scale)), -127, 127)                   (float64)
 * x: [M, K] of x_dtype; weights from q8_quantize_weight(Q8_INT8_ASYM); bias:
 * float [N] or NULL; yq: int8 [M, N].  workspace:
 * q8_workspace_bytes(Q8_OP_STATIC, M, N, K) bytes.  Errors: Q8_ERR_BAD_ARG
 * unless both scales are finite and positive.
 */
q8_status q8_linear_static(const void* x, q8_dtype x_dtype, int64_t M, int64_t K, float x_scale,
                           const int8_t* wq, const float* w_scale, const float* w_zp, int64_t N,
                           const float* bias, float y_scale, int8_t* yq, void* workspace,
                           size_t workspace_bytes, void* stream);

/*
 * q8_linear_w8a16 -- weight-only linear for decode-sized M: the INT8
 * asymmetric weights are dequantized for a product with the 16-bit
 * activations, which are not quantized ("lecture notes on LLM quantization",
 * PTQ section, weight quantization):
 *     y[m,n] = S_w[n] Sum_k x[m,k] (wq[n,k] - Z_w[n])  (+ bias[n])
 * The widened weights are exact; products accumulate in fp32.
 * x: [M, K] of x_dtype (BF16 or F16 only); wq/w_scale/w_zp: from
 * q8_quantize_weight(Q8_INT8_ASYM); bias: float [N] or NULL; y: [M, N] of
 * y_dtype (F32, F16, BF16).  No workspace.
 * Errors: Q8_ERR_BAD_DTYPE for an F32 x; Q8_ERR_BAD_SHAPE for M > 16, besides
 * the preconditions above.
 */
q8_status q8_linear_w8a16(const void* x, q8_dtype x_dtype, int64_t M, int64_t K,
                          const int8_t* wq, const float* w_scale, const float* w_zp,
                          int64_t N, const float* bias, void* y, q8_dtype y_dtype,
                          void* stream);

/*
 * q8_quantize_weight_grouped -- per-group asymmetric INT8 weights ("大模型量化
 * 技术概述" §2.2, granularity: groups of 64 to 128 parameters, each with its
 * own parameters; lecture notes' granularity passage: per-group blocks with
 * their own scale and zero point).  Group j of row n is w[n, j g .. j g + g-1];
 * each group is quantized as Q8_INT8_ASYM quantizes a row:
 *     lo = min(0, min w), hi = max(0, max w), S = max((hi - lo)/255, 1e-8),
 *     Z = -128 - rne(lo / S),  q = clamp(rne(w / S) + Z, -128, 127)
 * w: [N, K] of w_dtype; group: 64 or 128 and K a multiple of it (else
 * Q8_ERR_BAD_SHAPE); wq: int8 [N, K]; w_scale, w_zp: float [K/group, N],
 * group-major (w_scale[j * N + n] belongs to group j of row n; w_zp holds the
 * integer Z).
 */
q8_status q8_quantize_weight_grouped(const void* w, q8_dtype w_dtype, int64_t N, int64_t K,
                                     int64_t group, int8_t* wq, float* w_scale, float* w_zp,
                                     void* stream);

/*
 * q8_linear_grouped -- W8A8 linear with per-group weights: the activations are
 * quantized per token as q8_quantize_act(Q8_INT8_SYM) does, and the
 * quantized-matmul identity is taken group by group ([OV] §2.1 with r = S (q - Z)):
 *     C_j[m,n] = sum_{k in j} xq[m,k] wq[n,k] - Z[j,n] sum_{k in j} xq[m,k]   (exact)
 *     y[m,n]   = S_x[m] sum_j S[j,n] C_j[m,n]  (+ bias[n])                    (fp32)
 * x: [M, K] of x_dtype; wq/w_scale/w_zp from q8_quantize_weight_grouped with
 * the same group; bias: float [N] or NULL; y: [M, N] of y_dtype.  workspace:
 * q8_workspace_bytes(Q8_OP_GROUPED, M, N, K) bytes: none up to 10 tokens
 * (the quantization is fused into the decode kernel), else codes, scales and
 * group code sums, sized for group 64.  Errors: Q8_ERR_BAD_SHAPE for a group
 * other than 64 or 128 or a K that is not a multiple of it.
 */
q8_status q8_linear_grouped(const void* x, q8_dtype x_dtype, int64_t M, int64_t K,
                            const int8_t* wq, const float* w_scale, const float* w_zp,
                            int64_t group, int64_t N, const float* bias, void* y,
                            q8_dtype y_dtype, void* workspace, size_t workspace_bytes,
                            void* stream);

/*
 * q8_linear_noalloc -- q8_linear with no workspace argument, for callers that
 * cannot allocate device memory around a call (code under HIP graph capture,
 * tight serving loops, harnesses that forbid allocation).  Same arguments,
 * computation, kernels and results as q8_linear, bit for bit.  The scratch
 * that q8_linear takes from the workspace (above 10 tokens: the activation
 * codes, scales and code sums, q8_workspace_bytes(Q8_OP_LINEAR, M, N, K)
 * bytes) comes from a library-owned 32 MiB device array per GPU, created with
 * the library and kept until the process ends; nothing is allocated or freed
 * by the call.  Every call on one GPU shares that GPU's array: calls that may
 * overlap on one GPU (other streams, other host threads) race and must be
 * ordered by the caller.  The array keeps the last call's contents; nothing
 * in it needs to start at zero.  The first call on a device looks up the
 * array's address there (host side, once per device).
 * Errors: as q8_linear, and Q8_ERR_WORKSPACE if the scratch the shape needs
 * exceeds 32 MiB (M * K + 8 M plus alignment: e.g. M = 4096 at K = 8192).
 */
q8_status q8_linear_noalloc(const void* x, q8_dtype x_dtype, int64_t M, int64_t K,
                            const int8_t* wq, const float* w_scale, const float* w_zp,
                            int64_t N, const float* bias, void* y, q8_dtype y_dtype,
                            int32_t* acc_out, void* stream);

/*
 * The paged 8-bit key/value cache
 * -------------------------------
 * Keys and values of a layer are held as OCP e4m3fn codes in pages of `page`
 * tokens (32, 64 or 128), with one power-of-two scale per page, kv head and
 * tensor, kept as an exponent byte b: a code c stands for e4m3(c) 2^(b - 127).
 *   k_cache  uint8 [num_pages, Hkv, page, D]   keys, the features of a token together
 *   v_cache  uint8 [num_pages, Hkv, D, page]   values, the tokens of a feature together
 *   k_exp, v_exp  uint8 [num_pages, Hkv]       exponent bytes
 * D is 64, 128 or 256.  A scale that is a power of two costs e4m3 no precision
 * (its precision is relative), lets a page's older codes be re-expressed
 * exactly when a larger value joins them (bar values that leave e4m3's range
 * below), and is applied by exponent arithmetic.  A byte of 255 must not occur.
 *
 * A batch of S sequences over the cache:
 *   q_start      int32 [S + 1]: tokens q_start[s] .. q_start[s+1]-1 of the
 *                token arrays are sequence s's new tokens (n of them, may be 0)
 *   kv_len       int32 [S]: its length with the new tokens; new token i has
 *                position kv_len[s] - n + i
 *   block_table  int32 [S, max_pages]: page of positions page * j ..
 *                page * j + page - 1 of sequence s at [s, j]
 * All three are device memory, read on the device only.  max_q and max_kv are
 * the caller's bounds on n and kv_len (they size grids and splits: too small a
 * bound costs time, not results).  q_start is clamped to [0, T], a decreasing
 * pair counts as no tokens; positions before 0 or past max_pages * page do not
 * exist; page numbers outside [0, num_pages) are skipped by the append and read
 * as the nearest page by the attention.  Nothing outside the arrays is read or
 * written whatever these arrays hold.
 */

/*
 * q8_kv_append -- put new keys and values into the cache and rotate the new
 * queries, in one launch.  For sequence s's token at position p:
 *     rotation (cos, sin given; features 0 .. rot_dim-1 of each head, r = rot_dim / 2):
 *       interleaved = 0: pairs (i, i + r);  1: pairs (2 i, 2 i + 1);  i < r
 *       (a, b) -> (a cos[p,i] - b sin[p,i], b cos[p,i] + a sin[p,i])   (binary32, uncontracted)
 *     keys are rotated, values are not; q_out receives the rotated queries
 *     rounded to their type.
 * Each (page, kv head, tensor) that receives tokens:
 *     want = least b >= 0 with max |new values| <= 448 2^(b - 127)
 *     b'   = want if no older token lies in the page (it is started anew), else max(b, want)
 *     older codes c -> e4m3_rne(e4m3(c) 2^(b - b')), new codes e4m3_rne(x 2^(127 - b'))
 * Slots at or past kv_len, and those of other pages, keep their bytes.  Two
 * sequences must not append to the same page in one call.
 * k, v: [T, Hkv, D] and q: [T, Hq, D] of `dtype` (F32, F16, BF16), tokens
 * k_stride, v_stride, q_stride elements apart (slices of one fused projection,
 * say; multiples of 16 bytes), heads and features dense.  q and q_out may both
 * be NULL (then Hq is ignored); q_out: [T, Hq, D] dense, may be q if q is dense.
 * cos, sin: float [positions, rot_dim / 2], or both NULL (no rotation);
 * positions past the table use its last row.  rot_dim: a multiple of 16 up to D.
 * No workspace.  T = 0: arguments are checked, nothing is enqueued.
 */
q8_status q8_kv_append(const void* q, int64_t q_stride, const void* k, int64_t k_stride,
                       const void* v, int64_t v_stride, q8_dtype dtype, int64_t T, int64_t Hq,
                       int64_t Hkv, int64_t D, const float* cos, const float* sin,
                       int64_t positions, int64_t rot_dim, int interleaved,
                       const int32_t* q_start, const int32_t* kv_len, const int32_t* block_table,
                       int64_t S, int64_t max_pages, int64_t max_q, uint8_t* k_cache,
                       uint8_t* k_exp, uint8_t* v_cache, uint8_t* v_exp, int64_t num_pages,
                       int64_t page, void* q_out, void* stream);

/*
 * q8_kv_append_norm -- q8_kv_append with each head of the new keys and queries
 * normalised before it is rotated, and positions of the tokens' own.  A head x:
 *     r = 1 / sqrt(sum_i x_i^2 / D + eps)   (sum and root in binary64, r rounded to binary32)
 *     x_i -> (x_i r) w_i                    (binary32, each product rounded)
 * then rotation and the append's rule as above.  Values are not normalised.
 * q_weight, k_weight: [D] of w_dtype (F32, F16, BF16); NULL: that side is not
 * normalised.  eps is positive and finite (ignored if both are NULL).
 * token_positions: int32 [T] in device memory, the position that each token is
 * rotated by (a drafted token's depth behind the cached ones, while its slot is
 * its place among the new tokens), below 0 read as 0; NULL: its slot's.  The
 * slots are q_start's and kv_len's in either case.
 * Everything else is q8_kv_append's, with `positions` the rows of cos and sin.
 */
q8_status q8_kv_append_norm(const void* q, int64_t q_stride, const void* k, int64_t k_stride,
                            const void* v, int64_t v_stride, q8_dtype dtype, int64_t T, int64_t Hq,
                            int64_t Hkv, int64_t D, const void* q_weight, const void* k_weight,
                            q8_dtype w_dtype, float eps, const float* cos, const float* sin,
                            int64_t positions, int64_t rot_dim, int interleaved,
                            const int32_t* token_positions, const int32_t* q_start,
                            const int32_t* kv_len, const int32_t* block_table, int64_t S,
                            int64_t max_pages, int64_t max_q, uint8_t* k_cache, uint8_t* k_exp,
                            uint8_t* v_cache, uint8_t* v_exp, int64_t num_pages, int64_t page,
                            void* q_out, void* stream);

/*
 * q8_attention_kv8 -- softmax attention of the new queries over the cache.
 * Query token at position p, head h (reads kv head h / (Hq / Hkv)); keys j of
 * its sequence with j < kv_len, j <= p if causal, j > p - window if window > 0:
 *     w_j = softmax_j(scale q . k_j),   out = sum_j w_j v_j,   lse = log sum_j exp(scale q . k_j)
 * A query that sees no key gets out = 0 and lse = -inf, one with a NaN among the
 * scores that it sees NaN in both.  Codes of keys that a query does not see have
 * no part in its output, NaN codes included; pages that no query sees need not
 * exist.  Scores are exact products of codes and 16-bit queries.
 * The weight of a key's value codes, w_j times its page's 2^(b - 127), is
 * rounded to f16 (2^-11 of it, or 2^-24 of the row's largest such weight where
 * that is more); its products with the codes are exact.  All sums, the maximum
 * and the output accumulator are binary32.
 * q: [T, Hq, D] of `dtype` (F16 or BF16), tokens q_stride elements apart (a
 * multiple of 8); out: [T, Hq, D] of dtype; lse: float [T, Hq] or NULL.  Rows of
 * tokens that belong to no sequence are left alone.  Hq is a multiple of Hkv.
 * workspace: q8_attention_workspace_bytes(...) with the same sizes (0 where the
 * keys are not split over workgroups).
 */
q8_status q8_attention_kv8(const void* q, int64_t q_stride, q8_dtype dtype, int64_t T, int64_t Hq,
                           int64_t Hkv, int64_t D, const int32_t* q_start, const int32_t* kv_len,
                           const int32_t* block_table, int64_t S, int64_t max_pages, int64_t max_q,
                           int64_t max_kv, const uint8_t* k_cache, const uint8_t* k_exp,
                           const uint8_t* v_cache, const uint8_t* v_exp, int64_t num_pages,
                           int64_t page, float scale, int causal, int64_t window, void* out,
                           float* lse, void* workspace, size_t workspace_bytes, void* stream);

/* Bytes of workspace q8_attention_kv8 needs at these sizes; 0 for invalid ones,
 * which the call itself then rejects. */
size_t q8_attention_workspace_bytes(int64_t T, int64_t Hq, int64_t Hkv, int64_t D, int64_t S,
                                    int64_t max_q, int64_t max_kv, int64_t window);

/*
 * q8_attention_kv8_tree -- q8_attention_kv8 where the new tokens of a sequence
 * are drafts that continue each other as a tree (they lie in the cache already,
 * put there by an append).  New token i of a sequence with n of them, `past` =
 * kv_len - n cached before, sees
 *     cached keys j < past, of them those with j > p - window if window > 0
 *     new keys past + j with bit j % 64 of mask[t, j / 64] set (t = q_start + i; whatever the window)
 * p: token_positions[t], taken within past .. past + n - 1; NULL: past + i.  A
 * token sees itself only if its own bit is set; new keys without a bit in the
 * row (j >= 64 mask_words) are not seen.
 * mask: uint64 [T, mask_words] in device memory, 8-byte aligned; mask_words
 * from 1 to 32768.  Everything else, a query that sees no key among it, is as
 * q8_attention_kv8 has it.
 * workspace: q8_attention_tree_workspace_bytes(...) with the same sizes.
 */
q8_status q8_attention_kv8_tree(const void* q, int64_t q_stride, q8_dtype dtype, int64_t T,
                                int64_t Hq, int64_t Hkv, int64_t D, const int32_t* q_start,
                                const int32_t* kv_len, const int32_t* block_table, int64_t S,
                                int64_t max_pages, int64_t max_q, int64_t max_kv,
                                const uint8_t* k_cache, const uint8_t* k_exp, const uint8_t* v_cache,
                                const uint8_t* v_exp, int64_t num_pages, int64_t page,
                                const uint64_t* mask, int64_t mask_words,
                                const int32_t* token_positions, float scale, int64_t window,
                                void* out, float* lse, void* workspace, size_t workspace_bytes,
                                void* stream);

/* Bytes of workspace q8_attention_kv8_tree needs at these sizes; 0 for invalid ones. */
size_t q8_attention_tree_workspace_bytes(int64_t T, int64_t Hq, int64_t Hkv, int64_t D, int64_t S,
                                         int64_t max_q, int64_t max_kv, int64_t window);

/*
 * Calls over the caches of all layers, which share one block table: k_cache,
 * k_exp, v_cache and v_exp are arrays in HOST memory of `layers` device pointers
 * (1 to 512, read before the call returns).  None of the caches' arrays overlaps
 * another one or any other array of the call (Q8_ERR_BAD_ARG).
 *
 * q8_kv_compact -- the drafts of a batch that are kept go to the front of their
 * slots, in place.  keep[s, i], i < n_keep[s]: the new token (0 .. n-1, as
 * q_start numbers them) that becomes new token i of sequence s.  They grow
 * (a path of a tree whose tokens follow the ones they continue); the list ends
 * before an entry that does not, or is n or more.  Tokens with keep[s, i] = i at
 * its front are in place.  The others, in slots p + keep[s, i] (p = kv_len - n),
 * go to p + i by the append's rule, their values being what their codes stand
 * for: each (page, kv head, tensor) that receives tokens:
 *     want = least b >= 0 with max |moved values| <= 448 2^(b - 127)
 *     b'   = want if the page's first slot is one of the p + i, else max(b, want)
 *     slots before the first of the p + i in the page: codes c -> e4m3_rne(e4m3(c) 2^(b - b'))
 *     a token from a page of byte u: code c -> e4m3_rne(e4m3(c) 2^(u - b')); NaN codes stay as they are
 * Other slots keep their bytes (those behind the kept tokens are no longer
 * read).  len_out[s] = p + the number kept.
 * Tokens whose slot or target does not exist, or whose page number lies outside
 * [0, num_pages), are not moved.  Two sequences must not share a page that one
 * of them moves tokens in.
 * keep: int32 [S, max_keep], n_keep, len_out: int32 [S], device memory; len_out
 * overlaps no other array (Q8_ERR_BAD_ARG).  q_start, kv_len, block_table and
 * the sizes as for q8_kv_append.  No workspace.
 */
q8_status q8_kv_compact(uint8_t* const* k_cache, uint8_t* const* k_exp, uint8_t* const* v_cache,
                        uint8_t* const* v_exp, int64_t layers, int64_t Hkv, int64_t D,
                        const int32_t* q_start, const int32_t* kv_len, const int32_t* block_table,
                        int64_t S, int64_t max_pages, int64_t num_pages, int64_t page,
                        const int32_t* keep, int64_t max_keep, const int32_t* n_keep,
                        int32_t* len_out, void* stream);

/*
 * q8_kv_fork -- a batch of S_out sequences that continue those of a batch of S:
 * beams after a step, samples of a prompt, sequences that end, room for the next
 * tokens.  refs[x] counts the block table entries that hold page x; 0: free.
 * Sequence s of the new batch continues parent[s] (outside [0, S): it is empty
 * and has no pages), L = kv_len[parent[s]] within [0, max_pages page] tokens:
 *     entries j < L / page (full pages) are the parent's, shared
 *     entries from there to (L + room) / page, rounded up, max_pages at most:
 *       the parent's, if s is the first that continues it, it has one there and refs of it is 1;
 *       else a new page, and if L ends inside it (j = L / page) the parent's page copied into it,
 *       codes and exponent bytes, in every layer
 *     further entries are -1
 *     refs_out[x] = refs[x] - (entries of block_table that hold x) + (of table_out)
 * Entries outside [0, num_pages) are none.  New pages are numbered by sequence
 * and entry and are, in that order, the lowest pages that no entry holds any more
 * (refs 0 once block_table's are let go and the shared and kept ones counted;
 * pages that are copied from excepted).  missing[0] receives how many there were
 * too few of: those entries are -1, and a sequence whose last tokens would be in
 * one ends at the page before (len_out).  Else len_out[s] = L.
 * The old table is let go as a whole: with parent = 0 .. S-1 a batch goes on as
 * it is and gets its room, with fewer the others' pages are free afterwards.
 * block_table: int32 [S, max_pages], kv_len: [S], refs: [num_pages], parent:
 * [S_out]; table_out: [S_out, max_pages], len_out: [S_out], refs_out:
 * [num_pages], missing: [1]; device memory, outputs and workspace overlap
 * neither inputs nor each other (Q8_ERR_BAD_ARG).  room: 0 to 2^30; table_out has
 * fewer than 2^31 entries.
 * workspace: q8_kv_fork_workspace_bytes(S, S_out, num_pages) bytes.
 */
q8_status q8_kv_fork(uint8_t* const* k_cache, uint8_t* const* k_exp, uint8_t* const* v_cache,
                     uint8_t* const* v_exp, int64_t layers, int64_t Hkv, int64_t D,
                     int64_t num_pages, int64_t page, const int32_t* block_table,
                     const int32_t* kv_len, const int32_t* refs, int64_t S, int64_t max_pages,
                     const int32_t* parent, int64_t S_out, int64_t room, int32_t* table_out,
                     int32_t* len_out, int32_t* refs_out, int32_t* missing, void* workspace,
                     size_t workspace_bytes, void* stream);

/* Bytes of workspace q8_kv_fork needs; 0 for invalid sizes. */
size_t q8_kv_fork_workspace_bytes(int64_t S, int64_t S_out, int64_t num_pages);

/*
 * Block-scaled FP8 linear: e4m3 codes with one scale per token and 128
 * features of X and one per 128 rows x 128 features of W, the granularity of
 * block-quantized FP8 checkpoints.  G = ceil(K / 128); the last block of a
 * dimension may be short.
 *
 * q8_quantize_weight_block (once per weight) and q8_quantize_act_block:
 *     S = max(max |.| over the block / 448, 1e-8),  q = e4m3_rne(clamp(. / S, -448, 448))
 * w: [N, K], wq: uint8 [N, K], w_scale: float [ceil(N / 128), G].
 * x: [M, K], xq: uint8 [M, K], x_scale: float [G, M] (block-major).
 * A NaN or an infinity makes its block's S one, and what is computed from the
 * block is not finite (NaN for a NaN).
 * w, x of type F32, F16 or BF16.
 */
q8_status q8_quantize_weight_block(const void* w, q8_dtype w_dtype, int64_t N, int64_t K,
                                   uint8_t* wq, float* w_scale, void* stream);
q8_status q8_quantize_act_block(const void* x, q8_dtype x_dtype, int64_t M, int64_t K, uint8_t* xq,
                                float* x_scale, void* stream);

/*
 * q8_gemm_fp8_block -- the product on quantized operands:
 *     y[m,n] = sum_j S_x[j,m] S_w[n / 128, j] (sum_{k in block j} e4m3(xq[m,k]) e4m3(wq[n,k]))  (+ bias[n])
 * The inner sums run on the FP8 matrix instruction, the outer in binary32.
 * bias: float [N] or NULL; y: [M, N] of y_dtype (F16 or BF16: the
 * instruction's sums do not carry binary32 precision).  No workspace.
 */
q8_status q8_gemm_fp8_block(const uint8_t* xq, const float* x_scale, int64_t M, int64_t K,
                            const uint8_t* wq, const float* w_scale, int64_t N, const float* bias,
                            void* y, q8_dtype y_dtype, void* stream);

/*
 * q8_linear_fp8_block -- q8_quantize_act_block followed by q8_gemm_fp8_block;
 * for M <= 4 in one launch, the codes passing through LDS.
 * x: [M, K] of x_dtype (F32, F16, BF16); y of y_dtype (F16 or BF16).
 * workspace: q8_workspace_bytes(Q8_OP_FP8_BLOCK, M, N, K) bytes (0 for M <= 4).
 */
q8_status q8_linear_fp8_block(const void* x, q8_dtype x_dtype, int64_t M, int64_t K,
                              const uint8_t* wq, const float* w_scale, int64_t N,
                              const float* bias, void* y, q8_dtype y_dtype, void* workspace,
                              size_t workspace_bytes, void* stream);

/* Bytes of workspace the call `op` needs at this shape (0 if none); returns 0
 * for invalid shapes as well, which the call itself then rejects. */
size_t q8_workspace_bytes(q8_op op, int64_t M, int64_t N, int64_t K);

/* Static, human-readable name of a status code. */
const char* q8_status_str(q8_status s);

#ifdef __cplusplus
}
#endif

#endif /* Q8_H */
