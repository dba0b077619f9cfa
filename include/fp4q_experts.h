/*
 * fp4q_experts.h -- C ABI of the mixture-of-experts entry points of libfp4q:
 * one feed-forward layer of experts with FP4 products, from the router's
 * choices to the weighted sum of the experts' outputs.
 *
 *   fp4q_expert_sort         choices -> rows of the expert order
 *   fp4q_expert_quantize     tokens -> quantized rows in expert order
 *   fp4q_expert_gemm         rows x their expert's weights (W4A4)
 *   fp4q_glu_quantize        gated activation -> quantized rows
 *   fp4q_expert_combine      rows -> tokens, weighted sum
 *   fp4q_glu_bwd, fp4q_expert_combine (weights NULL), fp4q_expert_combine_bwd
 *                            gradients, straight through the quantizer
 *
 * The formats, the storage of codes, the status codes and every convention of
 * fp4q.h hold here too (device pointers owned by the caller, 16-byte aligned,
 * nothing allocated, nothing synchronised, arguments validated on the host
 * before anything is enqueued, an empty call enqueues nothing). Device-side
 * integers (ids, counts, starts, slots) cannot be checked on the host; what
 * the kernels do with bad ones is said at each entry point.
 *
 * State beyond fp4q.h's list: the resident CTAs per SM of each row quantize
 * kernel, and one bit per product or sort kernel and device (its shared-memory limit
 * has been raised, to the most that any call needs). The product's waits are bounded like the TMA-fed
 * quantizer's; one that runs out ends the call early and adds to the counter of
 * fp4q_device_errors.
 *
 * The row layout. The choices of T tokens, k each, are spread over
 * `experts` segments of rows: expert e's rows are starts[e] ..
 * starts[e] + counts[e] - 1, in the order of the choices, and every start is a
 * multiple of 128 (the row tile of the block-scaled MMA's scale layout). The
 * buffers of all entry points have `rows` rows, a multiple of 128 that is at
 * least fp4q_expert_rows(T * k, experts), which covers every routing. Rows that hold no choice (the
 * end of a segment's last 128 rows, rows behind the last segment) are
 * neither read for a result nor written: they stay as they were. slots[t * k + j]
 * is the row of choice j of token t, or -1 for a choice that is dropped; no two
 * choices share a row. A token may choose the same expert twice; each choice gets a row.
 */
#ifndef FP4Q_EXPERTS_H
#define FP4Q_EXPERTS_H

#include "fp4q.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Limits: 1 <= k <= 64, 1 <= experts <= 1024, and padded rows below 2^31. */
#define FP4Q_MAX_EXPERTS 1024
#define FP4Q_MAX_CHOICES 64
/* Floats of the abs-max scratch of fp4q_expert_quantize and fp4q_glu_quantize. */
#define FP4Q_AMAX_WORK 1024

/* Gate of the gated linear unit: a(g) = g * sigmoid(z(g)) with
 * SILU z = g; GELU_TANH z = 2 sqrt(2/pi) (g + 0.044715 g^3), which is
 * g/2 (1 + tanh(sqrt(2/pi) (g + 0.044715 g^3))). */
typedef enum { FP4Q_ACT_SILU = 0, FP4Q_ACT_GELU_TANH = 1 } fp4q_activation;

/* Rows that n choices among `experts` experts need at most: 128 *
 * floor((n + 127 min(n, experts)) / 128). 0 for n == 0; -1 for arguments out
 * of range. Host only. */
int64_t fp4q_expert_rows(int64_t n, int64_t experts);

/* Bytes of the scratch `work` of fp4q_expert_sort. -1 for arguments out of
 * range. Host only. */
int64_t fp4q_expert_sort_work(int64_t n, int64_t experts);

/*
 * fp4q_expert_sort -- stable counting sort of the choices by expert.
 * ids      int32 (id_bytes 4) or int64 (id_bytes 8) [n], n = T * k choices in
 *          token order; a value outside 0 .. experts-1 drops the choice.
 * counts   int32 [experts]; starts int32 [experts + 1], starts[experts] is the
 *          end of the last segment; slots int32 [n].
 * work     fp4q_expert_sort_work(n, experts) bytes of scratch (NULL when 0).
 * The result is a function of the ids alone (no atomic's order enters it).
 * n == 0 writes zero counts and starts.
 * Errors: UNSUPPORTED (id_bytes), SHAPE (n, experts), NULL, ALIGN, CUDA.
 */
fp4q_status fp4q_expert_sort(const void* ids, int id_bytes, int64_t n, int64_t experts,
                             int32_t* counts, int32_t* starts, int32_t* slots, void* work,
                             cudaStream_t stream);

/*
 * fp4q_expert_quantize -- fp4q_quantize_mma of every token, written to the
 * rows of its choices: for a given abs-max (and for MXFP4) bit for bit the codes and scale
 * bytes that quantizing the gathered rows gives. A token is quantized once.
 * x            bf16 [tokens, cols]; cols a multiple of 32 and of rot, tokens *
 *              cols / 32 at most 0xF0000000.
 * slots        int32 [tokens, k]; a value outside 0 .. rows-1 is skipped.
 * rows         rows of the outputs, a multiple of 128.
 * fmt, strat, rot as fp4q_quantize_mma (NVFP4 block 16, MXFP4 block 32).
 * global_amax_in   NVFP4: device float with a calibrated abs-max (s_g = amax /
 *              2688, one division, as fp4q_quantize), or NULL to
 *              take the abs-max of all of x (rotated; tokens without a choice
 *              included) in an extra pass; s_g is then that maximum times fp32(1 / 2688), which
 *              may be one unit in the last place from the quotient, and codes at ties with it (for
 *              fp4q_quantize's own bits pass fp4q_global_amax's value). Ignored for MXFP4.
 * global_scale_out NVFP4: device float, receives s_g.
 * amax_work    FP4Q_AMAX_WORK device floats of scratch, needed when fmt is NVFP4 and
 *              global_amax_in is NULL; distinct from global_scale_out.
 * codes        uint8 [rows, cols/2].
 * mma_scales   fp4q_mma_scale_bytes(rows, cols, fmt) bytes in the layout of
 *              fp4q_scales_to_mma; the padding blocks of written rows become
 *              zero (the buffer need not be cleared).
 * dq           NULL, or [rows, cols] of dq_dtype: the values of the codes.
 * tokens == 0: only global_scale_out is written (1.0), as fp4q_quantize.
 */
fp4q_status fp4q_expert_quantize(const void* x, int64_t tokens, int64_t cols, int k,
                                 const int32_t* slots, int64_t rows, fp4q_format fmt,
                                 fp4q_strategy strat, int rot, const float* global_amax_in,
                                 float* global_scale_out, float* amax_work, uint8_t* codes,
                                 uint8_t* mma_scales, void* dq, fp4q_dtype dq_dtype,
                                 cudaStream_t stream);

/*
 * fp4q_expert_gemm -- the grouped W4A4 product: for every row r of expert e,
 * d[r, m] = alpha_e * sum_k a[r, k] * w[e, m, k]; NVFP4 alpha_e = s_g(a) *
 * s_g(w_e), MXFP4 alpha_e = 1. Each operand as fp4q_quantize_mma writes it.
 * a_codes      uint8 [rows, K/2]; a_mma_scales in MMA layout; a_global_scale
 *              one device float (NVFP4).
 * w_codes      uint8 [experts, N, K/2]; w_mma_scales [experts] consecutive
 *              buffers of fp4q_mma_scale_bytes(N, K, fmt) bytes;
 *              w_global_scale float [experts] (NVFP4).
 * counts, starts  as written by fp4q_expert_sort. A segment that does not lie
 *              inside 0 .. rows or does not start at a multiple of 128 is left out.
 * mean_rows    the caller's estimate of the rows of an expert that has any: picks
 *              the tile (one CTA or a pair), nothing else. Results of the two forms may
 *              differ by the order of the fp32 sums.
 * d            [rows, N] of d_dtype; rows without a choice stay as they were.
 * K a multiple of 32, N of 4 (fp32 output) or 8 (bf16). Products accumulate
 * in fp32 on the tensor cores. rows == 0 enqueues nothing.
 */
fp4q_status fp4q_expert_gemm(const uint8_t* a_codes, const uint8_t* a_mma_scales,
                             const float* a_global_scale, const uint8_t* w_codes,
                             const uint8_t* w_mma_scales, const float* w_global_scale,
                             const int32_t* counts, const int32_t* starts, int64_t experts,
                             int64_t rows, int64_t N, int64_t K, fp4q_format fmt,
                             int64_t mean_rows, void* d, fp4q_dtype d_dtype, cudaStream_t stream);

/*
 * fp4q_glu_quantize -- h = bf16(fp32(a(g) * u)) for the gate g and the value u
 * of each row, then fp4q_quantize_mma of h.
 * gu           bf16 [rows, 2 * cols]: the gate in columns 0 .. cols-1, the value
 *              in cols .. 2 cols - 1. a(g) * u is rounded to fp32 and then to
 *              bf16 from its real value (not from a rounded sigmoid), so h and
 *              everything behind it is a function of the input bits.
 * slots, n     int32 [n]: the rows to take (a value outside 0 .. rows-1 is skipped;
 *              a row named twice is written twice with the same bits), or
 *              NULL for all rows (n is ignored; a call that takes none has rows 0 or
 *              slots that are not NULL, n 0).
 * cols         a multiple of 32 and of rot (rows taken * cols / 32 at most
 *              0xF0000000); other arguments as fp4q_expert_quantize. global_amax_in NULL (NVFP4) takes the
 *              abs-max of the rotated h over the rows taken, and s_g from it as there. Without slots,
 *              rows may be any number and mma_scales has
 *              fp4q_mma_scale_bytes(rows, cols, fmt) bytes.
 * Inputs and a(g) * u must be finite.
 */
fp4q_status fp4q_glu_quantize(const void* gu, int64_t rows, int64_t cols, const int32_t* slots,
                              int64_t n, fp4q_activation act, fp4q_format fmt, fp4q_strategy strat,
                              int rot, const float* global_amax_in, float* global_scale_out,
                              float* amax_work, uint8_t* codes, uint8_t* mma_scales, void* dq,
                              fp4q_dtype dq_dtype, cudaStream_t stream);

/*
 * fp4q_glu_bwd -- gradient of h's gate and value, straight through the
 * quantizer: dh is first taken back through the rotation (dh <- R dh, blockwise;
 * R is its own transpose), then du = dh a(g), dg = dh u a'(g),
 * a'(g) = s + g s (1 - s) z'(g), s = sigmoid(z(g)). fp32 throughout, rounded
 * once to bf16. s below 2^-126 counts as zero.
 * gu           bf16 [rows, 2 * cols]; dh bf16 [rows, cols]; cols a multiple of
 *              8 and of rot (of 32 for rot > 0).
 * slots, n     as fp4q_glu_quantize.
 * dgu          bf16 [rows, 2 * cols]; rows not taken stay as they were.
 */
fp4q_status fp4q_glu_bwd(const void* gu, const void* dh, int64_t rows, int64_t cols,
                         const int32_t* slots, int64_t n, fp4q_activation act, int rot, void* dgu,
                         cudaStream_t stream);

/*
 * fp4q_expert_combine -- out[t] = R sum_j weights[t, j] * y[slots[t, j]], the
 * sum in fp32 with j ascending, one fused multiply-add a term (a sum of the
 * rows for weights NULL), rounded once. Dropped choices add nothing (their
 * weight is not read); a token with none left gives zeros.
 * With weights NULL and the rot of the forward call this is the gradient of
 * fp4q_expert_quantize with respect to x, straight through its rounding.
 * y            [rows, cols] of y_dtype; cols a multiple of 8, and of rot.
 * slots        int32 [tokens, k]; a value outside 0 .. rows-1 counts as dropped.
 * weights      fp32 [tokens, k] or NULL. out [tokens, cols] of out_dtype.
 */
fp4q_status fp4q_expert_combine(const void* y, fp4q_dtype y_dtype, int64_t rows, int64_t cols,
                                const int32_t* slots, int64_t tokens, int k, const float* weights,
                                int rot, void* out, fp4q_dtype out_dtype, cudaStream_t stream);

/*
 * fp4q_expert_combine_bwd -- gradients of fp4q_expert_combine (rot 0):
 * dy[slots[t, j]] = weights[t, j] * g[t] (one rounding), dweights[t, j] =
 * <g[t], y[slots[t, j]]>, summed in 64 bits and rounded once (0 for a dropped choice).
 * g            [tokens, cols] of g_dtype; y, dy [rows, cols] of y_dtype. y and
 *              dweights may both be NULL, to leave dweights out; weights NULL counts as
 *              ones. Rows of dy without a choice stay as they were.
 */
fp4q_status fp4q_expert_combine_bwd(const void* g, fp4q_dtype g_dtype, const void* y,
                                    fp4q_dtype y_dtype, int64_t rows, int64_t cols,
                                    const int32_t* slots, int64_t tokens, int k,
                                    const float* weights, void* dy, float* dweights,
                                    cudaStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* FP4Q_EXPERTS_H */
