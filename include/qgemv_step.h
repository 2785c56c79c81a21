/*
 * qgemv_step.h -- C ABI of libqgemv.so, third part: what a decoder step does
 * around its products (qgemv.h) and its attention (qgemv_attn.h): the norm in
 * front of a product, with its result in 16 bits or in 8 bits for a W4A8
 * product, and the choice of the next token.
 *
 * Conventions of qgemv.h hold: [dev] pointers, the caller owns every buffer,
 * calls enqueue kernels on `stream` and return at once (no allocation, no
 * synchronization, no memset or copy nodes, so they can be captured in a HIP
 * graph), arguments are checked before anything is enqueued, and a failing
 * call enqueues nothing.  Data on the device is not validated on the host; any
 * value there gives a result, never an access outside the caller's buffers.
 * Results are deterministic.
 */
#ifndef QGEMV_STEP_H
#define QGEMV_STEP_H

#include "qgemv_attn.h"

#ifdef __cplusplus
extern "C" {
#endif

/* A [rows, dim] array whose last dimension is contiguous: element (r, d) is
 * data[r * row + d], row in elements, not negative; that of a single row is not
 * looked at.  Any alignment of whole elements (16-byte aligned data, row and
 * dim multiples of 8 are faster). */
typedef struct {
  uint16_t *data;
  int64_t row;
} qgemv_rows;

/* ------------------------------------------------------------------------
 * Root-mean-square norm, with the residual's addition:
 *     h[r, d] = x[r, d] + residual[r, d]      (x[r, d] without residual)
 *     y[r, d] = h[r, d] * weight[d] / sqrt(sum_d h[r, d]^2 / dim + eps)
 *   dtype     QGEMV_F16 or QGEMV_BF16, of all arrays
 *   residual, sum [dev]  both or neither NULL; sum takes h, rounded once (y is
 *             computed from h as it is before that)
 *   weight [dev] [dim]
 *   eps       finite and not negative
 * Sums are in fp32: rows whose squares add up past its range, or that hold
 * infinities or NaN, have 0 or NaN in y, as the formula gives in fp32.
 *
 * y may be x or residual, and sum may be x or residual (the same data and
 * stride); apart from that y, sum and what is read may not overlap (VALUE), and
 * rows of y and sum may not overlap each other (SHAPE).  rows of 0 does
 * nothing; 1 <= dim <= 2^24 (SHAPE otherwise).  Checks, in order: null, dtype
 * (UNSUPPORTED), shape, eps (VALUE), alignment, overlap.
 * ------------------------------------------------------------------------ */
int qgemv_rms_norm(int dtype, int rows, int dim, float eps, const qgemv_rows *x, const qgemv_rows *residual,
                   const uint16_t *weight, const qgemv_rows *sum, const qgemv_rows *y, qgemv_stream_t stream);

/* The same with y in 8 bits, as qgemv_w4a8_rows takes it:
 *     step[r] = max_d |y[r, d]| / 127,  y8[r, d] = rint(y[r, d] / step[r])
 * from y in fp32 (it is not rounded to 16 bits first).  A row whose y is 0
 * throughout has step 0 and codes 0; one whose y is not finite throughout (zeros
 * with an eps of 0 among them) has step NaN and codes 0.
 *   y8 [dev]    int8 [rows][dim]
 *   step [dev]  fp32 [rows]
 * y8 and step may not overlap anything else (VALUE). */
int qgemv_rms_norm_q8(int dtype, int rows, int dim, float eps, const qgemv_rows *x, const qgemv_rows *residual,
                      const uint16_t *weight, const qgemv_rows *sum, int8_t *y8, float *step, qgemv_stream_t stream);

/* qgemv_w4a8 for activations that are in 8 bits already:
 *     y[m, n] = step[m] * sum_k s[n, k/128] * (q[n, k] - z[n, k/128]) * x8[m, k]
 * the same kernel and rules, without the pass that makes x8 and step and so
 * without a workspace.  x8 is int8 [M][K], 16-byte aligned; step fp32 [M],
 * 4-byte aligned. */
int qgemv_w4a8_rows(int M, int N, int K, const int8_t *x8, const float *step, const uint32_t *wq,
                    const uint16_t *scales, const uint32_t *zeros, uint16_t *y, qgemv_stream_t stream);

/* ------------------------------------------------------------------------
 * The next token of every row.  With M the row's largest logit and
 * w[i] = exp((l[i] - M) / T), the tokens in the order of falling logits, equal
 * ones by rising index, are cut to
 *   top_k  the first top_k,
 *   top_p  of those, with S the sum of their weights, each that has less than
 *          top_p * S in front of it,
 *   min_p  of those, each with w >= min_p;
 * the first always stays.  token[r] is the first one, now by rising index, for
 * which the kept weights up to and with it exceed u[r] times their sum.
 *
 *   type        QGEMV_F16, QGEMV_BF16 or QGEMV_F32, of the logits
 *   logits [dev] [rows][vocab], rows `row` elements apart (not looked at for a
 *               single row), aligned to an element
 *   u [dev]     fp32 [rows], in [0, 1); smaller ones and NaN count as 0, larger
 *               ones as the largest below 1
 *   temperature, top_p, min_p [dev] fp32 [rows], top_k [dev] int32 [rows]; each
 *               may be NULL: T = 1, off.  T not above 0 (or NaN): the row's
 *               largest logit, the first of equal ones.  top_k below 1, top_p
 *               of 1 and more and min_p of 0 and less, and NaN: off; top_p below
 *               0 counts as 0, min_p above 1 as 1.
 *   token [dev] int32 [rows]; -1 where no logit is above -infinity
 *   ws [dev]    scratch of qgemv_sample_workspace_bytes bytes, 16-byte aligned,
 *               no initial contents; calls that share it must not overlap in time
 * Logits of -infinity, and NaN, are never chosen; of a row with infinities only
 * these are.  Weights are held to 2^-42 of the largest (smaller ones round to 0
 * or that), worked out in 64 bits; they add up exactly.
 *
 * 1 <= vocab <= 2^21, rows below 2^21 and rows * ceil(vocab / 16384) below 2^23
 * (SHAPE otherwise, and a workspace size of 0); row not negative, at most 2^40, and
 * rows * row at most 2 * 10^17 (SHAPE).  rows of 0 does nothing.  Checks, in order:
 * null, type (UNSUPPORTED), shape, alignment, overlap of token or ws with anything
 * else (VALUE), workspace.
 * ------------------------------------------------------------------------ */
#define QGEMV_F32 2
size_t qgemv_sample_workspace_bytes(int rows, int vocab);
int qgemv_sample(int type, int rows, int vocab, const void *logits, int64_t row, const float *u,
                 const float *temperature, const int32_t *top_k, const float *top_p, const float *min_p,
                 int32_t *token, void *ws, size_t ws_bytes, qgemv_stream_t stream);

#ifdef __cplusplus
}
#endif
#endif /* QGEMV_STEP_H */
