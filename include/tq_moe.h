/*
 * tq_moe.h -- C ABI of libtq.so, mixture-of-experts calls: the router, the exchange of rows
 * between tokens and experts, and the experts' products with packed low-bit weights.
 *
 * The conventions of tq.h hold (device pointers owned by the caller, row-major contiguous
 * tensors, asynchronous on `stream` and the current device, argument errors returned before
 * anything is launched, no allocation, graph capturable), with one difference: the kernels here
 * read nothing, weights included, before the preceding work on the stream has finished.
 *
 * A layer of E experts, T tokens and top_k choices per token runs
 *
 *   tq_moe_route      scores [T, E]  ->  weights [T, top_k], ids [T, top_k]
 *   tq_moe_sort       ids            ->  offsets [E + 1], order [R], pos [T, top_k],  R = T top_k
 *   w4g_gemm_experts / tq_gemm_experts   x [T, K] read through `order`  ->  y [R, N], by expert
 *   (activation, second product on the sorted rows)
 *   tq_moe_combine    y [R, H], pos, weights  ->  out [T, H]
 *
 * or, with the rows copied first, tq_moe_gather and the products without `order`.  A slot is a
 * (token, choice) pair, numbered token * top_k + choice.  A slot whose id is outside [0, E)
 * belongs to no expert here (a rank of an expert-parallel group subtracts its first expert from
 * the ids): it is sorted last, has position -1, and takes part in nothing.
 *
 * Types: TQ_F32, TQ_F16 and TQ_BF16 for scores and rows (`dtype`); the products are fp16 as in
 * tq.h.  Sums are in fp32; every output is rounded once.  The one rounding besides is that of the
 * INT4 weights on the PREFILL path (below).
 */
#ifndef TQ_MOE_H
#define TQ_MOE_H

#include "tq.h"

#ifdef __cplusplus
extern "C" {
#endif

/* tq_dtype of the calls in this header only (the others return TQ_ERR_DTYPE for it). */
enum { TQ_BF16 = 2 };

#define TQ_MOE_MAX_EXPERTS 1024
#define TQ_MOE_MAX_TOP_K 32

/* --------------------------------------------------------------------------------------------
 * tq_moe_route -- softmax over the experts and the top_k of each token.
 *
 *   logits   [T, E] of `dtype`.  -inf marks an expert that may not be chosen; a NaN counts as
 *            -inf; +inf entries share the whole probability.
 *   weights  [T, top_k] fp32, written: p[t, ids[t, j]], p = softmax(logits[t]); with
 *            `renormalize` divided by their sum (the softmax over the chosen experts).
 *   ids      [T, top_k] int32, written: the experts in decreasing order of their logits, the
 *            lowest index first among equals.  A row with fewer than top_k experts above -inf
 *            ends in ids of -1 with weight 0.
 * 1 <= E <= 1024, 1 <= top_k <= min(E, 32), T top_k < 2^31.
 *
 * tq_moe_route_backward -- dlogits [T, E] of `dtype`, written in full, from dweights [T, top_k]
 * fp32 and the forward call's logits, weights and ids:
 *   renormalize:  dlogits[i] = w_j (g_j - sum g w) for i = ids[j], 0 elsewhere;
 *   otherwise:    dlogits[i] = p_i (g[i] - sum g w), g[i] = g_j for i = ids[j] and 0 elsewhere.
 * The chosen ids of a token are distinct; ids outside [0, E) are skipped.
 * ------------------------------------------------------------------------------------------ */
TQ_API int tq_moe_route(const void* logits, int dtype, float* weights, int32_t* ids, int64_t T,
                        int64_t E, int top_k, int renormalize, void* stream);
TQ_API int tq_moe_route_backward(const float* dweights, const void* logits, int dtype,
                                 const float* weights, const int32_t* ids, void* dlogits,
                                 int64_t T, int64_t E, int top_k, int renormalize, void* stream);

/* --------------------------------------------------------------------------------------------
 * tq_moe_sort -- slots sorted by expert, in slot order within an expert (the same result on
 * every run).
 *
 *   ids      [R] int32 (the [T, top_k] ids in a row).
 *   offsets  [E + 1] int32, written: expert e has sorted rows offsets[e] .. offsets[e + 1] - 1.
 *   order    [R] int32, written: the slot of each sorted row; slots of no expert come after
 *            offsets[E], in slot order.
 *   pos      [R] int32, written: the sorted row of each slot, -1 for slots of no expert.
 * 1 <= E <= 1024, 0 <= R < 2^31 (R = 0 writes offsets only).
 * ------------------------------------------------------------------------------------------ */
TQ_API int tq_moe_sort(const int32_t* ids, int32_t* offsets, int32_t* order, int32_t* pos,
                       int64_t R, int64_t E, void* stream);

/* --------------------------------------------------------------------------------------------
 * tq_moe_gather -- rows[r] = x[order[r] / top_k] for r < offsets[E]; rows from offsets[E] on are
 * left as they were, and so is a row whose order is not a slot of the T tokens.
 *   x [T, H], rows [T top_k, H], both of `dtype`, not overlapping; order and offsets from
 *   tq_moe_sort.  Its gradient is tq_moe_combine without weights: dx[t] = sum_j drows[pos[t, j]].
 *
 * tq_moe_combine -- out[t] = sum_j weights[t, j] y[pos[t, j]] over the slots with a row, summed
 * in fp32 in the order of j; zeros for a token without any.
 *   y [R, H] and out [T, H] of `dtype`, not overlapping; pos [T, top_k] int32 (positions outside
 *   [0, R) are skipped); weights [T, top_k] fp32, or NULL for 1.
 *
 * tq_moe_combine_backward -- from dout [T, H]:
 *   dy[pos[t, j]]   = weights[t, j] dout[t]       (rows of y that no slot names are left as they were)
 *   dweights[t, j]  = sum_h dout[t, h] y[pos[t, j], h]     (fp32; 0 for a slot without a row)
 *   dy or dweights may be NULL (not wanted; y is read for dweights only, weights for dy only).
 *   Positions of different slots are distinct.  dy must not overlap y or dout.
 * 1 <= H <= 2^24, 1 <= top_k <= 32, T top_k < 2^31, 0 <= R < 2^31.
 * ------------------------------------------------------------------------------------------ */
TQ_API int tq_moe_gather(const void* x, int dtype, const int32_t* order, const int32_t* offsets,
                         void* rows, int64_t T, int64_t H, int top_k, int64_t E, void* stream);
TQ_API int tq_moe_combine(const void* y, int dtype, const int32_t* pos, const float* weights,
                          void* out, int64_t T, int64_t R, int64_t H, int top_k, void* stream);
TQ_API int tq_moe_combine_backward(const void* dout, const void* y, int dtype, const int32_t* pos,
                                   const float* weights, void* dy, float* dweights, int64_t T,
                                   int64_t R, int64_t H, int top_k, void* stream);

/* --------------------------------------------------------------------------------------------
 * tq_gemm_experts / w4g_gemm_experts -- each expert's rows times its packed weights: for
 * e < E and offsets[e] <= r < offsets[e + 1],
 *     y[r, :] = x[row(r), :] . What_e^T (+ bias[e, :]),     row(r) = order ? order[r] / top_k : r
 * What_e as in tq_gemm / w4g_gemm / w4g_gemm_zp (same formats, fp32 accumulation).  Weights enter the
 * sum exactly and the result is rounded once, except on the PREFILL path of w4g_gemm_experts: there, as
 * on that of w4g_gemm, each weight (u - z) s is rounded to fp16 first (2^-11 of its value at most), and
 * one of 65520 and above becomes infinite, so that scales must keep |(u - z) s| below that: any scale up
 * to 4364 does.  AUTO may take that path; DECODE and GENERIC take any scale and round no weight.
 *
 *   x        fp16 [X, K]: X = T tokens with `order`, X = R sorted rows without.
 *   packed   ternary uint8 [E, N, ceil(K/4)] (tq_quantize_pack of the [E N, K] matrix)
 *   scale    fp16 [E, N]
 *   qweight  W4A16 int32 [E, N, K/8] (w4g_quantize_pack of the [E N, K] matrix), K % 128 == 0
 *   scales   fp16 [E, N, K/128]
 *   zeros    uint8 [E, N, K/128], values 0 .. 15, or NULL (symmetric)
 *   bias     fp16 [E, N] or NULL
 *   y        fp16 [R, N], written for offsets[0] <= r < offsets[E]; other rows are left as they
 *            were.  Must not overlap x.
 *   offsets  int32 [E + 1] (tq_moe_sort, or E + 1 consecutive ones of a sort of more experts):
 *            non-decreasing, within [0, R].
 *   order    int32 [R] or NULL; a negative slot or a row(r) past X reads as zeros.
 *   rows     fp16 [R, K] scratch, 16-byte aligned, or NULL: the PREFILL path with `order` copies the
 *            rows there in sorted order before the product.  Without it AUTO takes the DECODE path
 *            (right, slower), and PREFILL returns TQ_ERR_NULL.  Not read or written otherwise.
 *            Calls (or captured graphs) that may run at once need a scratch each.
 *   path     TQ_PATH_AUTO, or one path (tests): DECODE takes few rows per expert (mma.sync on
 *            in-register decode, up to 8 rows of an expert per pass over its weights), PREFILL
 *            many (tcgen05.mma), GENERIC any shape and alignment.  DECODE and PREFILL need
 *            K % 64 == 0 (TQ_ERR_PATH) and 16-byte aligned x, weights and y (TQ_ERR_ALIGN).
 *            Every path is right for any numbers of rows per expert; AUTO goes by the average
 *            R / E, which the host knows.  R counts the slots of other ranks' experts too: a rank
 *            of an expert-parallel group takes the better path by passing what tq_experts_path
 *            returns for the number of rows that it expects.
 * 1 <= E <= 1024, N E <= 2^31 - 1024, 0 < K <= 2^28, top_k >= 1, 0 <= R < 2^31, 0 <= X < 2^31.
 * R == 0 or N == 0: nothing is launched.  Errors as in tq_gemm.
 * ------------------------------------------------------------------------------------------ */
TQ_API int tq_gemm_experts(const uint16_t* x, const uint8_t* packed, const uint16_t* scale,
                           const uint16_t* bias, uint16_t* y, const int32_t* offsets,
                           const int32_t* order, uint16_t* rows, int64_t X, int64_t R, int64_t E,
                           int64_t N, int64_t K, int top_k, int path, void* stream);
TQ_API int w4g_gemm_experts(const uint16_t* x, const int32_t* qweight, const uint16_t* scales,
                            const uint8_t* zeros, const uint16_t* bias, uint16_t* y,
                            const int32_t* offsets, const int32_t* order, uint16_t* rows,
                            int64_t X, int64_t R, int64_t E, int64_t N, int64_t K, int top_k,
                            int path, void* stream);

/* tq_experts_path -- the rule TQ_PATH_AUTO applies to R rows (host arithmetic only; fmt is a
 * tq_format; aligned16: x, weights and y are 16-byte aligned).  Returns a tq_path or a negative tq_status. */
TQ_API int tq_experts_path(int fmt, int64_t R, int64_t E, int64_t N, int64_t K, int aligned16);

#ifdef __cplusplus
}
#endif

#endif /* TQ_MOE_H */
