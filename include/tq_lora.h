/*
 * tq_lora.h -- C ABI of libtq.so, low-rank adapters beside the packed projections: the adapters' rows
 * of many requests at once, their gradients, dropout from a counter-based generator, and the packed
 * products' gradient for x.
 *
 * The conventions of tq.h hold (device pointers owned by the caller, row-major contiguous tensors,
 * asynchronous on `stream` and the current device, argument errors returned before anything is
 * launched, no allocation, graph capturable), with one difference: the kernels here read nothing,
 * weights included, before the preceding work on the stream has finished.
 *
 * A frozen projection shared by all requests and L adapters of rank r:
 *
 *   y [M, N]    = x What^T                                   tq_gemm / w4g_gemm
 *   out[m]      = y[m] + s_l (drop(x[m]) A_l^T) B_l^T        tq_lora,  l the adapter of row m
 *
 * and, from dy [M, N], a training step's gradients:
 *
 *   dx [M, K]   = dy What                                    tq_gemm_backward / w4g_gemm_backward
 *   dx, dA, dB  of the adapters, dx added to the above       tq_lora_backward
 *
 * The adapter of each row comes as a plan that all layers of a step share: tq_moe_sort of the rows'
 * adapter ids (a slot is a row here, top_k = 1) gives
 *   order    int32 [M]: the row at each sorted position, rows of adapter 0 first, or NULL: row = position;
 *   offsets  int32 [L + 1], non-decreasing, within [0, M]: adapter l has the positions from offsets[l] to
 *            offsets[l + 1] - 1.
 * Positions before offsets[0] and from offsets[L] on belong to no adapter: their rows get the base alone.
 * The rows that `order` names are distinct; an entry outside [0, M) names no row.
 *
 * Types: x, A, B, base, out, dy and the gradients have one dtype, TQ_F16 or TQ_BF16 (the packed products and their
 * gradient for x are fp16: beside them bf16 adapters need base and base_dx as bf16 copies).  Sums are in fp32, v and dv
 * are kept in fp32, and every output is rounded once.  Where v and dv enter a tensor-core product, each is
 * the sum of two 16-bit numbers, off by at most 2^-22 (fp16) or 2^-16 (bf16) of it; in dA and dB of fp16, where one
 * power of two serves all of an adapter's numbers, by 2^-39 of the largest finite one where that is more (what is
 * below 2^-17 of the largest loses bits).
 * A tensor core adds up to 16 products at a time and cuts the fp32 sum off instead of rounding it, by less than a unit
 * in the last place: on PREFILL and DECODE a sum of n products is off by at most n 2^-27 of its largest partial sum,
 * toward zero.  Measured on v, fp16, most of 4096 elements, of that partial sum: 2.8e-5 for n = 4096 terms of one sign,
 * 3.5e-5 for 16384, 7.9e-5 for 65536 (a split over CTAs makes the parts shorter); of random sign 0.7e-5, 1.6e-5 and
 * 4.1e-5.  GENERIC rounds each addition.
 *
 * Numbers that are not finite: an output element in whose formula they do not occur is as without them; one that the
 * formula makes infinite or NaN is not finite, but an infinity may come as NaN (on PREFILL and DECODE an infinite
 * operand meets both parts of v or dv, which may differ in sign or be zero).
 *
 * Dropout: element e = k % 8 of the group i = m ceil(K / 8) + k / 8 of x [M, K] takes the 16 bits
 *   (e even: low half, odd: high half) of word e / 2 of Philox4x32-10 (Salmon, Moraes, Dror, Shaw: Parallel
 *   random numbers: as easy as 1, 2, 3; SC 2011) with the counter (i, offset) and the key seed, 64 bits
 *   each, low word first.  It is dropped where they are below T = floor(65536 p + 1/2); what is kept is
 *   multiplied by 65536 / (65536 - T).  A dropped element is zero whatever it holds.  No mask is stored:
 *   every call that names the same p, seed, offset and shape drops the same elements.
 *   rng      int64 [2] on the device: seed, offset.  A captured graph reads it when it runs, so that a
 *            kernel which advances the offset between replays gives each its own mask.
 *   0 <= p < 1 and T <= 65535 (TQ_ERR_SHAPE otherwise); p = 0 reads no rng (it may be NULL).
 */
#ifndef TQ_LORA_H
#define TQ_LORA_H

#include "tq_moe.h"

#ifdef __cplusplus
extern "C" {
#endif

#define TQ_LORA_MAX_ADAPTERS 1024
#define TQ_LORA_MAX_RANK 128

/* --------------------------------------------------------------------------------------------
 * tq_lora -- out[m] = base[m] + scaling[l] (drop(x[m]) A_l^T) B_l^T.
 *
 *   x        [M, K]
 *   a        [L, rank, K], b [L, N, rank].  A rank above 128 is the sum of two calls, the second with
 *            the first's out as base.
 *   scaling  fp32 [L], or NULL for 1
 *   base     [M, N], or NULL for zeros; may be `out`
 *   out      [M, N], written in full.  Must not overlap x, a or b.
 *   v        fp32 [M, rank], or NULL: drop(x) A^T by sorted position, without `scaling`, written for
 *            the positions of adapters; tq_lora_backward reads it.  PREFILL and GENERIC need it
 *            (TQ_ERR_NULL); AUTO without it takes DECODE where it can, however many rows there are: give
 *            it for more than a few rows per adapter, since DECODE reads an adapter's weights once per eight.
 *            Calls (or captured graphs) that may run at once need one each.
 *   path     TQ_PATH_AUTO, or one path (tests): DECODE takes few rows (one launch, up to 8 rows of an
 *            adapter per pass over its weights), PREFILL many (tensor cores), GENERIC is the plain form.
 *            DECODE needs p = 0, M <= 65535, K % 8 == 0 and N % 8 == 0 (TQ_ERR_PATH) and 16-byte aligned x, a, b, base,
 *            out and v (TQ_ERR_ALIGN).  PREFILL needs a 16-byte aligned v (TQ_ERR_ALIGN); widths that are multiples
 *            of 8 and aligned tensors are read in whole vectors, others element by element.
 *            Every path is right for any numbers of rows per adapter.
 * 1 <= L <= 1024, 1 <= rank <= 128, 0 < K, N <= 2^24 (N = 0: nothing), 0 <= M < 2^31.
 * M == 0 or N == 0: nothing is launched.
 *
 * tq_lora_path -- the rule TQ_PATH_AUTO applies with a v (host arithmetic only; aligned16: all of the pointers
 * that are not NULL are 16-byte aligned).  Returns a tq_path or a negative tq_status.
 * ------------------------------------------------------------------------------------------ */
TQ_API int tq_lora(const void* x, int dtype, const void* a, const void* b, const float* scaling, const void* base,
                   void* out, float* v, const int32_t* offsets, const int32_t* order, double p, const int64_t* rng,
                   int64_t M, int64_t L, int64_t N, int64_t K, int rank, int path, void* stream);
TQ_API int tq_lora_path(int64_t M, int64_t L, int64_t N, int64_t K, int rank, int dropout, int aligned16);

/* --------------------------------------------------------------------------------------------
 * tq_lora_backward -- the gradients of tq_lora, from dy [M, N] and the forward call's x, a, b, scaling,
 * plan, p, rng and v:
 *   dv[r]    = scaling[l] dy[m] B_l              fp32 [M, rank], by sorted position, in the workspace
 *   dx[m]    = base_dx[m] + drop'(dv[r] A_l)     drop': zero where drop(x) dropped, else times the same factor
 *   da_l     = sum over its rows of dv[r]^T drop(x[m])             [L, rank, K]
 *   db_l     = scaling[l] sum over its rows of dy[m]^T v[r]        [L, N, rank]
 *   (r: sorted position, m: its row).  An adapter without rows gets zeros.
 *   v        fp32 [M, rank], as tq_lora left it
 *   workspace  tq_lora_workspace_size() bytes or more (TQ_ERR_SHAPE), 16-byte aligned (TQ_ERR_ALIGN); nothing in it
 *            lasts from call to call.  Calls (or captured graphs) that may run at once need one each.
 *   base_dx  [M, K], or NULL for zeros; may be `dx` (the projection's own gradient for x, to which this adds)
 *   dx, da, db  each may be NULL (not wanted).  None may overlap what the call reads (dx may be base_dx).
 *   path     AUTO, PREFILL (16-byte aligned v: TQ_ERR_ALIGN) or GENERIC.
 * The gradient for base is dy itself; `scaling` has none.  Sums are taken in a fixed order.
 * ------------------------------------------------------------------------------------------ */
TQ_API int tq_lora_backward(const void* dy, const void* x, int dtype, const void* a, const void* b,
                            const float* scaling, const float* v, void* workspace, size_t workspace_bytes,
                            const void* base_dx, void* dx, void* da, void* db, const int32_t* offsets,
                            const int32_t* order, double p, const int64_t* rng, int64_t M, int64_t L, int64_t N,
                            int64_t K, int rank, int path, void* stream);

/* Bytes of workspace that tq_lora_backward needs (host arithmetic only; 0: invalid sizes). */
TQ_API size_t tq_lora_workspace_size(int64_t M, int64_t L, int rank);

/* --------------------------------------------------------------------------------------------
 * tq_dropout -- out = drop(x), x and out [M, K] of `dtype` (TQ_F32, TQ_F16, TQ_BF16); out may be x.  Its
 * gradient is the same call on the gradient of out.
 * 0 <= M < 2^31, 0 <= K <= 2^28.
 * ------------------------------------------------------------------------------------------ */
TQ_API int tq_dropout(const void* x, int dtype, void* out, double p, const int64_t* rng, int64_t M, int64_t K,
                      void* stream);

/* --------------------------------------------------------------------------------------------
 * tq_gemm_backward / w4g_gemm_backward -- dx = dy What, the gradient for x of tq_gemm / w4g_gemm / w4g_gemm_zp
 * (that of bias is the sum of dy's rows; the packed weights have none).
 * A matrix in activation order (w4g_repack_act_order) gives the gradient of the permuted columns x_out[m, j] = x[m,
 * perm[j]]: tq_permute_columns with the inverse permutation (inv[perm[j]] = j) makes it that of x.
 *   dy       fp16 [M, N]
 *   packed, scale / qweight, scales, zeros   as in the products (zeros NULL: symmetric, else 0 .. 15)
 *   dx       fp16 [M, K], written in full.  Must not overlap dy.
 *   rows     fp16 [M, N rounded up to a multiple of 8] scratch, 16-byte aligned, or NULL: PREFILL copies the rows of
 *            dy there first where N % 8 != 0 or dy is not 16-byte aligned (without it: AUTO takes GENERIC, PREFILL
 *            returns TQ_ERR_NULL).  Not read or written otherwise.  Calls that may run at once need one each.
 *   path     TQ_PATH_AUTO, PREFILL (tensor cores) or GENERIC (any shape and alignment; weights enter the sum
 *            exactly).  PREFILL needs K % 64 == 0 (TQ_ERR_PATH) and 16-byte aligned weights and dx (TQ_ERR_ALIGN).
 *            There a ternary weight enters exactly and an INT4 weight (u - z) s is rounded to fp16, as on that path
 *            of w4g_gemm (scales must keep it below 65520): dx is 2.7e-4 off relative rms where its own
 *            rounding alone makes 2.1e-4.
 * Shapes and errors as in tq_gemm / w4g_gemm.
 * ------------------------------------------------------------------------------------------ */
TQ_API int tq_gemm_backward(const uint16_t* dy, const uint8_t* packed, const uint16_t* scale, uint16_t* dx,
                            uint16_t* rows, int64_t M, int64_t N, int64_t K, int path, void* stream);
TQ_API int w4g_gemm_backward(const uint16_t* dy, const int32_t* qweight, const uint16_t* scales, const uint8_t* zeros,
                             uint16_t* dx, uint16_t* rows, int64_t M, int64_t N, int64_t K, int path,
                             void* stream);

#ifdef __cplusplus
}
#endif

#endif /* TQ_LORA_H */
