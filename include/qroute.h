/*
 * qroute.h — C ABI of the routed calls of the MI355X (gfx950) library: rows
 * that each go through one of several weight sets (the experts of a mixture,
 * MUL_MAT_ID of "metal: TQ1_0 kernel performance", section "Correctness"; the
 * low-rank adapters of many requests).
 *
 * A routed step has T tokens with k choices each: slot s = t*k + j is token
 * t's choice j, n = T*k slots in all.  qroute_sort turns the router's ids
 * into a plan, the other calls read it:
 *     offsets[e] .. offsets[e+1]   the sorted positions of weight set e
 *                                  (int32, E + 1 of them; offsets[E] = the
 *                                  number of slots that name a weight set)
 *     order[p]                     the slot at sorted position p, or -1 - slot
 *                                  for p >= offsets[E] (slots that name none)
 *     position[s]                  the inverse: slot s's sorted position, or
 *                                  -1 when it names no weight set
 *
 * Conventions are those of qgemv.h (device memory owned by the caller, 16-byte
 * alignment of matrices and rows, element alignment of vectors, work enqueued
 * on `stream`, host validation with negative QGEMV_E_* codes, nothing
 * allocated, no synchronisation).  The plan is device data and is not checked
 * on the host: entries that no qroute_sort writes (positions, slots or offsets
 * outside their ranges) never lead to an access outside the arrays, and give
 * unspecified values.  All results are the same bits on every run.
 * Limits: k <= 64, E <= 1024, n <= 2^24; the row movers take T*k*(C + 16) <= 2^35.
 * A product whose launch would take 2^32 work items or more is QGEMV_E_SHAPE: none does
 * while ceil(M / 64) * (T*k / 16 + min(T*k, E)) < 2^23.
 */
#ifndef QROUTE_H
#define QROUTE_H

#include "qgemv.h"

#ifdef __cplusplus
extern "C" {
#endif

#define QROUTE_MAX_E 1024
#define QROUTE_MAX_K 64
#define QROUTE_MAX_N (1 << 24)
#define QLORA_MAX_R 256

/* The plan of n slots over E >= 1 weight sets: a stable sort by ids[s] (slots
 * of one weight set keep their order).  An id outside [0, E) names no weight
 * set (padding tokens, requests without an adapter).  With n == 0 only
 * offsets is written (all zero), and the other pointers may be NULL.
 *   ids                       n int32
 *   order, position, offsets  n, n and E + 1 int32, all written whole; they
 *                             must not overlap ids or each other.
 *   workspace                 qroute_workspace_bytes(n, E) bytes, 256-byte
 *                             aligned (0 bytes: may be NULL); contents need
 *                             no initialisation and are overwritten, so calls
 *                             that overlap in time must not share it. */
int64_t qroute_workspace_bytes(int64_t n, int64_t E);
int qroute_sort(const int32_t* ids, int64_t n, int64_t E, int32_t* order, int32_t* position, int32_t* offsets,
                void* workspace, int64_t workspace_bytes, struct ihipStream_t* stream);

/* Rows into sorted order: out[p] = weights[order[p]] * x[order[p] / k] for every
 * p with order[p] >= 0 (one fp32 product, rounded once to the type).
 *   x        [T][C] of dtype;  out [T*k][C] of the same dtype.
 *   weights  [T][k] fp32, or NULL for plain copies (bit for bit).
 * Rows of out whose order[p] is negative are left as they were.  It is also
 * the gradient of a sum over choices, taken back to its rows. */
int qroute_gather(const void* x, const int32_t* order, const float* weights, void* out, int32_t dtype, int64_t T,
                  int64_t k, int64_t C, struct ihipStream_t* stream);

/* Rows back to their tokens: y[t] = sum_j weights[t][j] * rows[position[t*k+j]],
 * choices in ascending order, fp32 sums, one rounding to y_dtype.  Choices
 * with position -1 add nothing (their weights and rows are not read into the
 * sum); a token whose choices all do gets a zero row.
 *   rows     [T*k][C] of rows_dtype;  y [T][C] of y_dtype.
 *   weights  [T][k] fp32, or NULL for a plain sum (the gradient of
 *            qroute_gather without weights). */
int qroute_combine(const void* rows, int32_t rows_dtype, const int32_t* position, const float* weights, void* y,
                   int32_t y_dtype, int64_t T, int64_t k, int64_t C, struct ihipStream_t* stream);

/* Gradient of qroute_combine with weights: for every choice with a position
 *     drows[position[t*k+j]] = weights[t][j] * dy[t]        (rows_dtype)
 *     dweights[t][j] = sum_c dy[t][c] * rows[position[t*k+j]][c]   (fp32)
 * and dweights[t][j] = 0 for the others.  Rows of drows that no choice has a
 * position in are left as they were.
 *   dy  [T][C] of dy_dtype;  rows, drows  [T*k][C] of rows_dtype. */
int qroute_combine_grad(const void* dy, int32_t dy_dtype, const void* rows, int32_t rows_dtype,
                        const int32_t* position, const float* weights, void* drows, float* dweights, int64_t T,
                        int64_t k, int64_t C, struct ihipStream_t* stream);

/* Routed products (MUL_MAT_ID): y[p] = x[row(p)] . dequant(W_e)^T for every
 * weight set e and sorted position offsets[e] <= p < offsets[e+1].
 *   w        E packed matrices of M rows and K columns, one after the other,
 *            each laid out as for the GEMV of the format (qgemv.h).
 *   order    row(p) = order[p] / k: x is [T][K], one row a token (the first
 *            product of an expert).  NULL: row(p) = p, x is [T*k][K] in sorted
 *            order (the second).  x is fp16, for NVFP4 bf16.
 *   y        [T*k][M] of y_dtype, 16-byte aligned.  Rows that no weight set
 *            has are left as they were.
 * Sums are in fp32, each output is rounded once to y_dtype, and weights are never
 * rounded: NVFP4's and TQ1_0's are exact in 16 bits, and Q4_K enters as
 * d * sum(scale * q * x) - dmin * sum(min * x) over each block.  Infinite and NaN
 * activations and scales give what sum(weight * x) gives, in their own tokens' and rows'
 * outputs alone.
 * K as for the prefill (K <= 2^20, NVFP4 K % 64 == 0), M <= 2^24, and with
 * `order` x spans at most 2^30 bytes.  T == 0 or M == 0 is a no-op. */
int qgemm_q4k_routed(const void* w, const void* x_f16, const int32_t* order, const int32_t* offsets, void* y,
                     int32_t y_dtype, int64_t T, int64_t k, int64_t E, int64_t M, int64_t K,
                     struct ihipStream_t* stream);
int qgemm_nvfp4_routed(const void* w, const void* x_bf16, const int32_t* order, const int32_t* offsets, void* y,
                       int32_t y_dtype, int64_t T, int64_t k, int64_t E, int64_t M, int64_t K,
                       struct ihipStream_t* stream);
int qgemm_tq1_routed(const void* w, const void* x_f16, const int32_t* order, const int32_t* offsets, void* y,
                     int32_t y_dtype, int64_t T, int64_t k, int64_t E, int64_t M, int64_t K,
                     struct ihipStream_t* stream);

/* Low-rank adapters of many requests beside one shared projection: with the
 * plan of T slots (k = 1) over E adapters, for every token t
 *     y[t] = c[t] + scale[e] * B_e (A_e x[t])     t names adapter e
 *     y[t] = c[t]                                 t names none
 *   x        [T][K], fp16 (qlora_f16) or bf16 (qlora_bf16).
 *   a, b     [E][r][K] and [E][M][r] of x's type (adapters of a smaller rank
 *            are padded with zero rows of A or columns of B).
 *   scale    E fp32, or NULL for 1.
 *   c, y     [T][M] of y_dtype, 16-byte aligned.  c is the projection's
 *            output and may be y itself (in place: rows that name no adapter
 *            are then not touched); any other overlap is QGEMV_E_ALIAS.  c may
 *            be NULL for zero.
 *   workspace  qlora_workspace_bytes(T, E, r, M, K) bytes, 256-byte aligned;
 *            contents need no initialisation and are overwritten, so calls
 *            that overlap in time must not share it.
 * A_e x[t] is kept in fp32 (qlora_f16: bit for bit down to 2^-39 of the token's
 * largest component, smaller ones to 2^-63 of it) and the sum is rounded once to
 * y_dtype.  An infinite element of b gives NaN.
 * 0 < r <= 256, r % 8 == 0; K % 8 == 0, K <= 2^20; M <= 2^24; x spans at most
 * 2^30 bytes.  T == 0 or M == 0 is a no-op. */
int64_t qlora_workspace_bytes(int64_t T, int64_t E, int64_t r, int64_t M, int64_t K);
int qlora_f16(const void* x_f16, const void* a_f16, const void* b_f16, const float* scale, const int32_t* order,
              const int32_t* offsets, const void* c, void* y, int32_t y_dtype, int64_t T, int64_t E, int64_t r,
              int64_t M, int64_t K, void* workspace, int64_t workspace_bytes, struct ihipStream_t* stream);
int qlora_bf16(const void* x_bf16, const void* a_bf16, const void* b_bf16, const float* scale, const int32_t* order,
               const int32_t* offsets, const void* c, void* y, int32_t y_dtype, int64_t T, int64_t E, int64_t r,
               int64_t M, int64_t K, void* workspace, int64_t workspace_bytes, struct ihipStream_t* stream);

#ifdef __cplusplus
}
#endif

#endif /* QROUTE_H */
