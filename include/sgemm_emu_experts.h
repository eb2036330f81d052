/*
 * sgemm_emu_experts.h -- C ABI of libsgemm_emu's operators of feed-forward
 * experts and of weights held in 4 bits: tokens sorted by expert and back,
 * the experts' products with their gradients, products with 4-bit weights.
 *
 * Conventions, types and statuses are those of sgemm_emu_ops.h.  Further:
 *   pairs      a token t and its choice j (T tokens, k choices each) are the pair
 *              t k + j; P = T k.  ids[pair] is the expert, in [0, n); a pair with
 *              another id (a padded token's) comes nowhere.
 *   sorted     the pairs in the order of their experts, inside an expert in their
 *   rows       own: expert e's rows are [offsets[e], offsets[e + 1]); rows from
 *              offsets[n] on, as many as pairs come nowhere, belong to none.
 *              Outputs on sorted rows are zeros there, and what inputs hold there
 *              does not matter.
 *   arrays     offsets (n + 1), pairs (P: sorted row -> pair, -1 behind the last)
 *              and places (P: pair -> sorted row, -1: none) are int32 on the
 *              device, as sgemm_emu_sort_tokens writes them.  Entries outside
 *              [0, P] never lead outside the operands.
 *   limits     P, N, K up to 4,194,240; n up to SGEMM_EMU_MAX_EXPERTS; n N K up to
 *              2^55.
 * No call here takes memory but its arguments, so all can be captured into graphs.
 */
#ifndef SGEMM_EMU_EXPERTS_H
#define SGEMM_EMU_EXPERTS_H

#include "sgemm_emu_ops.h"

#ifdef __cplusplus
extern "C" {
#endif

#define SGEMM_EMU_MAX_EXPERTS 1024
#define SGEMM_EMU_GATE_NONE (-1)   /* a product without a gate */

/*
 * sgemm_emu_sort_tokens -- offsets, pairs and places of P pairs' ids.
 */
int64_t sgemm_emu_sort_tokens_workspace(int64_t P, int64_t n);
int sgemm_emu_sort_tokens(int64_t P, int64_t n, const int32_t *ids, int32_t *offsets, int32_t *pairs, int32_t *places,
                          void *ws, int64_t ws_bytes, sgemm_emu_stream_t stream);

/*
 * sgemm_emu_gather_tokens -- Xs[places[t k + j]] = X[t] (X: T x K, Xs: P x K).
 *   Its gradient is sgemm_emu_combine_tokens without weights.
 */
int sgemm_emu_gather_tokens(int dtype, int64_t T, int64_t k, int64_t K, int64_t n, const void *X, int64_t ldx,
                            const int32_t *offsets, const int32_t *places, void *Xs, int64_t ldxs,
                            sgemm_emu_stream_t stream);

/*
 * sgemm_emu_combine_tokens -- Y[t] = sum over j of weights[t k + j] Ys[places[t k + j]]
 *   (Ys: P x K, Y: T x K; weights: P floats or NULL (1)), added in FP32 with j
 *   ascending; pairs that come nowhere add nothing.
 */
int sgemm_emu_combine_tokens(int dtype, int64_t T, int64_t k, int64_t K, const void *Ys, int64_t ldys,
                             const int32_t *places, const float *weights, void *Y, int64_t ldy,
                             sgemm_emu_stream_t stream);

/*
 * sgemm_emu_combine_tokens_backward -- from dY (T x K):
 *   dYs[places[p]] = weights[p] dY[t] (P x K), dweights[p] = dY[t] . Ys[places[p]],
 *   0 for pairs that come nowhere.  Either may be NULL (not computed).
 */
int sgemm_emu_combine_tokens_backward(int dtype, int64_t T, int64_t k, int64_t K, int64_t n, const void *Ys,
                                      int64_t ldys, const int32_t *offsets, const int32_t *places,
                                      const float *weights, const void *dY, int64_t lddy, void *dYs, int64_t lddys,
                                      float *dweights, sgemm_emu_stream_t stream);

/*
 * sgemm_emu_expert_linear -- on the rows of expert e: Z = X W_e^T + bias_e, and
 *   H = Z, or, with a gate (enum sgemm_emu_gate; N = 2F even),
 *   H = act(Z[:, :F]) * Z[:, F:].
 *   X: P x K; W: n x N x K contiguous; bias: n x N contiguous or NULL; H: P x N, or
 *   P x F with a gate.  FP32: the six leading products of a three-way BF16 split to
 *   nearest (what is left out is at most 2^-24 of a product, an FP32 product's own
 *   rounding), summed in FP32 (in three bands, which hold at most 2.01 times the sum of
 *   |x w|: outputs where it passes 2^126 may be Inf or NaN); an Inf or NaN makes the outputs
 *   that it reaches, of its row or expert only, Inf or NaN.
 *   Zkeep: NULL, or with a gate P rows of 2 pad8(F) floats as in
 *   sgemm_emu_gated_linear, for the backward.
 */
int sgemm_emu_expert_linear(int dtype, int64_t P, int64_t N, int64_t K, int64_t n, const void *X, int64_t ldx,
                            const void *W, const void *bias, int gate, const int32_t *offsets, void *H, int64_t ldh,
                            float *Zkeep, sgemm_emu_stream_t stream);

/*
 * sgemm_emu_expert_linear_backward -- from dH and the forward's X, W, Zkeep, on the
 *   rows of expert e: dZ as in sgemm_emu_gated_linear_backward (dH itself without a
 *   gate), dX = dZ W_e (P x K), dW_e = dZ^T X (n x N x K contiguous),
 *   dbias_e = sum over the rows of dZ (n x N).  Experts without rows get zeros.
 *   Each of dX, dW, dbias may be NULL (not computed).  Sums are added in a fixed
 *   order: results are deterministic.
 */
int64_t sgemm_emu_expert_linear_backward_workspace(int dtype, int64_t P, int64_t N, int64_t K, int64_t n, int gate,
                                                   int dbias);
int sgemm_emu_expert_linear_backward(int dtype, int64_t P, int64_t N, int64_t K, int64_t n, const void *X, int64_t ldx,
                                     const void *W, const float *Zkeep, int gate, const int32_t *offsets,
                                     const void *dH, int64_t lddh, void *dX, int64_t lddx, void *dW, void *dbias,
                                     void *ws, int64_t ws_bytes, sgemm_emu_stream_t stream);

/*
 * Weights of 4 bits: n banks (1: a layer) of N x K values q in 0..15 which stand for
 * (q - zero) scale, scale (FP32) and zero (0..15, 8 where NULL) shared by `group`
 * (32, 64 or 128) consecutive columns of a row; scale, zero: n x N x ceil(K / group).
 *
 * sgemm_emu_quant4_quantize -- nearest such weights of W (n x N x K contiguous):
 *   zero NULL: symmetric, scale = max|w| / 7 and q - 8 in -7..7; else scale =
 *   (max(w, 0) - min(w, 0)) / 15, zero = -min / scale rounded.  Groups of zeros take
 *   scale 0, groups with a NaN or an Inf stand for NaN.  Values are rounded to
 *   nearest, ties to even.  No level passes the largest BF16: scales end there.
 * sgemm_emu_quant4_pack -- lays them out for sgemm_emu_quant4_linear: `packed` of
 *   sgemm_emu_quant4_bytes bytes, 16-byte aligned.  q's high four bits are ignored,
 *   and so are zero's.
 * sgemm_emu_quant4_unpack -- the weights (q - zero) scale in FP32, rounded to the
 *   call's type (W: n x N x K contiguous).
 */
int64_t sgemm_emu_quant4_bytes(int64_t n, int64_t N, int64_t K, int64_t group, int zeros);
int sgemm_emu_quant4_quantize(int dtype, int64_t n, int64_t N, int64_t K, int64_t group, const void *W, uint8_t *q,
                              float *scale, uint8_t *zero, sgemm_emu_stream_t stream);
int sgemm_emu_quant4_pack(int64_t n, int64_t N, int64_t K, int64_t group, const uint8_t *q, const float *scale,
                          const uint8_t *zero, void *packed, sgemm_emu_stream_t stream);
int sgemm_emu_quant4_unpack(int dtype, int64_t n, int64_t N, int64_t K, int64_t group, int zeros, const void *packed,
                            void *W, sgemm_emu_stream_t stream);

/*
 * sgemm_emu_quant4_linear -- sgemm_emu_expert_linear with such weights.  offsets NULL:
 *   one layer (n = 1) on all P rows.  Few rows read the packed weights and sum
 *   (q - zero) x in FP32, scaled group by group, for finite X of any size (an Inf in
 *   a row of X makes that row's outputs NaN); more rows (ws_bytes > 0) unpack the weights into ws first,
 *   rounded to the call's type.
 */
int64_t sgemm_emu_quant4_linear_workspace(int dtype, int64_t P, int64_t N, int64_t K, int64_t n, int64_t group,
                                          int zeros);
int sgemm_emu_quant4_linear(int dtype, int64_t P, int64_t N, int64_t K, int64_t n, int64_t group, int zeros,
                            const void *X, int64_t ldx, const void *packed, const void *bias, int gate,
                            const int32_t *offsets, void *H, int64_t ldh, void *ws, int64_t ws_bytes,
                            sgemm_emu_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* SGEMM_EMU_EXPERTS_H */
