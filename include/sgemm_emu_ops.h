/*
 * sgemm_emu_ops.h -- C ABI of libsgemm_emu's operators beside the GEMM: the
 * gated feed-forward projection and the linear layer with low-rank adapters,
 * forward and backward, for FP32 and bfloat16 tensors.
 *
 * Conventions are those of sgemm_emu.h (row-major, device pointers on the
 * current HIP device, int64_t sizes, leading dimensions in elements, work
 * enqueued on `stream`, arguments checked before any HIP call, nothing enqueued
 * on an error status other than SGEMM_EMU_ELAUNCH, which a call's later kernels
 * can give too), and:
 *   dtype      SGEMM_EMU_F32: float tensors; products are the nine BF16
 *              products of sgemm_bf16x9, or FP32 matrix instructions where a
 *              call has few rows.  SGEMM_EMU_BF16: bfloat16 tensors (uint16_t
 *              bit patterns); a bfloat16 value is its own first component, so
 *              one product; sums are FP32, outputs rounded once to nearest
 *              even.
 *   pointers   void * of the call's type, aligned to one element.  16-byte
 *              aligned operands with leading dimensions that are multiples of
 *              16 bytes take the fastest loads; others are read element by
 *              element, or copied into `ws` first.
 *   plan       a weight laid out by sgemm_emu_plan_weight, 16-byte aligned,
 *              K padded with zeros.  It depends on the weight's values: a
 *              weight that changes is laid out again.
 *   ws         caller's scratch memory, 256-byte aligned, of at least the bytes
 *              that the matching *_workspace function returns for the same
 *              arguments (0: may be NULL; negative: invalid arguments).
 *              Its contents do not matter before or after the call; two calls
 *              that may overlap in time need one each.  FP32 products on small
 *              tile grids additionally use the library's per-stream workspace
 *              for their stream-K partial results (see sgemm_emu_split_k), and
 *              products of at least 1024 rows and 4096 columns for A's BF16
 *              planes.  Without memory for the former, a call returns
 *              SGEMM_EMU_ENOMEM, or SGEMM_EMU_ECAPTURE on a stream being
 *              captured into a graph; without the latter the kernel splits A
 *              itself (bitwise the same result).
 *   limits     leading dimensions up to 8,388,544 elements; M, F, N, K up to
 *              4,194,240; up to 65,535 adapters, n r (K + N) up to 2^55.
 * Outputs must not overlap inputs (not checked).
 */
#ifndef SGEMM_EMU_OPS_H
#define SGEMM_EMU_OPS_H

#include "sgemm_emu.h"

#ifdef __cplusplus
extern "C" {
#endif

enum sgemm_emu_dtype { SGEMM_EMU_F32 = 0, SGEMM_EMU_BF16 = 1 };

/* act of the gated projection */
enum sgemm_emu_gate {
    SGEMM_EMU_GATE_SILU = 0,      /* z / (1 + exp(-z)) */
    SGEMM_EMU_GATE_GELU = 1,      /* exact (erf) form */
    SGEMM_EMU_GATE_GELU_TANH = 2, /* 0.5 z (1 + tanh(sqrt(2/pi) (z + 0.044715 z^3))) */
    SGEMM_EMU_GATE_SIGMOID = 3,
    SGEMM_EMU_GATE_RELU = 4
};

/* How a weight is laid out: its rows, the rows of its transpose, or (an even
   number of) rows whose first half are gate rows and second half up rows. */
enum sgemm_emu_plan_layout {
    SGEMM_EMU_PLAN_ROWS = 0,       /* sgemm_emu_adapter_linear's W */
    SGEMM_EMU_PLAN_TRANSPOSED = 1, /* W^T, for sgemm_emu_adapter_linear_backward */
    SGEMM_EMU_PLAN_GATED = 2       /* sgemm_emu_gated_linear's W */
};

/*
 * sgemm_emu_plan_weight -- lays the rows x cols weight W out for the products
 * below.  FP32: three BF16 planes; bfloat16: one.  Rows of pad(k) = k rounded up
 * to a multiple of 64 elements, zeros past k.  sgemm_emu_plan_bytes gives the
 * size (negative on invalid arguments).
 */
int64_t sgemm_emu_plan_bytes(int dtype, int64_t rows, int64_t cols, int layout);
int sgemm_emu_plan_weight(int dtype, int64_t rows, int64_t cols, const void *W, int64_t ldw, int layout,
                          void *plan, sgemm_emu_stream_t stream);

/*
 * sgemm_emu_gated_linear -- H = act(Z[:, :F]) * Z[:, F:], Z = X W^T + bias.
 *   X: M x K (ldx >= K); W: 2F x K (ldw >= K), the gate's F rows, then the up
 *   projection's F rows; bias: 2F values or NULL; H: M x F (ldh >= F).
 *   plan: W's plan (SGEMM_EMU_PLAN_GATED), or NULL: calls of at most
 *   sgemm_emu_few_rows() rows read W itself, and so do bfloat16 calls whose W is
 *   16-byte aligned with K and ldw multiples of 8; other calls lay W out in ws.
 *   Z: NULL, or M rows of 2 pad8(F) floats (pad8: rounded up to a multiple of 8),
 *   16-byte aligned: the pre-activations, in 32 bits whatever the call's type,
 *   the gate's from column 0 and the up projection's from column pad8(F), as
 *   sgemm_emu_gated_linear_backward takes them (the other columns are not set).
 */
int64_t sgemm_emu_gated_linear_workspace(int dtype, int64_t M, int64_t F, int64_t K, const void *X, int64_t ldx,
                                         const void *W, int64_t ldw, const void *plan, const void *Z);
int sgemm_emu_gated_linear(int dtype, int64_t M, int64_t F, int64_t K, const void *X, int64_t ldx, const void *W,
                           int64_t ldw, const void *plan, const void *bias, int gate, void *H, int64_t ldh, float *Z,
                           void *ws, int64_t ws_bytes, sgemm_emu_stream_t stream);

/*
 * sgemm_emu_gated_linear_backward -- from dH (M x F) and the forward's X, W, Z:
 *   dZ = [dH * Z[:, F:] * act'(Z[:, :F]) | dH * act(Z[:, :F])],
 *   dX = dZ W (M x K), dW = dZ^T X (2F x K), dbias[j] = sum over rows of dZ.
 *   Each of dX, dW, dbias may be NULL (not computed).  bfloat16: dZ is rounded
 *   to bfloat16 as an operand of the two products; dbias sums it in FP32 before
 *   that rounding.  Sums are added in a fixed order: results are deterministic.
 */
int64_t sgemm_emu_gated_linear_backward_workspace(int dtype, int64_t M, int64_t F, int64_t K);
int sgemm_emu_gated_linear_backward(int dtype, int64_t M, int64_t F, int64_t K, const void *X, int64_t ldx,
                                    const void *W, int64_t ldw, const float *Z, int gate, const void *dH, int64_t lddh,
                                    void *dX, int64_t lddx, void *dW, int64_t lddw, void *dbias,
                                    void *ws, int64_t ws_bytes, sgemm_emu_stream_t stream);

/*
 * sgemm_emu_adapter_linear -- Y[t] = W X[t] + bias + scale[i] up_i (down_i X[t]),
 *   i = ids[t]; a row whose id lies outside [0, n) has no adapter.
 *   X: M x K; W: N x K; bias: N values or NULL; down: n x r x K and up: n x N x r,
 *   contiguous, of the call's type; scale: n floats or NULL (1); ids: M int32 in
 *   any order; Y: M x N.  n = 0 or r = 0: no adapters (down, up, ids unused).
 *   plan: W's plan (SGEMM_EMU_PLAN_ROWS) or NULL, as for sgemm_emu_gated_linear.
 *   S: NULL, or 4 M pad16(r) bytes (r rounded up to a multiple of 16), 16-byte
 *   aligned: the low-rank activations scale[i] down_i X[t], as
 *   sgemm_emu_adapter_linear_backward takes them (floats for FP32; for bfloat16 a
 *   row's pad16(r) high and pad16(r) low BF16 parts, 16 significant bits).
 *   Inf and NaN in one adapter's weights reach only the rows that use it.
 */
int64_t sgemm_emu_adapter_linear_workspace(int dtype, int64_t M, int64_t N, int64_t K, const void *X, int64_t ldx,
                                           const void *W, int64_t ldw, const void *plan, int64_t n, int64_t r,
                                           const void *up, const float *S);
int sgemm_emu_adapter_linear(int dtype, int64_t M, int64_t N, int64_t K, const void *X, int64_t ldx, const void *W,
                             int64_t ldw, const void *plan, const void *bias, int64_t n, int64_t r, const void *down,
                             const void *up, const float *scale, const int32_t *ids, void *Y, int64_t ldy, float *S,
                             void *ws, int64_t ws_bytes, sgemm_emu_stream_t stream);

/*
 * sgemm_emu_adapter_linear_backward -- from dY (M x N), with W and bias fixed:
 *   P[t] = scale[i] up_i^T dY[t],  dX = dY W + P down_i,
 *   d_down_i = sum over the adapter's rows of P[t] X[t]^T  (n x r x K),
 *   d_up_i = sum over the adapter's rows of dY[t] S[t]^T   (n x N x r);
 *   adapters without rows get zeros.  dX, d_down, d_up may be NULL (not
 *   computed).  W^T enters through its plan (SGEMM_EMU_PLAN_TRANSPOSED, required for dX).
 *   S: the forward's.  Sums are added in a fixed order: deterministic.
 */
int64_t sgemm_emu_adapter_linear_backward_workspace(int dtype, int64_t M, int64_t N, int64_t K, int64_t n, int64_t r);
int sgemm_emu_adapter_linear_backward(int dtype, int64_t M, int64_t N, int64_t K, const void *X, int64_t ldx,
                                      const void *plan_t, int64_t n, int64_t r, const void *down, const void *up,
                                      const float *scale, const int32_t *ids, const float *S, const void *dY,
                                      int64_t lddy, void *dX, int64_t lddx, void *d_down, void *d_up, void *ws,
                                      int64_t ws_bytes, sgemm_emu_stream_t stream);

/* Rows up to which the forward calls read the weight itself in one pass. */
int sgemm_emu_few_rows(void);

#ifdef __cplusplus
}
#endif

#endif /* SGEMM_EMU_OPS_H */
