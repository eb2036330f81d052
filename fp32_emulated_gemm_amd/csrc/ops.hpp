// ops.hpp -- internal launch interface of the operators beside the GEMM (gated
// projection, linear layer with low-rank adapters).  Not part of the public
// headers.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "launch.hpp"

namespace sgemm_emu_dev {

constexpr int64_t kPadK = 64;   // K of a laid-out operand is padded with zeros to a multiple of this
inline int64_t pad_k(int64_t k) { return (k + kPadK - 1) / kPadK * kPadK; }
inline int64_t round_up(int64_t v, int64_t a) { return (v + a - 1) / a * a; }

// ---------------------------------------------------------------- low-rank adapters
// Row t of X belongs to adapter ids[t]; an id outside [0, n) means none.
// down: n x r x K, up: n x N x r, both contiguous; scale: n floats or null (1).
struct Adapters {
    const int32_t *ids;
    int64_t n, r;
    const void *down, *up;
    const float *scale;
};
inline int64_t rank_pad(int64_t r) { return round_up(r, 16); }   // row pitch of S (zeros past r)

// S[t][0..rp) = scale[i] * down[i] X[t] (zeros for rows without an adapter),
// float32, rp = rank_pad(r).
hipError_t launch_shrink(int dtype, int64_t M, int64_t K, const void *X, int64_t ldx, const Adapters &ad, float *S,
                         int num_cus, hipStream_t stream);

// Y[t] += up[i] S[t] for the rows that have an adapter.
hipError_t launch_expand(int dtype, int64_t M, int64_t N, const float *S, const Adapters &ad, void *Y, int64_t ldy,
                         int num_cus, hipStream_t stream);

// offs[0..n]: where each adapter's rows start in rows[]; rows[]: the row
// numbers that have an adapter, grouped by it, ascending inside a group.
hipError_t launch_group(int64_t M, const int32_t *ids, int64_t n, int32_t *offs, int32_t *rows, hipStream_t stream);

// G[i] = sum over the adapter's rows t of L[t][0..r) (x) R[t][0..C): n x r x C,
// or n x C x r with `transposed`, in the operands' type.  L float32 with pitch
// rank_pad(r); partials: lowrank_grad_floats() floats.
int64_t lowrank_grad_floats(int64_t M, int64_t C, int64_t n, int64_t r, int num_cus);
hipError_t launch_lowrank_grad(int dtype, int64_t M, int64_t C, int64_t n, int64_t r, const float *L, const void *R,
                               int64_t ldr, const int32_t *offs, const int32_t *rows, bool transposed, void *G,
                               float *partials, int num_cus, hipStream_t stream);

// ---------------------------------------------------------------- few rows
// Y = X W^T + bias (+ up[i] S[t]), or, with gate >= 0, the gated product of a
// weight of 2F rows (N = F).  Any M; made for few rows.
struct FewRows {
    int64_t M, N, K;
    const void *X;
    int64_t ldx;
    const void *W;
    int64_t ldw;
    const void *bias;       // N values (2N with a gate) or null
    int gate;               // -1: none
    void *Y;
    int64_t ldy;
    const Adapters *ad;     // or null
    const float *S;
};
hipError_t launch_few_rows(int dtype, const FewRows &a, int num_cus, hipStream_t stream);

// ---------------------------------------------------------------- bfloat16 GEMM
// C = A B^T (+ bias) with A M x K and B N x K, both bfloat16 with k contiguous,
// 16-byte aligned rows and K a multiple of 8.
struct Bf16Gemm {
    int64_t M, N, K;
    const uint16_t *A;
    int64_t lda;
    const uint16_t *B;
    int64_t ldb;
    const uint16_t *bias;    // N values or null
    uint16_t *C;             // M x N, or M x N/2 with a gate
    int64_t ldc;
    int gate;                // -1: none; else B holds F = N/2 gate rows, then F up rows
    uint16_t *Z;             // with a gate: M x N pre-activations (gate | up), or null
    int64_t ldz;
    const int32_t *ids;      // adapters (or null): rows' ids, S (M x rp), up (n x N x r)
    int64_t n, r, rp;
    const uint16_t *up;
    const float *S;
    float *partials;         // K slices: splits x M x N floats
    int splits;
    int64_t k_per_split;
    int tiles_m, tiles_n, group_m;
};
// Floats of `partials` the product takes (0: one pass over K).
int64_t bf16_gemm_partial_floats(int64_t M, int64_t N, int64_t K, bool plain, int num_cus);
hipError_t launch_bf16_gemm(const Bf16Gemm &g, int num_cus, hipStream_t stream);

// ---------------------------------------------------------------- layouts and elementwise
// Three BF16 planes of X (rows x cols FP32), rows x pad_k(cols) with zeros past
// cols; planes at P, P + rows * pad_k(cols), P + 2 rows * pad_k(cols).
hipError_t launch_split_padded(int64_t rows, int64_t cols, const float *X, int64_t ldx, uint16_t *P,
                               hipStream_t stream);
// bfloat16 rows x cols -> rows x pad_k(cols), zeros past cols.
hipError_t launch_copy_padded(int64_t rows, int64_t cols, const uint16_t *X, int64_t ldx, uint16_t *P,
                              hipStream_t stream);
// bfloat16 rows x cols -> cols x pad_k(rows), zeros past rows.
hipError_t launch_transpose_padded(int64_t rows, int64_t cols, const uint16_t *X, int64_t ldx, uint16_t *P,
                                   hipStream_t stream);
// src n x rows x cols -> dst n x cols x rows (contiguous).
hipError_t launch_transpose_bank(int dtype, int64_t n, int64_t rows, int64_t cols, const void *src, void *dst,
                                 hipStream_t stream);

// H = act(Z[:, :F]) * Z[:, F:], float32.
hipError_t launch_gate(int64_t M, int64_t F, const float *Z, int64_t ldz, int gate, float *H, int64_t ldh,
                       hipStream_t stream);

// dZ (M x 2F, pitch ldd, columns 2F..ldd zero; null: skipped), its transpose
// (2F x pad_k(M), zeros past M; null: skipped) and the column sums' partials
// (gate_tiles(M) x 2F floats; null: skipped) from Z and dH.
inline int64_t gate_tiles(int64_t M) { return (M + 63) / 64; }
hipError_t launch_gate_backward(int dtype, int64_t M, int64_t F, const void *Z, int64_t ldz, const void *dH,
                                int64_t lddh, int gate, void *dZ, int64_t ldd, void *dZt, float *sums,
                                hipStream_t stream);
// out[c] = sum over t of sums[t][c], t ascending.
hipError_t launch_sum_tiles(int dtype, int64_t tiles, int64_t cols, const float *sums, void *out, hipStream_t stream);

// ---------------------------------------------------------------- FP32 products (api.hip)
// C = A B^T (+ bias) with FP32 A (M x K, lda) and B as zero-padded planes
// (launch_split_padded of an N x K matrix): nine products.
int gemm_padded_planes(int64_t M, int64_t N, int64_t K, const float *A, int64_t lda, const uint16_t *planes,
                       const float *bias, float *C, int64_t ldc, hipStream_t stream);
// The current device's CU count if it is a gfx950 (SGEMM_EMU_EARCH otherwise).
int current_cus(int *num_cus);

}  // namespace sgemm_emu_dev
