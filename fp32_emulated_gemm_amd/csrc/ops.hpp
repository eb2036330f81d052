// ops.hpp -- internal launch interface of the operators beside the GEMM (gated
// projection, linear layer with low-rank adapters).  Not part of the public
// headers.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "launch.hpp"

namespace sgemm_emu_dev {

constexpr int64_t kPadK = 64;   // K of a laid-out operand is padded with zeros to a multiple of this
constexpr int64_t pad_k(int64_t k) { return (k + kPadK - 1) / kPadK * kPadK; }
constexpr int64_t round_up(int64_t v, int64_t a) { return (v + a - 1) / a * a; }

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

// S[t][0..rp) = scale[i] * down[i] X[t] (zeros for rows without an adapter and
// past r), rp = rank_pad(r): floats for FP32; for bfloat16 rp high and rp low
// BF16 parts in a row's 4 rp bytes.
hipError_t launch_shrink(int dtype, int64_t M, int64_t K, const void *X, int64_t ldx, const Adapters &ad, float *S,
                         int num_cus, hipStream_t stream);

// FP32: Y[t] += up[i] S[t] for the rows that have an adapter.
hipError_t launch_expand(int64_t M, int64_t N, const GemmEpilogue &ad, float *Y, int64_t ldy, hipStream_t stream);

// What the adapters' backward needs first, in one launch: up to two banks
// transposed (n x rows x cols -> n x cols x rows, contiguous), and the rows
// grouped: offs[0..n] tells where each adapter's rows start in rows[], the row
// numbers that have an adapter, ascending inside a group.
struct AdapterPrepare {
    struct Bank {
        int64_t rows, cols;
        const void *src;
        void *dst;            // null: not wanted
    } bank[2];
    int64_t n, M;
    const int32_t *ids;
    int32_t *offs, *rows;     // null: not wanted
    int64_t groups;           // set by the launch
};
hipError_t launch_adapter_prepare(int dtype, AdapterPrepare q, hipStream_t stream);

// down[i] = sum over the adapter's rows of P[t] (x) X[t] (n x r x K), up[i] = sum
// of dY[t] (x) S[t] (n x N x r); either may be null.  P, S as launch_shrink writes
// them; partials: lowrank_grad_floats() floats.
struct LowrankGrads {
    int64_t M, K, N, n, r;
    const float *P, *S;
    const void *X;
    int64_t ldx;
    const void *dY;
    int64_t lddy;
    const int32_t *offs, *rows;
    void *down, *up;
    float *partials;
};
int64_t lowrank_grad_floats(int dtype, int64_t M, int64_t K, int64_t N, int64_t n, int64_t r, int num_cus);
hipError_t launch_lowrank_grad(int dtype, const LowrankGrads &q, int num_cus, hipStream_t stream);

// ---------------------------------------------------------------- few rows
// At most kFewRows rows: Y = X W^T + bias + up[i] (scale[i] down[i] X[t]), or,
// with gate >= 0, the gated product of a weight of 2F rows (N = F).
constexpr int64_t kFewRows = 64;
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
    float *S;               // with adapters: M x rank_pad(r) floats of scratch
    float *partials;        // few_rows_partial_floats() floats (null where that is 0)
};
int64_t few_rows_partial_floats(int dtype, int64_t M, int64_t N, int64_t K, int gate, int num_cus);
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
    float *Z;                // with a gate: pre-activations (see z_pitch), or null
    int64_t ldz;
    const int32_t *ids;      // adapters (or null): rows' ids, up (n x N x r)
    int64_t n, r, rp;        // r (up's row pitch) even, up 4-byte aligned
    const uint16_t *up;
    const uint16_t *S;       // M x 2 rp: high parts, low parts
    float *partials;         // K slices: splits x M x N floats
    int splits;
    int64_t k_per_split;
    int64_t m_base, n_base;  // the launch's first row and column
    int tiles_m, tiles_n, group_m;
};
// Floats of `partials` the product takes (0: one pass over K).
int64_t bf16_gemm_partial_floats(int64_t M, int64_t N, int64_t K, bool plain, int num_cus);
hipError_t launch_bf16_gemm(const Bf16Gemm &g, int num_cus, hipStream_t stream);

// ---------------------------------------------------------------- layouts and elementwise
// Three BF16 planes of X (rows x cols FP32), rows x pad_k(cols) with zeros past
// cols; planes at P, P + rows * pad_k(cols), P + 2 rows * pad_k(cols).
// interleave: plane rows 2 f, 2 f + 1 are X's rows f, rows / 2 + f.
hipError_t launch_split_padded(int64_t rows, int64_t cols, const float *X, int64_t ldx, uint16_t *P, bool interleave,
                               hipStream_t stream);
// rows x cols -> rows of `pitch` (a multiple of 8), zeros past cols.
hipError_t launch_copy_padded(int dtype, int64_t rows, int64_t cols, const void *X, int64_t ldx, void *P,
                              int64_t pitch, hipStream_t stream);
// bfloat16 rows x cols -> cols x out_rows with pitch ldp, zeros past rows.
hipError_t launch_transpose_padded(int64_t rows, int64_t cols, const uint16_t *X, int64_t ldx, uint16_t *P,
                                   int64_t out_rows, int64_t ldp, hipStream_t stream);
// Pre-activations Z are floats whatever the call's type: rows of z_pitch(F), the
// gate's from column 0, the up projection's from column z_pitch(F) / 2.
constexpr int64_t z_pitch(int64_t F) { return 2 * round_up(F, 8); }


// K == 0: H = act(bias) * bias of the halves (bias null: zeros), and Z where kept.
hipError_t launch_gate_bias(int64_t M, int64_t F, const float *bias, int gate, float *H, int64_t ldh, float *Z,
                            hipStream_t stream);

// From Z and dH: dZ (rows of dz_pitch(F): gate from 0, up from dz_pitch / 2,
// zeros between and after), its transpose (2F x pad_k(M), zeros past M), and the
// column sums' partials (gate_tiles(M) x 2F floats); each may be null.
constexpr int64_t dz_pitch(int64_t F) { return 2 * round_up(F, 32); }
inline int64_t gate_tiles(int64_t M) { return (M + 63) / 64; }
hipError_t launch_gate_backward(int dtype, int64_t M, int64_t F, const float *Z, const void *dH, int64_t lddh,
                                int gate, void *dZ, void *dZt, float *sums, hipStream_t stream);
// out[c] = sum over t of sums[t][c], t ascending.
hipError_t launch_sum_tiles(int dtype, int64_t tiles, int64_t cols, const float *sums, void *out, hipStream_t stream);

// ---------------------------------------------------------------- FP32 products (gemm_fused.hip)
// The kernels of gemm_padded_planes (workspace.hpp).
const PlaneLaunchers &plain_launchers();     // bias
const PlaneLaunchers &gated_launchers();     // bias, gate (args.epi; B's columns alternate gate, up)
const PlaneLaunchers &adapter_launchers();   // bias, adapters (args.epi)
// The current device's CU count if it is a gfx950 (SGEMM_EMU_EARCH otherwise).
int current_cus(int *num_cus);

}  // namespace sgemm_emu_dev
