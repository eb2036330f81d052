// experts.hpp -- internal launch interface of the experts' operators and of the
// products with 4-bit weights.  Not part of the public headers.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "ops.hpp"

namespace sgemm_emu_dev {

// A launch holds fewer than 2^32 work-items along x, which many experts beside wide
// weights pass: workgroups go on along y (expert_device.hpp: workgroup()).
constexpr int kGridX = 1 << 22;              // of up to 512 work-items
inline bool grid_ok(int64_t blocks) { return blocks < (int64_t)1 << 31; }
inline dim3 grid_of(int64_t blocks)
{
    return dim3((unsigned)(blocks < kGridX ? blocks : kGridX), (unsigned)((blocks + kGridX - 1) / kGridX));
}

constexpr int kMaxExperts = 1024;            // SGEMM_EMU_MAX_EXPERTS

// ---------------------------------------------------------------- tokens (route.hip)
// int32 values of scratch that the sort of P pairs takes.
int64_t sort_counts(int64_t P, int64_t n);
hipError_t launch_sort(int64_t P, int64_t n, const int32_t *ids, int32_t *offsets, int32_t *pairs, int32_t *places,
                       int32_t *counts, hipStream_t stream);

enum { kGather, kCombine, kCombineBackward };
template <class T>
struct Route {
    int64_t P, tokens, k, K, n;
    const int32_t *offsets, *places;
    const float *weights;        // P or null
    const T *x;                  // tokens: X (gather), dY (combine's backward)
    int64_t ldx;
    const T *rows;               // sorted rows: Ys
    int64_t ldr;
    T *x_out;                    // tokens: Y
    int64_t ldx_out;
    T *rows_out;                 // sorted rows: Xs, dYs (or null)
    int64_t ldr_out;
    float *dweights;             // or null
    bool past;                   // set by the launch
};
hipError_t launch_route(int what, const Route<float> &a, hipStream_t stream);
hipError_t launch_route(int what, const Route<uint16_t> &a, hipStream_t stream);

hipError_t launch_clear_floats(float *p, int64_t n, hipStream_t stream);

// ---------------------------------------------------------------- products (expert_gemm.hip)
// Rows of a matrix that stand for the two halves of a gated weight: logical index
// k is row k for k < F, row F + k - h for h <= k < h + F, no row elsewhere.
struct Halves {
    int64_t F, h;
    __host__ __device__ int64_t row(int64_t k) const
    {
        return k < F ? k : k >= h && k - h < F ? F + k - h : -1;
    }
};

struct ExpertProduct {
    int64_t P, M, N, K, n;       // rows of X; outputs' rows (dW only); columns; inner extent (not dW)
    const int32_t *offsets;      // null: one expert has all rows
    const void *A;               // P x K, or dZ
    int64_t lda;
    const void *B;               // the bank, n x (N x K) or, for dX, n x (rows x N); or X
    int64_t ldb, bank;           // and its elements per expert
    const void *bias;            // n x N or null
    int gate;                    // -1: none
    void *C;
    int64_t ldc;
    float *Z;                    // with a gate: pre-activations (see z_pitch), or null
    int64_t ldz;
    Halves map;                  // dX: rows of B behind k; dW: rows of the weight behind dZ's columns
    float *partials;             // dW: sums of pieces of `chunk` rows, M x N each, or null
    int64_t chunk;
    int num_cus;
    int tiles_m, tiles_n;        // set by the launch
};
// A weight gradient with few tiles runs over pieces of the experts' rows, so that one
// expert with many rows does not hold the others up: rows of a piece (0: the tiles
// suffice), such that there are about two tiles to a CU, and the pieces at most.
constexpr int64_t kPlanCus = 256;            // MI355X
constexpr int64_t weight_chunk(int64_t P, int64_t M, int64_t N, int64_t n)
{
    const int64_t per = ((M + 127) / 128) * ((N + 127) / 128), even = round_up(P * per / (2 * kPlanCus), 64);
    return n * per >= 3 * kPlanCus || P <= 256 || per == 0 ? 0 : even < 256 ? 256 : even >= P ? 0 : even;
}
__host__ __device__ inline int64_t weight_chunks(const ExpertProduct &g)
{
    return g.partials == nullptr ? g.n : g.P / g.chunk + (g.n < g.P ? g.n : g.P);
}
// kForward: C[r] = A[r] B_e^T (+ bias, gate) on the rows r of expert e.
// kBackX: C[r] = A[r] B_e with B_e's rows by `map`: A = dZ (K columns), N columns.
// Both leave zeros on rows of no expert.
// kBackW: C_e (map's rows x N) = A_e^T B_e over the rows of expert e: A = dZ (M
// columns), B = X (N columns).
enum { kForward, kBackX, kBackW };
hipError_t launch_expert(int op, int dtype, const ExpertProduct &g, hipStream_t stream);
hipError_t launch_expert_f32(int op, const ExpertProduct &g, hipStream_t stream);
// For bfloat16 operands whose rows start at 16-byte pieces and hold whole ones;
// expert_lies() tells whether a product's do.
bool expert_lies(int op, const ExpertProduct &g);
hipError_t launch_expert_bf16(int op, const ExpertProduct &g, hipStream_t stream);
// Whether a forward product of few rows takes the kernel made for them.
bool expert_few(int dtype, const ExpertProduct &g);
hipError_t launch_expert_few(int dtype, const ExpertProduct &g, hipStream_t stream);

// ---------------------------------------------------------------- gate backward (expert_gate.hip)
// Halves of a row of dZ are padded to whole tiles, so that no step over its columns
// and no tile of them meets both.
constexpr int64_t expert_dz_pitch(int64_t F) { return 2 * round_up(F, 128); }
// dZ (rows of expert_dz_pitch(F): gate from 0, up from the half, zeros between and
// after) from Z and dH, and the bias gradients' partial sums, a row of 2F floats
// (N without a gate) for each tile of 64 rows of an expert; each may be null.
struct ExpertGate {
    int64_t P, F, n;             // F: outputs of a row (N without a gate)
    const int32_t *offsets;
    const float *Z;
    const void *dH;
    int64_t lddh;
    int gate;                    // -1: sums of dH alone
    void *dZ;
    float *sums;                 // expert_gate_tiles() rows
    void *dbias;                 // n x 2F (N)
};
__host__ __device__ inline int64_t expert_gate_tiles(int64_t P, int64_t n) { return P / 64 + (n < P ? n : P); }
hipError_t launch_expert_gate(int dtype, const ExpertGate &g, hipStream_t stream);

// ---------------------------------------------------------------- 4-bit weights (quant4.hip)
// A bank's packed bytes: values, scales, zeros (16 added), see quant4.hip; and spare
// bytes behind, which a tile that begins inside another reads past the last row.
struct Quant4 {
    int64_t n, N, K, group;
    bool zeros;
    __host__ __device__ int64_t rows() const { return round_up(N, 16); }
    __host__ __device__ int64_t blocks() const { return (K + 127) / 128; }          // of 128 columns
    __host__ __device__ int64_t groups() const { return blocks() * (128 / group); }
    __host__ __device__ int64_t value_bytes() const { return rows() * blocks() * 64; }
    __host__ __device__ int64_t scale_bytes() const { return groups() * rows() * 4; }
    __host__ __device__ int64_t zero_bytes() const { return zeros ? round_up(groups() * rows(), 16) : 0; }
    __host__ __device__ int64_t bank_bytes() const { return value_bytes() + scale_bytes() + zero_bytes() + 64; }
};
hipError_t launch_quant4_quantize(int dtype, const Quant4 &w, const void *W, uint8_t *q, float *scale, uint8_t *zero,
                                  hipStream_t stream);
hipError_t launch_quant4_pack(const Quant4 &w, const uint8_t *q, const float *scale, const uint8_t *zero, void *packed,
                              hipStream_t stream);
hipError_t launch_quant4_unpack(int dtype, const Quant4 &w, const void *packed, void *W, hipStream_t stream);

struct Quant4Product {
    int64_t P;
    const void *X;
    int64_t ldx;
    const void *packed;
    const void *bias;
    int gate;
    const int32_t *offsets;
    void *H;
    int64_t ldh;
    int num_cus;
};
// Whether a call of P rows reads the packed weights (else it unpacks them first).
bool quant4_few(int dtype, const Quant4 &w, int64_t P);
hipError_t launch_quant4_few(int dtype, const Quant4 &w, const Quant4Product &g, hipStream_t stream);

}  // namespace sgemm_emu_dev
