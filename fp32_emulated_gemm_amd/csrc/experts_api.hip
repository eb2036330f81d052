// experts_api.hip -- the C ABI declared in include/sgemm_emu_experts.h: argument
// validation, the workspace layouts, and the order of the kernels.
//
// As in ops_api.hip every argument is checked before the first HIP call, and scratch
// memory is the caller's, laid out by the code that sizes it.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "../../include/sgemm_emu_experts.h"
#include "abi_checks.hpp"
#include "experts.hpp"

using namespace sgemm_emu_dev;

namespace {

static_assert(SGEMM_EMU_MAX_EXPERTS == kMaxExperts, "header and kernels agree");

bool experts_ok(int64_t n) { return n >= 0 && n <= kMaxExperts; }

// A bank of n N x K matrices, contiguous; N and K are extents.
bool bank_ok(int64_t n, int64_t N, int64_t K)
{
    return experts_ok(n) && extent_ok(N) && extent_ok(K) && (n == 0 || N == 0 || K <= kMaxBankElems / n / N);
}

int check_tokens(int64_t T, int64_t k, int64_t n, const void *offsets, const void *places)
{
    if (!extent_ok(T) || k < 0 || !experts_ok(n) || (T > 0 && !extent_ok(k)) || !extent_ok(T * k)) return SGEMM_EMU_EINVAL;
    CHECK(check_vector(n + 1, offsets, 4, false));
    return check_vector(T * k, places, 4, false);
}

int check_gate(int gate, int64_t N)
{
    if (gate == SGEMM_EMU_GATE_NONE) return SGEMM_EMU_OK;
    return gate >= 0 && gate <= SGEMM_EMU_GATE_RELU && N % 2 == 0 ? SGEMM_EMU_OK : SGEMM_EMU_EINVAL;
}

template <class T>
Route<T> route_args(int64_t tokens, int64_t k, int64_t K, int64_t n, const int32_t *offsets, const int32_t *places)
{
    Route<T> a{};
    a.P = tokens * k; a.tokens = tokens; a.k = k; a.K = K; a.n = n;
    a.offsets = offsets; a.places = places;
    return a;
}

struct SortWs {
    int32_t *counts;
    int64_t bytes;
    SortWs(void *ws, int64_t P, int64_t n)
    {
        Carve c(ws);
        counts = c.take<int32_t>(sort_counts(P, n));
        bytes = c.bytes;
    }
};

struct BackwardWs {
    void *dZ;
    float *sums, *partials;
    int64_t chunk, bytes;
    BackwardWs(void *ws, int dtype, int64_t P, int64_t N, int64_t K, int64_t n, int gate, bool dbias)
    {
        Carve c(ws);
        dZ = gate >= 0 ? (void *)c.take<char>(P * expert_dz_pitch(N / 2) * size_of(dtype)) : nullptr;
        sums = dbias ? c.take<float>(expert_gate_tiles(P, n) * N) : nullptr;
        const int64_t M = gate >= 0 ? expert_dz_pitch(N / 2) : N;
        chunk = weight_chunk(P, M, K, n);
        partials = chunk > 0 ? c.take<float>((P / chunk + (n < P ? n : P)) * M * K) : nullptr;
        bytes = c.bytes;
    }
};

bool group_ok(int64_t group) { return group == 32 || group == 64 || group == 128; }

Quant4 quant4(int64_t n, int64_t N, int64_t K, int64_t group, int zeros) { return Quant4{n, N, K, group, zeros != 0}; }

}  // namespace

extern "C" {

int64_t sgemm_emu_sort_tokens_workspace(int64_t P, int64_t n)
{
    if (!extent_ok(P) || !experts_ok(n)) return SGEMM_EMU_EINVAL;
    return SortWs(nullptr, P, n).bytes;
}

int sgemm_emu_sort_tokens(int64_t P, int64_t n, const int32_t *ids, int32_t *offsets, int32_t *pairs, int32_t *places,
                          void *ws, int64_t ws_bytes, sgemm_emu_stream_t stream)
{
    if (!extent_ok(P) || !experts_ok(n)) return SGEMM_EMU_EINVAL;
    CHECK(check_vector(P, ids, 4, false));
    CHECK(check_vector(n + 1, offsets, 4, false));
    CHECK(check_vector(P, pairs, 4, false));
    CHECK(check_vector(P, places, 4, false));
    const SortWs w(ws, P, n);
    CHECK(check_ws(ws, ws_bytes, w.bytes));
    int cus = 0;
    CHECK(current_cus(&cus));
    LAUNCH(launch_sort(P, n, ids, offsets, pairs, places, w.counts, (hipStream_t)stream));
    return SGEMM_EMU_OK;
}

int sgemm_emu_gather_tokens(int dtype, int64_t T, int64_t k, int64_t K, int64_t n, const void *X, int64_t ldx,
                            const int32_t *offsets, const int32_t *places, void *Xs, int64_t ldxs,
                            sgemm_emu_stream_t stream)
{
    if (!dtype_ok(dtype) || !extent_ok(K)) return SGEMM_EMU_EINVAL;
    CHECK(check_tokens(T, k, n, offsets, places));
    CHECK(check_operand(dtype, T, K, X, ldx));
    CHECK(check_operand(dtype, T * k, K, Xs, ldxs));
    int cus = 0;
    CHECK(current_cus(&cus));
    auto call = [&](auto *x, auto *rows) {
        auto a = route_args<std::remove_const_t<std::remove_pointer_t<decltype(x)>>>(T, k, K, n, offsets, places);
        a.x = x; a.ldx = ldx; a.rows_out = rows; a.ldr_out = ldxs;
        return launch_route(kGather, a, (hipStream_t)stream);
    };
    LAUNCH(dtype == SGEMM_EMU_F32 ? call((const float *)X, (float *)Xs) : call((const uint16_t *)X, (uint16_t *)Xs));
    return SGEMM_EMU_OK;
}

int sgemm_emu_combine_tokens(int dtype, int64_t T, int64_t k, int64_t K, const void *Ys, int64_t ldys,
                             const int32_t *places, const float *weights, void *Y, int64_t ldy,
                             sgemm_emu_stream_t stream)
{
    if (!dtype_ok(dtype) || !extent_ok(K)) return SGEMM_EMU_EINVAL;
    const int32_t none = 0;
    CHECK(check_tokens(T, k, 0, &none, places));
    CHECK(check_operand(dtype, T * k, K, Ys, ldys));
    CHECK(check_vector(T * k, weights, 4, true));
    CHECK(check_operand(dtype, T, K, Y, ldy));
    int cus = 0;
    CHECK(current_cus(&cus));
    auto call = [&](auto *rows, auto *y) {
        auto a = route_args<std::remove_pointer_t<decltype(y)>>(T, k, K, 0, nullptr, places);
        a.weights = weights; a.rows = rows; a.ldr = ldys; a.x_out = y; a.ldx_out = ldy;
        return launch_route(kCombine, a, (hipStream_t)stream);
    };
    LAUNCH(dtype == SGEMM_EMU_F32 ? call((const float *)Ys, (float *)Y) : call((const uint16_t *)Ys, (uint16_t *)Y));
    return SGEMM_EMU_OK;
}

int sgemm_emu_combine_tokens_backward(int dtype, int64_t T, int64_t k, int64_t K, int64_t n, const void *Ys,
                                      int64_t ldys, const int32_t *offsets, const int32_t *places,
                                      const float *weights, const void *dY, int64_t lddy, void *dYs, int64_t lddys,
                                      float *dweights, sgemm_emu_stream_t stream)
{
    if (!dtype_ok(dtype) || !extent_ok(K)) return SGEMM_EMU_EINVAL;
    CHECK(check_tokens(T, k, n, offsets, places));
    CHECK(check_operand(dtype, T * k, K, Ys, ldys, dweights == nullptr));
    CHECK(check_vector(T * k, weights, 4, true));
    CHECK(check_operand(dtype, T, K, dY, lddy));
    CHECK(check_operand(dtype, T * k, K, dYs, lddys, true));
    CHECK(check_vector(T * k, dweights, 4, true));
    int cus = 0;
    CHECK(current_cus(&cus));
    if (K == 0) {
        if (dweights != nullptr) LAUNCH(launch_clear_floats(dweights, T * k, (hipStream_t)stream));
        return SGEMM_EMU_OK;
    }
    if (dYs == nullptr && dweights == nullptr) return SGEMM_EMU_OK;
    auto call = [&](auto *ys, auto *dys) {
        auto a = route_args<std::remove_pointer_t<decltype(dys)>>(T, k, K, n, offsets, places);
        a.weights = weights; a.rows = ys; a.ldr = ldys; a.x = (decltype(ys))dY; a.ldx = lddy;
        a.rows_out = dys; a.ldr_out = lddys; a.dweights = dweights;
        return launch_route(kCombineBackward, a, (hipStream_t)stream);
    };
    LAUNCH(dtype == SGEMM_EMU_F32 ? call((const float *)Ys, (float *)dYs) : call((const uint16_t *)Ys, (uint16_t *)dYs));
    return SGEMM_EMU_OK;
}

int sgemm_emu_expert_linear(int dtype, int64_t P, int64_t N, int64_t K, int64_t n, const void *X, int64_t ldx,
                            const void *W, const void *bias, int gate, const int32_t *offsets, void *H, int64_t ldh,
                            float *Zkeep, sgemm_emu_stream_t stream)
{
    if (!dtype_ok(dtype) || !extent_ok(P) || !bank_ok(n, N, K)) return SGEMM_EMU_EINVAL;
    CHECK(check_gate(gate, N));
    const int64_t outs = gate >= 0 ? N / 2 : N;
    CHECK(check_operand(dtype, P, K, X, ldx));
    CHECK(check_vector(n * N * K, W, size_of(dtype), false));
    CHECK(check_vector(n * N, bias, size_of(dtype), true));
    CHECK(check_vector(n + 1, offsets, 4, false));
    CHECK(check_operand(dtype, P, outs, H, ldh));
    if ((uintptr_t)Zkeep % 16 != 0 || (Zkeep != nullptr && gate < 0)) return SGEMM_EMU_EINVAL;
    int cus = 0;
    CHECK(current_cus(&cus));
    ExpertProduct g{};
    g.P = P; g.N = N; g.K = K; g.n = n;
    g.offsets = offsets;
    g.A = X; g.lda = ldx;
    g.B = W; g.ldb = K; g.bank = N * K;
    g.bias = bias;
    g.gate = gate;
    g.C = H; g.ldc = ldh;
    g.Z = Zkeep; g.ldz = z_pitch(outs);
    g.num_cus = cus;
    LAUNCH(launch_expert(kForward, dtype, g, (hipStream_t)stream));
    return SGEMM_EMU_OK;
}

int64_t sgemm_emu_expert_linear_backward_workspace(int dtype, int64_t P, int64_t N, int64_t K, int64_t n, int gate,
                                                   int dbias)
{
    if (!dtype_ok(dtype) || !extent_ok(P) || !bank_ok(n, N, K)) return SGEMM_EMU_EINVAL;
    CHECK(check_gate(gate, N));
    return BackwardWs(nullptr, dtype, P, N, K, n, gate, dbias != 0).bytes;
}

int sgemm_emu_expert_linear_backward(int dtype, int64_t P, int64_t N, int64_t K, int64_t n, const void *X, int64_t ldx,
                                     const void *W, const float *Zkeep, int gate, const int32_t *offsets,
                                     const void *dH, int64_t lddh, void *dX, int64_t lddx, void *dW, void *dbias,
                                     void *ws, int64_t ws_bytes, sgemm_emu_stream_t stream)
{
    if (!dtype_ok(dtype) || !extent_ok(P) || !bank_ok(n, N, K)) return SGEMM_EMU_EINVAL;
    CHECK(check_gate(gate, N));
    const int64_t outs = gate >= 0 ? N / 2 : N, elem = size_of(dtype);
    CHECK(check_operand(dtype, P, K, X, ldx, dW == nullptr));
    CHECK(check_vector(n * N * K, W, elem, dX == nullptr));
    if (gate >= 0) {
        CHECK(check_vector(P * outs, Zkeep, 16, false));
    }
    CHECK(check_vector(n + 1, offsets, 4, false));
    CHECK(check_operand(dtype, P, outs, dH, lddh));
    CHECK(check_operand(dtype, P, K, dX, lddx, true));
    CHECK(check_vector(n * N * K, dW, elem, true));
    CHECK(check_vector(n * N, dbias, elem, true));
    const BackwardWs w(ws, dtype, P, N, K, n, gate, dbias != nullptr);
    CHECK(check_ws(ws, ws_bytes, w.bytes));
    int cus = 0;
    CHECK(current_cus(&cus));
    const hipStream_t s = (hipStream_t)stream;
    if (gate >= 0 || dbias != nullptr) {
        ExpertGate q{};
        q.P = P; q.F = outs; q.n = n;
        q.offsets = offsets;
        q.Z = Zkeep;
        q.dH = dH; q.lddh = lddh;
        q.gate = gate;
        q.dZ = dX != nullptr || dW != nullptr ? w.dZ : nullptr;
        q.sums = w.sums;
        q.dbias = dbias;
        LAUNCH(launch_expert_gate(dtype, q, s));
    }
    const void *const dZ = gate >= 0 ? w.dZ : dH;
    const int64_t pitch = gate >= 0 ? expert_dz_pitch(outs) : N;
    ExpertProduct g{};
    g.P = P; g.n = n;
    g.offsets = offsets;
    g.A = dZ; g.lda = gate >= 0 ? pitch : lddh;
    g.gate = -1;
    g.map = Halves{outs, pitch / (gate >= 0 ? 2 : 1)};
    g.num_cus = cus;
    g.N = K;
    if (dX != nullptr) {
        g.K = pitch;
        g.B = W; g.ldb = K; g.bank = N * K;
        g.C = dX; g.ldc = lddx;
        LAUNCH(launch_expert(kBackX, dtype, g, s));
    }
    if (dW != nullptr) {
        g.M = pitch;
        g.B = X; g.ldb = ldx; g.bank = N * K;
        g.C = dW; g.ldc = K;
        g.partials = w.partials; g.chunk = w.chunk;
        LAUNCH(launch_expert(kBackW, dtype, g, s));
    }
    return SGEMM_EMU_OK;
}

int64_t sgemm_emu_quant4_bytes(int64_t n, int64_t N, int64_t K, int64_t group, int zeros)
{
    if (!bank_ok(n, N, K) || !group_ok(group)) return SGEMM_EMU_EINVAL;
    return n * quant4(n, N, K, group, zeros).bank_bytes();
}

int sgemm_emu_quant4_quantize(int dtype, int64_t n, int64_t N, int64_t K, int64_t group, const void *W, uint8_t *q,
                              float *scale, uint8_t *zero, sgemm_emu_stream_t stream)
{
    if (!dtype_ok(dtype) || !bank_ok(n, N, K) || !group_ok(group)) return SGEMM_EMU_EINVAL;
    CHECK(check_vector(n * N * K, W, size_of(dtype), false));
    CHECK(check_vector(n * N * K, q, 1, false));
    CHECK(check_vector(n * N * K, scale, 4, false));
    int cus = 0;
    CHECK(current_cus(&cus));
    LAUNCH(launch_quant4_quantize(dtype, quant4(n, N, K, group, zero != nullptr), W, q, scale, zero,
                                  (hipStream_t)stream));
    return SGEMM_EMU_OK;
}

int sgemm_emu_quant4_pack(int64_t n, int64_t N, int64_t K, int64_t group, const uint8_t *q, const float *scale,
                          const uint8_t *zero, void *packed, sgemm_emu_stream_t stream)
{
    if (!bank_ok(n, N, K) || !group_ok(group)) return SGEMM_EMU_EINVAL;
    CHECK(check_vector(n * N * K, q, 1, false));
    CHECK(check_vector(n * N * K, scale, 4, false));
    CHECK(check_vector(n * N * K, packed, 16, false));
    int cus = 0;
    CHECK(current_cus(&cus));
    LAUNCH(launch_quant4_pack(quant4(n, N, K, group, zero != nullptr), q, scale, zero, packed, (hipStream_t)stream));
    return SGEMM_EMU_OK;
}

int sgemm_emu_quant4_unpack(int dtype, int64_t n, int64_t N, int64_t K, int64_t group, int zeros, const void *packed,
                            void *W, sgemm_emu_stream_t stream)
{
    if (!dtype_ok(dtype) || !bank_ok(n, N, K) || !group_ok(group)) return SGEMM_EMU_EINVAL;
    CHECK(check_vector(n * N * K, packed, 16, false));
    CHECK(check_vector(n * N * K, W, size_of(dtype), false));
    int cus = 0;
    CHECK(current_cus(&cus));
    LAUNCH(launch_quant4_unpack(dtype, quant4(n, N, K, group, zeros), packed, W, (hipStream_t)stream));
    return SGEMM_EMU_OK;
}

int64_t sgemm_emu_quant4_linear_workspace(int dtype, int64_t P, int64_t N, int64_t K, int64_t n, int64_t group,
                                          int zeros)
{
    if (!dtype_ok(dtype) || !extent_ok(P) || !bank_ok(n, N, K) || !group_ok(group)) return SGEMM_EMU_EINVAL;
    return quant4_few(dtype, quant4(n, N, K, group, zeros), P) ? 0 : round_up(n * N * K * size_of(dtype), 256);
}

int sgemm_emu_quant4_linear(int dtype, int64_t P, int64_t N, int64_t K, int64_t n, int64_t group, int zeros,
                            const void *X, int64_t ldx, const void *packed, const void *bias, int gate,
                            const int32_t *offsets, void *H, int64_t ldh, void *ws, int64_t ws_bytes,
                            sgemm_emu_stream_t stream)
{
    if (!dtype_ok(dtype) || !extent_ok(P) || !bank_ok(n, N, K) || !group_ok(group)) return SGEMM_EMU_EINVAL;
    CHECK(check_gate(gate, N));
    if (offsets == nullptr && n != 1) return SGEMM_EMU_EINVAL;
    const int64_t outs = gate >= 0 ? N / 2 : N;
    CHECK(check_operand(dtype, P, K, X, ldx));
    CHECK(check_vector(n * N * K, packed, 16, false));
    CHECK(check_vector(n * N, bias, size_of(dtype), true));
    if ((uintptr_t)offsets % 4 != 0) return SGEMM_EMU_EINVAL;
    CHECK(check_operand(dtype, P, outs, H, ldh));
    CHECK(check_ws(ws, ws_bytes, sgemm_emu_quant4_linear_workspace(dtype, P, N, K, n, group, zeros)));
    int cus = 0;
    CHECK(current_cus(&cus));
    const Quant4 w = quant4(n, N, K, group, zeros);
    const hipStream_t s = (hipStream_t)stream;
    if (quant4_few(dtype, w, P)) {
        Quant4Product g{P, X, ldx, packed, bias, gate, offsets, H, ldh, cus};
        LAUNCH(launch_quant4_few(dtype, w, g, s));
        return SGEMM_EMU_OK;
    }
    LAUNCH(launch_quant4_unpack(dtype, w, packed, ws, s));
    ExpertProduct g{};
    g.P = P; g.N = N; g.K = K; g.n = n;
    g.offsets = offsets;
    g.A = X; g.lda = ldx;
    g.B = ws; g.ldb = K; g.bank = N * K;
    g.bias = bias;
    g.gate = gate;
    g.C = H; g.ldc = ldh;
    g.num_cus = cus;
    LAUNCH(launch_expert(kForward, dtype, g, s));
    return SGEMM_EMU_OK;
}

}  // extern "C"
