// ops_api.hip -- the C ABI declared in include/sgemm_emu_ops.h: argument
// validation, the workspace layouts, and the order of the kernels.
//
// As in api.hip every argument is checked before the first HIP call.  Scratch
// memory is the caller's: each call lays its buffers out in `ws` with the same
// code that its *_workspace function sizes them with (Carve).  What the FP32
// products take of the stream's own workspace is leased before the first launch
// (lease_plane_workspace).
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/sgemm_emu_ops.h"
#include "abi_checks.hpp"
#include "ops.hpp"
#include "workspace.hpp"

using namespace sgemm_emu_dev;

namespace {

// Operands whose rows the GEMM reads as they lie, in 16-byte loads.  The FP32
// kernels also take others, element by element, but then run out of registers:
// 3328 x 371 x 2 5744 gated took 2030 us where the copy makes it 264.
bool direct(int dtype, const void *p, int64_t ld, int64_t K)
{
    const int64_t v = 16 / size_of(dtype);
    return K % v == 0 && ld % v == 0 && aligned(p, 16);
}
// The gated FP32 kernels take K in multiples of the padding only: the masks of a
// ragged K cost registers that they need.
bool gated_direct(int dtype, const void *p, int64_t ld, int64_t K)
{
    return direct(dtype, p, ld, K) && (dtype == SGEMM_EMU_BF16 || K % kPadK == 0);
}
// The K that a bfloat16 product runs over: operands are padded copies unless K is a multiple of 8.
int64_t bf16_k(int64_t K) { return K % 8 == 0 ? K : pad_k(K); }

// The arguments of an FP32 product C = A B^T + bias (B as padded planes, K > 0).
GemmArgs product_f32(int64_t M, int64_t N, int64_t K, const float *A, int64_t lda, const uint16_t *planes,
                     const float *bias, float *C, int64_t ldc)
{
    const int64_t plane = N * pad_k(K);
    GemmArgs g{};
    g.M = M; g.N = N; g.K = K;
    g.A = A; g.lda = lda;
    g.B0 = planes; g.B1 = planes + plane; g.B2 = planes + 2 * plane;
    g.C = C; g.ldc = ldc;
    g.bias = bias;
    g.act = SGEMM_EMU_ACT_NONE;
    return g;
}

// A product without a fused epilogue; an empty K leaves zeros.
int plain_f32(int64_t M, int64_t N, int64_t K, const float *A, int64_t lda, const uint16_t *planes, float *C,
              int64_t ldc, int num_cus, WsLease &lease, hipStream_t stream)
{
    if (M == 0 || N == 0) return SGEMM_EMU_OK;
    if (K == 0) {
        LAUNCH(launch_zero(M, N, C, ldc, nullptr, SGEMM_EMU_ACT_NONE, num_cus, stream));
        return SGEMM_EMU_OK;
    }
    return gemm_padded_planes(product_f32(M, N, K, A, lda, planes, nullptr, C, ldc), plain_launchers(), lease,
                              stream);
}

// The product with the adapters' part (or none).  A ragged K whose rows lie takes
// the plain kernels and a pass over C: a padded copy of A for the fused ones cost
// as much or more (3136 x 336 x 3592: 128 us against 114).
int adapted_f32(int64_t M, int64_t N, int64_t K, const float *A, int64_t lda, const uint16_t *planes,
                const float *bias, const Adapters *ad, const float *S, float *C, int64_t ldc, WsLease &lease,
                hipStream_t stream)
{
    GemmArgs g = product_f32(M, N, K, A, lda, planes, bias, C, ldc);
    if (ad == nullptr) return gemm_padded_planes(g, plain_launchers(), lease, stream);
    g.epi.gate = -1;
    g.epi.ids = ad->ids;
    g.epi.n = ad->n; g.epi.r = ad->r; g.epi.rp = rank_pad(ad->r);
    g.epi.up = (const float *)ad->up;
    g.epi.S = S;
    if (K % kPadK == 0) return gemm_padded_planes(g, adapter_launchers(), lease, stream);
    CHECK(gemm_padded_planes(g, plain_launchers(), lease, stream));
    LAUNCH(launch_expand(M, N, g.epi, C, ldc, stream));
    return SGEMM_EMU_OK;
}

// ---------------------------------------------------------------- gated projection

int check_gated(int dtype, int64_t M, int64_t F, int64_t K, int gate)
{
    // F by itself first: 2 F of an F near INT64_MIN wraps to a small number
    if (!dtype_ok(dtype) || !extent_ok(M) || !extent_ok(F) || !extent_ok(2 * F) || !extent_ok(K))
        return SGEMM_EMU_EINVAL;
    if (gate < SGEMM_EMU_GATE_SILU || gate > SGEMM_EMU_GATE_RELU) return SGEMM_EMU_EINVAL;
    return SGEMM_EMU_OK;
}

// Few rows read W in one pass; pre-activations to keep come from the tiles.
bool gated_few(int64_t M, int64_t K, const void *Z) { return M <= kFewRows && Z == nullptr && K > 0; }

struct GatedWs {
    uint16_t *plan;       // W laid out
    void *x;              // X in padded rows
    float *partials;      // few rows' K slices
    int64_t bytes;
};
GatedWs gated_ws(int dtype, int64_t M, int64_t F, int64_t K, const void *X, int64_t ldx, const void *W, int64_t ldw,
                 const void *plan, const void *Z, int num_cus, void *ws)
{
    Carve c(ws);
    GatedWs w{};
    if (M == 0 || F == 0) return w;
    if (gated_few(M, K, Z)) {
        w.partials = c.take<float>(few_rows_partial_floats(dtype, M, F, K, SGEMM_EMU_GATE_SILU, num_cus));
    } else if (dtype == SGEMM_EMU_F32) {
        if (plan == nullptr) w.plan = c.take<uint16_t>(3 * 2 * F * pad_k(K));
        if (!gated_direct(dtype, X, ldx, K)) w.x = c.take<float>(M * pad_k(K));
    } else {
        if (plan == nullptr && !direct(dtype, W, ldw, K)) w.plan = c.take<uint16_t>(2 * F * pad_k(K));
        if (!gated_direct(dtype, X, ldx, K)) w.x = c.take<uint16_t>(M * pad_k(K));
    }
    w.bytes = c.bytes;
    return w;
}

struct GatedBackWs {
    void *dz, *dzt;          // M x dz_pitch(F), 2F x pad(M)
    uint16_t *wt, *xt;       // W^T (columns as dz's) and X^T laid out
    float *sums, *part_x, *part_w;
    int64_t bytes;
};
GatedBackWs gated_back_ws(int dtype, int64_t M, int64_t F, int64_t K, int num_cus, void *ws)
{
    Carve c(ws);
    GatedBackWs w{};
    const int64_t size = size_of(dtype), comps = dtype == SGEMM_EMU_F32 ? 3 : 1, pitch = dz_pitch(F);
    w.dz = c.take<char>(M * pitch * size);
    w.dzt = c.take<char>(2 * F * pad_k(M) * size);
    w.wt = c.take<uint16_t>(comps * K * pitch);
    w.xt = c.take<uint16_t>(comps * K * pad_k(M));
    w.sums = c.take<float>(gate_tiles(M) * 2 * F);
    if (dtype == SGEMM_EMU_BF16) {
        w.part_x = c.take<float>(bf16_gemm_partial_floats(M, K, pitch, true, num_cus));
        w.part_w = c.take<float>(bf16_gemm_partial_floats(2 * F, K, pad_k(M), true, num_cus));
    }
    w.bytes = c.bytes;
    return w;
}

// W^T with the columns of dZ: F gate columns, zeros to dz_pitch / 2, F up columns, zeros.
hipError_t lay_out_wt(int dtype, int64_t F, int64_t K, const void *W, int64_t ldw, uint16_t *wt, int num_cus,
                      hipStream_t s)
{
    const int64_t pitch = dz_pitch(F), half = pitch / 2, plane = K * pitch;
    for (int64_t h = 0; h < 2; ++h) {
        uint16_t *const P = wt + h * half;
        hipError_t e;
        if (dtype == SGEMM_EMU_F32)
            e = launch_split_transpose(F, K, (const float *)W + h * F * ldw, ldw, P, P + plane, P + 2 * plane, pitch,
                                       num_cus, s, false, half);
        else
            e = launch_transpose_padded(F, K, (const uint16_t *)W + h * F * ldw, ldw, P, half, pitch, s);
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

// ---------------------------------------------------------------- adapters

int check_adapters(int dtype, int64_t M, int64_t N, int64_t K, int64_t n, int64_t r)
{
    if (!dtype_ok(dtype) || !extent_ok(M) || !extent_ok(N) || !extent_ok(K) || !extent_ok(r)) return SGEMM_EMU_EINVAL;
    if (n < 0 || n > kMaxAdapters) return SGEMM_EMU_EINVAL;
    // The banks, their copies (ranks padded up to 16 times) and their gradients' partial
    // sums then take less than 2^62 bytes.
    if (n > 0 && r > 0 && K + N > 0 && n > kMaxBankElems / (r * (K + N))) return SGEMM_EMU_EINVAL;
    return SGEMM_EMU_OK;
}

// Few rows read W in one pass; low-rank activations to keep come from the tiles' path.
bool adapter_few(int64_t M, const float *S) { return M <= kFewRows && S == nullptr; }

// A bfloat16 bank of up factors whose rows the GEMM reads as they lie (whole dwords).
bool bank_lies(int64_t r, const void *up) { return r % 2 == 0 && aligned(up, 4); }

struct AdapterWs {
    uint16_t *plan, *up;
    void *x;
    float *s, *partials;
    int64_t bytes;
};
AdapterWs adapter_ws(int dtype, int64_t M, int64_t N, int64_t K, const void *X, int64_t ldx, const void *W,
                     int64_t ldw, const void *plan, int64_t n, int64_t r, const void *up, const float *S, int num_cus,
                     void *ws)
{
    Carve c(ws);
    AdapterWs w{};
    if (M == 0 || N == 0) return w;
    if (n > 0 && r > 0 && S == nullptr) w.s = c.take<float>(M * rank_pad(r));
    if (adapter_few(M, S)) {
        w.partials = c.take<float>(few_rows_partial_floats(dtype, M, N, K, -1, num_cus));
    } else if (dtype == SGEMM_EMU_F32) {
        if (plan == nullptr) w.plan = c.take<uint16_t>(3 * N * pad_k(K));
        if (!direct(dtype, X, ldx, K)) w.x = c.take<float>(M * pad_k(K));
    } else {
        if (plan == nullptr && !direct(dtype, W, ldw, K)) w.plan = c.take<uint16_t>(N * pad_k(K));
        if (!direct(dtype, X, ldx, K)) w.x = c.take<uint16_t>(M * pad_k(K));
        if (n > 0 && r > 0 && !bank_lies(r, up)) w.up = c.take<uint16_t>(n * N * rank_pad(r));
    }
    w.bytes = c.bytes;
    return w;
}

struct AdapterBackWs {
    void *up_t, *down_t;       // n x r x N, n x K x r
    float *p;                  // M x pad16(r)
    void *dy;                  // dY in padded rows
    uint16_t *down_p;          // down_t's rows padded
    int32_t *offs, *rows;
    float *partials;
    int64_t bytes;
};
AdapterBackWs adapter_back_ws(int dtype, int64_t M, int64_t N, int64_t K, int64_t n, int64_t r, int num_cus, void *ws)
{
    Carve c(ws);
    AdapterBackWs w{};
    const int64_t size = size_of(dtype);
    w.dy = c.take<char>(M * pad_k(N) * size);
    if (n > 0 && r > 0) {
        w.up_t = c.take<char>(n * r * N * size);
        w.down_t = c.take<char>(n * r * K * size);
        if (dtype == SGEMM_EMU_BF16 && r % 2 != 0) w.down_p = c.take<uint16_t>(n * K * rank_pad(r));
        w.p = c.take<float>(M * rank_pad(r));
        w.offs = c.take<int32_t>(n + 1);
        w.rows = c.take<int32_t>(M);
        w.partials = c.take<float>(lowrank_grad_floats(dtype, M, K, N, n, r, num_cus));
    }
    w.bytes = c.bytes;
    return w;
}

}  // namespace

extern "C" {

int sgemm_emu_few_rows(void) { return (int)kFewRows; }

int64_t sgemm_emu_plan_bytes(int dtype, int64_t rows, int64_t cols, int layout)
{
    if (!dtype_ok(dtype) || !extent_ok(rows) || !extent_ok(cols)) return SGEMM_EMU_EINVAL;
    if (layout < SGEMM_EMU_PLAN_ROWS || layout > SGEMM_EMU_PLAN_GATED) return SGEMM_EMU_EINVAL;
    if (layout == SGEMM_EMU_PLAN_GATED && rows % 2 != 0) return SGEMM_EMU_EINVAL;
    const bool transposed = layout == SGEMM_EMU_PLAN_TRANSPOSED;
    const int64_t comps = dtype == SGEMM_EMU_F32 ? 3 : 1;
    return 2 * comps * (transposed ? cols * pad_k(rows) : rows * pad_k(cols));
}

int sgemm_emu_plan_weight(int dtype, int64_t rows, int64_t cols, const void *W, int64_t ldw, int layout,
                          void *plan, sgemm_emu_stream_t stream)
{
    const int64_t bytes = sgemm_emu_plan_bytes(dtype, rows, cols, layout);
    const bool transposed = layout == SGEMM_EMU_PLAN_TRANSPOSED;
    if (bytes < 0) return (int)bytes;
    CHECK(check_operand(dtype, rows, cols, W, ldw));
    if (bytes > 0 && plan == nullptr) return SGEMM_EMU_ENULL;
    if ((uintptr_t)plan % 16 != 0) return SGEMM_EMU_EINVAL;
    if (bytes == 0) return SGEMM_EMU_OK;
    int num_cus = 0;
    CHECK(current_cus(&num_cus));
    hipStream_t s = (hipStream_t)stream;
    uint16_t *P = (uint16_t *)plan;
    if (dtype == SGEMM_EMU_F32) {
        if (transposed) {
            const int64_t rp = pad_k(rows), plane = cols * rp;
            LAUNCH(launch_split_transpose(rows, cols, (const float *)W, ldw, P, P + plane, P + 2 * plane, rp, num_cus,
                                          s, false, rp));
        } else {
            LAUNCH(launch_split_padded(rows, cols, (const float *)W, ldw, P, layout == SGEMM_EMU_PLAN_GATED, s));
        }
    } else if (transposed) {
        LAUNCH(launch_transpose_padded(rows, cols, (const uint16_t *)W, ldw, P, pad_k(rows), pad_k(rows), s));
    } else {
        LAUNCH(launch_copy_padded(dtype, rows, cols, W, ldw, P, pad_k(cols), s));
    }
    return SGEMM_EMU_OK;
}

int64_t sgemm_emu_gated_linear_workspace(int dtype, int64_t M, int64_t F, int64_t K, const void *X, int64_t ldx,
                                         const void *W, int64_t ldw, const void *plan, const void *Z)
{
    CHECK(check_gated(dtype, M, F, K, SGEMM_EMU_GATE_SILU));
    int num_cus = 0;
    CHECK(current_cus(&num_cus));
    return gated_ws(dtype, M, F, K, X, ldx, W, ldw, plan, Z, num_cus, nullptr).bytes;
}

int sgemm_emu_gated_linear(int dtype, int64_t M, int64_t F, int64_t K, const void *X, int64_t ldx, const void *W,
                           int64_t ldw, const void *plan, const void *bias, int gate, void *H, int64_t ldh, float *Z,
                           void *ws, int64_t ws_bytes, sgemm_emu_stream_t stream)
{
    CHECK(check_gated(dtype, M, F, K, gate));
    CHECK(check_operand(dtype, M, K, X, ldx));
    CHECK(check_operand(dtype, 2 * F, K, W, ldw));
    CHECK(check_vector(2 * F, bias, size_of(dtype), true));
    CHECK(check_operand(dtype, M, F, H, ldh));
    if ((uintptr_t)plan % 16 != 0 || (uintptr_t)Z % 16 != 0) return SGEMM_EMU_EINVAL;
    if (M == 0 || F == 0) return SGEMM_EMU_OK;
    int num_cus = 0;
    CHECK(current_cus(&num_cus));
    const GatedWs w = gated_ws(dtype, M, F, K, X, ldx, W, ldw, plan, Z, num_cus, ws);
    CHECK(check_ws(ws, ws_bytes, w.bytes));
    hipStream_t s = (hipStream_t)stream;
    if (gated_few(M, K, Z)) {
        FewRows a{};
        a.M = M; a.N = F; a.K = K;
        a.X = X; a.ldx = ldx; a.W = W; a.ldw = ldw;
        a.bias = bias; a.gate = gate;
        a.Y = H; a.ldy = ldh;
        a.partials = w.partials;
        LAUNCH(launch_few_rows(dtype, a, num_cus, s));
        return SGEMM_EMU_OK;
    }
    if (dtype == SGEMM_EMU_F32) {
        if (K == 0) {
            LAUNCH(launch_gate_bias(M, F, (const float *)bias, gate, (float *)H, ldh, Z, s));
            return SGEMM_EMU_OK;
        }
        const PlaneProduct product{M, 2 * F, pad_k(K)};
        WsLease lease;
        CHECK(lease_plane_workspace(&product, 1, s, lease));
        if (w.plan != nullptr) LAUNCH(launch_split_padded(2 * F, K, (const float *)W, ldw, w.plan, true, s));
        if (w.x != nullptr) LAUNCH(launch_copy_padded(dtype, M, K, X, ldx, w.x, pad_k(K), s));
        GemmArgs g = product_f32(M, 2 * F, pad_k(K), w.x != nullptr ? (const float *)w.x : (const float *)X,
                                 w.x != nullptr ? pad_k(K) : ldx,
                                 w.plan != nullptr ? w.plan : (const uint16_t *)plan, (const float *)bias, (float *)H,
                                 ldh);
        g.epi.gate = gate;
        g.epi.Z = Z;
        g.epi.ldz = z_pitch(F);
        return gemm_padded_planes(g, gated_launchers(), lease, s);
    }
    Bf16Gemm g{};
    g.M = M; g.N = 2 * F; g.K = bf16_k(K);
    g.A = (const uint16_t *)X; g.lda = ldx;
    if (w.x != nullptr) {
        LAUNCH(launch_copy_padded(dtype, M, K, X, ldx, w.x, pad_k(K), s));
        g.A = (const uint16_t *)w.x; g.lda = pad_k(K);
    }
    g.B = (const uint16_t *)W; g.ldb = ldw;
    if (plan != nullptr) {
        g.B = (const uint16_t *)plan; g.ldb = pad_k(K);
    } else if (w.plan != nullptr) {
        LAUNCH(launch_copy_padded(dtype, 2 * F, K, W, ldw, w.plan, pad_k(K), s));
        g.B = w.plan; g.ldb = pad_k(K);
    }
    g.bias = (const uint16_t *)bias;
    g.C = (uint16_t *)H; g.ldc = ldh;
    g.gate = gate;
    g.Z = Z; g.ldz = z_pitch(F);
    LAUNCH(launch_bf16_gemm(g, num_cus, s));
    return SGEMM_EMU_OK;
}

int64_t sgemm_emu_gated_linear_backward_workspace(int dtype, int64_t M, int64_t F, int64_t K)
{
    CHECK(check_gated(dtype, M, F, K, SGEMM_EMU_GATE_SILU));
    int num_cus = 0;
    CHECK(current_cus(&num_cus));
    return gated_back_ws(dtype, M, F, K, num_cus, nullptr).bytes;
}

int sgemm_emu_gated_linear_backward(int dtype, int64_t M, int64_t F, int64_t K, const void *X, int64_t ldx,
                                    const void *W, int64_t ldw, const float *Z, int gate, const void *dH,
                                    int64_t lddh, void *dX, int64_t lddx, void *dW, int64_t lddw, void *dbias,
                                    void *ws, int64_t ws_bytes, sgemm_emu_stream_t stream)
{
    CHECK(check_gated(dtype, M, F, K, gate));
    CHECK(check_operand(dtype, M, K, X, ldx, dW == nullptr));
    CHECK(check_operand(dtype, 2 * F, K, W, ldw, dX == nullptr));
    CHECK(check_vector(M > 0 ? F : 0, Z, 16, false));
    CHECK(check_operand(dtype, M, F, dH, lddh));
    CHECK(check_operand(dtype, M, K, dX, lddx, true));
    CHECK(check_operand(dtype, 2 * F, K, dW, lddw, true));
    CHECK(check_vector(2 * F, dbias, size_of(dtype), true));
    int num_cus = 0;
    CHECK(current_cus(&num_cus));
    const GatedBackWs w = gated_back_ws(dtype, M, F, K, num_cus, ws);
    CHECK(check_ws(ws, ws_bytes, w.bytes));
    hipStream_t s = (hipStream_t)stream;
    const int64_t n2 = 2 * F, pitch = dz_pitch(F), mp = pad_k(M);
    WsLease lease;
    if (dtype == SGEMM_EMU_F32 && M > 0 && F > 0 && K > 0) {
        PlaneProduct products[2];
        int count = 0;
        if (dX != nullptr) products[count++] = {M, K, pitch};
        if (dW != nullptr) products[count++] = {n2, K, mp};
        CHECK(lease_plane_workspace(products, count, s, lease));
    }
    if (M > 0 && F > 0)
        LAUNCH(launch_gate_backward(dtype, M, F, Z, dH, lddh, gate, dX != nullptr ? w.dz : nullptr,
                                    dW != nullptr ? w.dzt : nullptr, dbias != nullptr ? w.sums : nullptr, s));
    if (dbias != nullptr && F > 0) LAUNCH(launch_sum_tiles(dtype, gate_tiles(M), n2, w.sums, dbias, s));
    if (dX != nullptr && M > 0 && K > 0) {
        if (F > 0) LAUNCH(lay_out_wt(dtype, F, K, W, ldw, w.wt, num_cus, s));
        if (dtype == SGEMM_EMU_F32) {
            CHECK(plain_f32(M, K, pitch, (const float *)w.dz, pitch, w.wt, (float *)dX, lddx, num_cus, lease, s));
        } else {
            Bf16Gemm g{};
            g.M = M; g.N = K; g.K = pitch;
            g.A = (const uint16_t *)w.dz; g.lda = pitch;
            g.B = w.wt; g.ldb = pitch;
            g.C = (uint16_t *)dX; g.ldc = lddx;
            g.gate = -1;
            g.partials = w.part_x;
            LAUNCH(launch_bf16_gemm(g, num_cus, s));
        }
    }
    if (dW != nullptr && F > 0 && K > 0) {
        if (M > 0) CHECK(sgemm_emu_plan_weight(dtype, M, K, X, ldx, SGEMM_EMU_PLAN_TRANSPOSED, w.xt, stream));
        if (dtype == SGEMM_EMU_F32) {
            CHECK(plain_f32(n2, K, mp, (const float *)w.dzt, mp, w.xt, (float *)dW, lddw, num_cus, lease, s));
        } else {
            Bf16Gemm g{};
            g.M = n2; g.N = K; g.K = mp;
            g.A = (const uint16_t *)w.dzt; g.lda = mp;
            g.B = w.xt; g.ldb = mp;
            g.C = (uint16_t *)dW; g.ldc = lddw;
            g.gate = -1;
            g.partials = w.part_w;
            LAUNCH(launch_bf16_gemm(g, num_cus, s));
        }
    }
    return SGEMM_EMU_OK;
}

int64_t sgemm_emu_adapter_linear_workspace(int dtype, int64_t M, int64_t N, int64_t K, const void *X, int64_t ldx,
                                           const void *W, int64_t ldw, const void *plan, int64_t n, int64_t r,
                                           const void *up, const float *S)
{
    CHECK(check_adapters(dtype, M, N, K, n, r));
    int num_cus = 0;
    CHECK(current_cus(&num_cus));
    return adapter_ws(dtype, M, N, K, X, ldx, W, ldw, plan, n, r, up, S, num_cus, nullptr).bytes;
}

int sgemm_emu_adapter_linear(int dtype, int64_t M, int64_t N, int64_t K, const void *X, int64_t ldx, const void *W,
                             int64_t ldw, const void *plan, const void *bias, int64_t n, int64_t r, const void *down,
                             const void *up, const float *scale, const int32_t *ids, void *Y, int64_t ldy, float *S,
                             void *ws, int64_t ws_bytes, sgemm_emu_stream_t stream)
{
    CHECK(check_adapters(dtype, M, N, K, n, r));
    CHECK(check_operand(dtype, M, K, X, ldx));
    CHECK(check_operand(dtype, N, K, W, ldw));
    CHECK(check_vector(N, bias, size_of(dtype), true));
    CHECK(check_operand(dtype, M, N, Y, ldy));
    const bool low = n > 0 && r > 0;
    if (low) {
        CHECK(check_vector(K, down, size_of(dtype), false));
        CHECK(check_vector(N, up, size_of(dtype), false));
        CHECK(check_vector(n, scale, 4, true));
        CHECK(check_vector(M, ids, 4, false));
        if ((uintptr_t)S % 16 != 0) return SGEMM_EMU_EINVAL;
    }
    if ((uintptr_t)plan % 16 != 0) return SGEMM_EMU_EINVAL;
    if (M == 0 || (N == 0 && (!low || S == nullptr))) return SGEMM_EMU_OK;
    int num_cus = 0;
    CHECK(current_cus(&num_cus));
    const AdapterWs w = adapter_ws(dtype, M, N, K, X, ldx, W, ldw, plan, n, r, up, S, num_cus, ws);
    CHECK(check_ws(ws, ws_bytes, w.bytes));
    hipStream_t s = (hipStream_t)stream;
    const Adapters ad{ids, n, r, down, up, scale};
    if (adapter_few(M, S)) {
        FewRows a{};
        a.M = M; a.N = N; a.K = K;
        a.X = X; a.ldx = ldx; a.W = W; a.ldw = ldw;
        a.bias = bias; a.gate = -1;
        a.Y = Y; a.ldy = ldy;
        a.ad = low ? &ad : nullptr;
        a.S = w.s;
        a.partials = w.partials;
        LAUNCH(launch_few_rows(dtype, a, num_cus, s));
        return SGEMM_EMU_OK;
    }
    WsLease lease;
    const int64_t kx = w.x != nullptr ? pad_k(K) : K;            // the FP32 product's K
    if (dtype == SGEMM_EMU_F32 && N > 0 && K > 0) {
        const PlaneProduct product{M, N, kx};
        CHECK(lease_plane_workspace(&product, 1, s, lease));
    }
    if (low) {
        if (S == nullptr) S = w.s;
        LAUNCH(launch_shrink(dtype, M, K, X, ldx, ad, S, num_cus, s));
        if (N == 0) return SGEMM_EMU_OK;
    }
    if (dtype == SGEMM_EMU_F32) {
        if (K == 0) {
            // S is zero too: Y is the bias
            LAUNCH(launch_zero(M, N, (float *)Y, ldy, (const float *)bias, SGEMM_EMU_ACT_NONE, num_cus, s));
            return SGEMM_EMU_OK;
        }
        if (w.plan != nullptr) LAUNCH(launch_split_padded(N, K, (const float *)W, ldw, w.plan, false, s));
        if (w.x != nullptr) LAUNCH(launch_copy_padded(dtype, M, K, X, ldx, w.x, pad_k(K), s));
        return adapted_f32(M, N, kx, w.x != nullptr ? (const float *)w.x : (const float *)X,
                           w.x != nullptr ? kx : ldx, w.plan != nullptr ? w.plan : (const uint16_t *)plan,
                           (const float *)bias, low ? &ad : nullptr, S, (float *)Y, ldy, lease, s);
    }
    Bf16Gemm g{};
    g.M = M; g.N = N; g.K = bf16_k(K);
    g.A = (const uint16_t *)X; g.lda = ldx;
    if (w.x != nullptr) {
        LAUNCH(launch_copy_padded(dtype, M, K, X, ldx, w.x, pad_k(K), s));
        g.A = (const uint16_t *)w.x; g.lda = pad_k(K);
    }
    g.B = (const uint16_t *)W; g.ldb = ldw;
    if (plan != nullptr) {
        g.B = (const uint16_t *)plan; g.ldb = pad_k(K);
    } else if (w.plan != nullptr) {
        LAUNCH(launch_copy_padded(dtype, N, K, W, ldw, w.plan, pad_k(K), s));
        g.B = w.plan; g.ldb = pad_k(K);
    }
    g.bias = (const uint16_t *)bias;
    g.C = (uint16_t *)Y; g.ldc = ldy;
    g.gate = -1;
    if (low) {
        g.ids = ids; g.n = n; g.r = r; g.rp = rank_pad(r);
        g.up = (const uint16_t *)up;
        if (!bank_lies(r, up)) {
            LAUNCH(launch_copy_padded(dtype, n * N, r, up, r, w.up, rank_pad(r), s));
            g.r = rank_pad(r);
            g.up = w.up;
        }
        g.S = (const uint16_t *)S;
    }
    LAUNCH(launch_bf16_gemm(g, num_cus, s));
    return SGEMM_EMU_OK;
}

int64_t sgemm_emu_adapter_linear_backward_workspace(int dtype, int64_t M, int64_t N, int64_t K, int64_t n, int64_t r)
{
    CHECK(check_adapters(dtype, M, N, K, n, r));
    int num_cus = 0;
    CHECK(current_cus(&num_cus));
    return adapter_back_ws(dtype, M, N, K, n, r, num_cus, nullptr).bytes;
}

int sgemm_emu_adapter_linear_backward(int dtype, int64_t M, int64_t N, int64_t K, const void *X, int64_t ldx,
                                      const void *plan_t, int64_t n, int64_t r, const void *down, const void *up,
                                      const float *scale, const int32_t *ids, const float *S, const void *dY,
                                      int64_t lddy, void *dX, int64_t lddx, void *d_down, void *d_up, void *ws,
                                      int64_t ws_bytes, sgemm_emu_stream_t stream)
{
    CHECK(check_adapters(dtype, M, N, K, n, r));
    const bool low = n > 0 && r > 0;
    CHECK(check_operand(dtype, M, K, X, ldx, d_down == nullptr));
    CHECK(check_operand(dtype, M, N, dY, lddy));
    CHECK(check_operand(dtype, M, K, dX, lddx, true));
    if (dX != nullptr && M > 0 && N > 0 && K > 0 && plan_t == nullptr) return SGEMM_EMU_ENULL;
    if ((uintptr_t)plan_t % 16 != 0) return SGEMM_EMU_EINVAL;
    if (low) {
        CHECK(check_vector(K, down, size_of(dtype), false));
        CHECK(check_vector(N, up, size_of(dtype), false));
        CHECK(check_vector(n, scale, 4, true));
        CHECK(check_vector(M, ids, 4, false));
        CHECK(check_vector(M, S, 16, d_up == nullptr));
        CHECK(check_vector(K, d_down, size_of(dtype), true));
        CHECK(check_vector(N, d_up, size_of(dtype), true));
    }
    int num_cus = 0;
    CHECK(current_cus(&num_cus));
    const AdapterBackWs w = adapter_back_ws(dtype, M, N, K, n, r, num_cus, ws);
    CHECK(check_ws(ws, ws_bytes, w.bytes));
    hipStream_t s = (hipStream_t)stream;
    // P = scale up^T dY is the shrink of dY by the transposed up factors, and dX
    // the forward of dY through W^T with the factors' roles exchanged.
    const Adapters back{ids, n, r, w.up_t, w.down_t, scale};
    const bool need_dx = dX != nullptr && M > 0 && K > 0, need_down = low && d_down != nullptr && K > 0,
               need_up = low && d_up != nullptr && N > 0;
    const bool lies = direct(dtype, dY, lddy, N);
    WsLease lease;
    if (dtype == SGEMM_EMU_F32 && need_dx && N > 0) {
        const PlaneProduct product{M, K, lies ? N : pad_k(N)};
        CHECK(lease_plane_workspace(&product, 1, s, lease));
    }
    if (low) {
        const bool need_p = M > 0 && (need_dx || need_down), need_rows = need_down || need_up;
        AdapterPrepare q{};
        q.bank[0] = {N, r, up, need_p ? w.up_t : nullptr};
        q.bank[1] = {r, K, down, need_dx ? w.down_t : nullptr};
        q.n = n; q.M = M; q.ids = ids;
        q.offs = need_rows ? w.offs : nullptr;
        q.rows = w.rows;
        LAUNCH(launch_adapter_prepare(dtype, q, s));
        if (need_p) LAUNCH(launch_shrink(dtype, M, N, dY, lddy, back, w.p, num_cus, s));
    }
    if (need_dx) {
        if (!lies && N > 0) LAUNCH(launch_copy_padded(dtype, M, N, dY, lddy, w.dy, pad_k(N), s));
        if (dtype == SGEMM_EMU_F32) {
            if (N == 0)
                LAUNCH(launch_zero(M, K, (float *)dX, lddx, nullptr, SGEMM_EMU_ACT_NONE, num_cus, s));
            else
                CHECK(adapted_f32(M, K, lies ? N : pad_k(N), lies ? (const float *)dY : (const float *)w.dy,
                                  lies ? lddy : pad_k(N), (const uint16_t *)plan_t, nullptr, low ? &back : nullptr,
                                  w.p, (float *)dX, lddx, lease, s));
        } else {
            Bf16Gemm g{};
            g.M = M; g.N = K; g.K = bf16_k(N);
            g.A = (const uint16_t *)dY; g.lda = lddy;
            if (!lies) { g.A = (const uint16_t *)w.dy; g.lda = pad_k(N); }
            g.B = (const uint16_t *)plan_t; g.ldb = pad_k(N);
            g.C = (uint16_t *)dX; g.ldc = lddx;
            g.gate = -1;
            if (low) {
                g.ids = ids; g.n = n; g.r = r; g.rp = rank_pad(r);
                g.up = (const uint16_t *)w.down_t;
                if (r % 2 != 0) {
                    LAUNCH(launch_copy_padded(dtype, n * K, r, w.down_t, r, w.down_p, rank_pad(r), s));
                    g.r = rank_pad(r);
                    g.up = w.down_p;
                }
                g.S = (const uint16_t *)w.p;
            }
            LAUNCH(launch_bf16_gemm(g, num_cus, s));
        }
    }
    if (need_down || need_up) {
        LowrankGrads q{};
        q.M = M; q.K = K; q.N = N; q.n = n; q.r = r;
        q.P = w.p; q.S = S;
        q.X = X; q.ldx = ldx;
        q.dY = dY; q.lddy = lddy;
        q.offs = w.offs; q.rows = w.rows;
        q.down = need_down ? d_down : nullptr;
        q.up = need_up ? d_up : nullptr;
        q.partials = w.partials;
        LAUNCH(launch_lowrank_grad(dtype, q, num_cus, s));
    }
    return SGEMM_EMU_OK;
}

}  // extern "C"
