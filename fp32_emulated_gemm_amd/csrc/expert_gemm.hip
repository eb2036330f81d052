// expert_gemm.hip -- the experts' products: which kernels a call takes, and the
// bfloat16 products whose rows do not lie in 16-byte pieces (odd widths, odd strides).
//
// One workgroup per output tile; a row tile lies inside one expert, found from the
// offsets on the device, so nothing waits for the host.  The grid is the most
// tiles that any offsets can give; workgroups past the last tile end at once.
// Operands come in two layouts: rows with k contiguous (X, W in the forward), or
// rows of k with the other index contiguous (W in dX, dZ and X in dW); the second
// kind is read out of LDS by ds_read_b64_tr_b16.
//
// Here a step's operands pass through registers, loaded a step ahead, 16 bytes at a
// time at any element's address, with the ends of rows element by element: 509 TFLOP/s
// on 16382 x 2048 -> 2 x 1365 gated, where the copies of expert_bf16.hip reach 640.
#include "expert_stage.hpp"

namespace sgemm_emu_dev {

namespace {

typedef uint16_t T;
enum { FORWARD = kForward, BACK_X = kBackX, BACK_W = kBackW };

// What a tile multiplies: addresses of its operands' chunks.
struct Place {
    int64_t e, m0, m_end, n0, K;     // expert; rows and their end; first column; inner extent
    int64_t r0;                      // dW: the expert's first row
};

template <class TL, int OP, bool GATED>
__device__ __forceinline__ u32x4_t load_a(const ExpertProduct &g, const Place &t, int64_t k0, int piece)
{
    constexpr int V = Elem<T>::VEC, ROW = (OP == BACK_W ? TL::BM : BK) / V;
    const T *const A = (const T *)g.A;
    const int r = piece / ROW, c = piece % ROW * V;
    if constexpr (OP == BACK_W) return load_piece<T>(A + (t.r0 + k0 + r) * g.lda + t.m0 + c, k0 + r < t.K ? g.M - t.m0 - c : 0);
    else return load_piece<T>(A + lmin(t.m0 + r, t.m_end - 1) * g.lda + k0 + c, t.K - k0 - c);
}

template <class TL, int OP, bool GATED>
__device__ __forceinline__ u32x4_t load_b(const ExpertProduct &g, const Place &t, int64_t k0, int piece)
{
    constexpr int V = Elem<T>::VEC, ROW = (OP == FORWARD ? BK : TL::BN) / V;
    const T *const B = (const T *)g.B + (OP == BACK_W ? 0 : t.e * g.bank);
    const int r = piece / ROW, c = piece % ROW * V;
    if constexpr (OP == FORWARD) {
        const int64_t n = GATED ? gated_row(g.N >> 1, t.n0, r) : lmin(t.n0 + r, g.N - 1);
        return load_piece<T>(B + n * g.ldb + k0 + c, t.K - k0 - c);
    } else {
        const int64_t row = OP == BACK_W ? t.r0 + k0 + r : g.map.row(k0 + r);
        return load_piece<T>(B + row * g.ldb + t.n0 + c, k0 + r < t.K && row >= 0 ? g.N - t.n0 - c : 0);
    }
}

template <class TL, int OP, int GATE>
__global__ __launch_bounds__(TL::NT) void expert_kernel(ExpertProduct g)
{
    constexpr int NT = TL::NT;
    constexpr bool GATED = GATE >= 0;
    typedef Stage<T, TL::BM, OP == BACK_W, 1, NT> SA;
    typedef Stage<T, TL::BN, OP != FORWARD, 1, NT> SB;
    __shared__ __attribute__((aligned(16))) uint16_t lds[2][SA::ELEMS + SB::ELEMS];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wm = wave / TL::WAVES_N, wn = wave % TL::WAVES_N;

    Place t;
    int tm, tn;
    if constexpr (OP == BACK_W) {
        const int per = g.tiles_m * g.tiles_n;
        const int v = workgroup() % per;
        t.e = workgroup() / per;
        if (t.e >= g.n) return;
        tile_at(xcd_order(v, per), g.tiles_m, g.tiles_n, imin(g.tiles_m, 8), tm, tn);
        t.m0 = (int64_t)tm * TL::BM;
        t.m_end = g.M;
        t.r0 = expert_start(g.offsets, t.e, g.P);
        t.K = expert_end(g.offsets, t.e, g.n, g.P) - t.r0;
    } else {
        RowTiles<TL::BM> row_tiles(g.offsets, g.n, g.P, (int)g.n + 1, lane);
        const int rows = row_tiles.total, tiles = rows * g.tiles_n;
        if (workgroup() >= tiles) return;
        tile_at(xcd_order(workgroup(), tiles), rows, g.tiles_n, imin(rows, 8), tm, tn);
        const RowTile r = row_tiles.find(tm);
        if (r.segment < 0) return;
        t.e = r.segment;
        t.m0 = r.row;
        t.m_end = r.end;
        t.r0 = 0;
        t.K = t.e < g.n ? g.K : 0;                       // rows of no expert: zeros
    }
    t.n0 = (int64_t)tn * TL::BN;

    f32x4_t acc[TL::NI][TL::MI];
#pragma unroll
    for (int j = 0; j < TL::NI; ++j)
#pragma unroll
        for (int i = 0; i < TL::MI; ++i) acc[j][i] = f32x4_t{};

    const int steps = (int)((t.K + BK - 1) / BK);
    u32x4_t a[SA::MINE], b[SB::MINE];
    auto load = [&](int kt) {
#pragma unroll
        for (int c = 0; c < SA::MINE; ++c) a[c] = load_a<TL, OP, GATED>(g, t, (int64_t)kt * BK, (int)threadIdx.x + c * NT);
#pragma unroll
        for (int c = 0; c < SB::MINE; ++c) b[c] = load_b<TL, OP, GATED>(g, t, (int64_t)kt * BK, (int)threadIdx.x + c * NT);
    };
    auto put = [&](uint16_t *buf) {
#pragma unroll
        for (int c = 0; c < SA::MINE; ++c) put_piece<T, SA>(buf, SA::piece((int)threadIdx.x, c), a[c]);
#pragma unroll
        for (int c = 0; c < SB::MINE; ++c) put_piece<T, SB>(buf + SA::ELEMS, SB::piece((int)threadIdx.x, c), b[c]);
    };
    if (steps > 0) {
        load(0);
        put(lds[0]);
        if (steps > 1) load(1);
    }
    __syncthreads();
    for (int kt = 0; kt < steps; ++kt) {
        const uint16_t *const buf = lds[kt & 1];
        bf16x8_t fa[TL::MI], fb[TL::NI];
#pragma unroll
        for (int i = 0; i < TL::MI; ++i) fa[i] = SA::frag(buf, wm * TL::TM + i * 16, lane);
#pragma unroll
        for (int j = 0; j < TL::NI; ++j) fb[j] = SB::frag(buf + SA::ELEMS, wn * TL::TN + j * 16, lane);
#pragma unroll
        for (int i = 0; i < TL::MI; ++i)
#pragma unroll
            for (int j = 0; j < TL::NI; ++j)
                acc[j][i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(fb[j], fa[i], acc[j][i], 0, 0, 0);
        if (kt + 1 < steps) {
            put(lds[(kt + 1) & 1]);                      // whose readers passed the last barrier
            if (kt + 2 < steps) load(kt + 2);
        }
        __syncthreads();
    }

    // acc[..][j][i][q]: row 16 i + (lane & 15), column 16 j + 4 (lane >> 4) + q of the wave's block
    const int mlane = lane & 15, quad = 4 * (lane >> 4);
    const bool there = OP == BACK_W || t.e < g.n;
#pragma unroll
    for (int i = 0; i < TL::MI; ++i) {
        int64_t m = t.m0 + wm * TL::TM + i * 16 + mlane;
        bool in = m < t.m_end;
        T *row = (T *)g.C;
        if constexpr (OP == BACK_W) {
            m = g.map.row(m);
            in = in && m >= 0;
            row += t.e * g.bank;
        }
        row += m * g.ldc;
#pragma unroll
        for (int j = 0; j < TL::NI; j += GATED ? 2 : 1) {
            float v[4], u[4];
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                v[q] = acc[j][i][q];
                if constexpr (GATED) u[q] = acc[j + 1][i][q];
            }
            if constexpr (GATED) {
                const int64_t F = g.N >> 1, f = ((t.n0 + wn * TL::TN) >> 1) + j * 8 + quad;
                if (g.bias != nullptr && there) {
                    const T *const bias = (const T *)g.bias + t.e * g.N;
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const int64_t at = lmin(f + q, F - 1);
                        v[q] += Elem<T>::load(bias + at);
                        u[q] += Elem<T>::load(bias + F + at);
                    }
                }
                if (in && f < F) {
                    if (g.Z != nullptr && there) {
                        float *const z = g.Z + m * g.ldz + f;
                        *reinterpret_cast<f32x4_t *>(z) = f32x4_t{v[0], v[1], v[2], v[3]};
                        *reinterpret_cast<f32x4_t *>(z + g.ldz / 2) = f32x4_t{u[0], u[1], u[2], u[3]};
                    }
#pragma unroll
                    for (int q = 0; q < 4; ++q) v[q] = there ? gate_act<GATE>(v[q]) * u[q] : 0.0f;
                    store4<T>(row + f, v, F - f);
                }
            } else {
                const int64_t n = t.n0 + wn * TL::TN + j * 16 + quad;
                if (OP == FORWARD && g.bias != nullptr && there) {
                    const T *const bias = (const T *)g.bias + t.e * g.N;
#pragma unroll
                    for (int q = 0; q < 4; ++q) v[q] += Elem<T>::load(bias + lmin(n + q, g.N - 1));
                }
                if (in && n < g.N) store4<T>(row + n, v, g.N - n);
            }
        }
    }
}

using Tile128 = Tile<2, 4, 64, 32>;
using Tile64 = Tile<2, 2, 32, 32>;

template <class TL, int OP, int GATE>
hipError_t launch_tile(ExpertProduct g, hipStream_t stream)
{
    g.tiles_n = (int)((g.N + TL::BN - 1) / TL::BN);
    int64_t blocks;
    if constexpr (OP == BACK_W) {
        g.tiles_m = (int)((g.M + TL::BM - 1) / TL::BM);
        blocks = g.n * g.tiles_m * g.tiles_n;
    } else {
        const int64_t segments = g.n + 1;
        blocks = (g.P / TL::BM + (segments < g.P ? segments : g.P)) * g.tiles_n;
    }
    if (!grid_ok(blocks)) return hipErrorInvalidValue;
    hipLaunchKernelGGL((expert_kernel<TL, OP, GATE>), grid_of(blocks), dim3(TL::NT), 0, stream, g);
    return hipGetLastError();
}

// 128 x 128 tiles where they fill the CUs, else 64 x 64.
template <int OP, int GATE>
hipError_t launch_op(const ExpertProduct &g, hipStream_t stream)
{
    const int64_t tm = OP == BACK_W ? g.n * ((g.M + 127) / 128) : g.P / 128, tn = (g.N + 127) / 128;
    if (tm * tn >= g.num_cus) return launch_tile<Tile128, OP, GATE>(g, stream);
    return launch_tile<Tile64, OP, GATE>(g, stream);
}

// dW_e = the sum of its pieces' products, in order; zeros without one.
constexpr int SUM_ROWS = 8;
template <class D>
__global__ __launch_bounds__(256) void sum_chunks_kernel(ExpertProduct g)
{
    const int lane = threadIdx.x & 63, e = (int)blockIdx.y, across = (int)((g.N + 255) / 256);
    int before = 0;
    for (int i = lane; i < e; i += 64) before += (int)((expert_end(g.offsets, i, g.n, g.P) - expert_start(g.offsets, i, g.P) + g.chunk - 1) / g.chunk);
    before = __builtin_amdgcn_readfirstlane(wave_sum(before));
    // offsets that do not ascend may count more pieces than there are
    const int most = (int)weight_chunks(g), first = imin(before, most);
    const int64_t rows = expert_end(g.offsets, e, g.n, g.P) - expert_start(g.offsets, e, g.P);
    const int count = imin((int)((rows + g.chunk - 1) / g.chunk), most - first);
    const int64_t n = (int64_t)((int)blockIdx.x % across) * 256 + threadIdx.x, m0 = (int64_t)((int)blockIdx.x / across) * SUM_ROWS;
    if (n >= g.N) return;
    float v[SUM_ROWS];
#pragma unroll
    for (int i = 0; i < SUM_ROWS; ++i) v[i] = 0.0f;
    for (int c = 0; c < count; ++c) {
        const float *const p = g.partials + (first + c) * g.M * g.N + n;
#pragma unroll
        for (int i = 0; i < SUM_ROWS; ++i) v[i] += p[lmin(m0 + i, g.M - 1) * g.N];
    }
#pragma unroll
    for (int i = 0; i < SUM_ROWS; ++i) {
        const int64_t m = m0 + i < g.M ? g.map.row(m0 + i) : -1;
        if (m >= 0) ((D *)g.C)[e * g.bank + m * g.ldc + n] = Elem<D>::store(v[i]);
    }
}

hipError_t launch(int op, const ExpertProduct &g, hipStream_t stream)
{
    if (op == BACK_X) return launch_op<BACK_X, -1>(g, stream);
    if (op == BACK_W) return launch_op<BACK_W, -1>(g, stream);
    switch (g.gate) {
    case kSilu: return launch_op<FORWARD, kSilu>(g, stream);
    case kGelu: return launch_op<FORWARD, kGelu>(g, stream);
    case kGeluTanh: return launch_op<FORWARD, kGeluTanh>(g, stream);
    case kSigmoid: return launch_op<FORWARD, kSigmoid>(g, stream);
    case kRelu: return launch_op<FORWARD, kRelu>(g, stream);
    default: return launch_op<FORWARD, -1>(g, stream);
    }
}

}  // namespace

hipError_t launch_expert(int op, int dtype, const ExpertProduct &g, hipStream_t stream)
{
    if (op == kBackW ? g.n == 0 || g.M == 0 : g.P == 0) return hipSuccess;
    if (g.N == 0) return hipSuccess;
    if (op == kForward && expert_few(dtype, g)) return launch_expert_few(dtype, g, stream);
    const bool lies = dtype == kF32 || expert_lies(op, g);
    ExpertProduct q = g;
    if (!lies || q.chunk == 0) q.partials = nullptr;
    const hipError_t e = dtype == kF32 ? launch_expert_f32(op, q, stream)
                         : lies ? launch_expert_bf16(op, q, stream) : launch(op, q, stream);
    if (e != hipSuccess || q.partials == nullptr) return e;
    const dim3 grid((unsigned)(((g.N + 255) / 256) * ((g.M + SUM_ROWS - 1) / SUM_ROWS)), (unsigned)g.n);
    if (dtype == kF32) hipLaunchKernelGGL(sum_chunks_kernel<float>, grid, dim3(256), 0, stream, q);
    else hipLaunchKernelGGL(sum_chunks_kernel<uint16_t>, grid, dim3(256), 0, stream, q);
    return hipGetLastError();
}

}  // namespace sgemm_emu_dev
