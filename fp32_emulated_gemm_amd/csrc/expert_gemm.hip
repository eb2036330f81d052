// expert_gemm.hip -- the experts' products on sorted rows: forward, gradients of the
// rows and of the weights, FP32 and bfloat16.
//
// One workgroup per output tile; a row tile lies inside one expert, found from the
// offsets on the device, so nothing waits for the host.  The grid is the most
// tiles that any offsets can give; workgroups past the last tile end at once.
//
// Operands come in two layouts: rows with k contiguous (X, W in the forward), or
// rows of k with the other index contiguous (W in dX, dZ and X in dW).  The second
// kind is read out of LDS by ds_read_b64_tr_b16, which hands a lane four k of one
// column, so nothing is transposed in memory: no copies of W, and an expert's
// rows may start anywhere.
//
// FP32: each operand is split into three BF16 parts as it is staged, x = x0 + 2^-8
// x1 + 2^-16 x2, every stage rounded to nearest even.  Then |x1| <= |x| / 2 and |x2|
// <= |x| / 4, so the three products x1 w2, x2 w1 and x2 w2 together stay below 2^-25
// |x w|, half of an FP32 rounding, and are left out: six products in three bands of
// one weight each, summed in FP32 and added smallest first.
#include "expert_device.hpp"

namespace sgemm_emu_dev {

namespace {

constexpr int BK = 32;                       // K step: one MFMA's
typedef short s16x4_t __attribute__((ext_vector_type(4)));

enum { FORWARD = kForward, BACK_X = kBackX, BACK_W = kBackW };

// PLANES: BF16 parts of an element; BANDS: accumulators.
template <class T>
struct Parts {
    static constexpr int PLANES = sizeof(T) == 4 ? 3 : 1;
};

template <int WAVES_M_, int WAVES_N_, int TM_, int TN_>
struct Tile {
    static constexpr int WAVES_M = WAVES_M_, WAVES_N = WAVES_N_, NT = 64 * WAVES_M * WAVES_N;
    static constexpr int TM = TM_, TN = TN_, BM = WAVES_M * TM, BN = WAVES_N * TN;
    static constexpr int MI = TM / 16, NI = TN / 16;
};

// An operand's tile in LDS: R rows (outputs' rows or columns) by BK, one plane after
// another.  !KM: R rows of BK elements.  KM: BK rows of R elements.  16-byte slots
// are permuted so that the fragment reads spread over the banks.
template <int R, bool KM, int PLANES, int NT>
struct Stage {
    static constexpr int PLANE = R * BK, ELEMS = PLANES * PLANE;
    static constexpr int CHUNKS = R * BK / 8, MINE = CHUNKS / NT;      // of 8 elements
    static constexpr int WIDE = KM ? R / 8 : BK / 8;                   // chunks of a row
    static_assert(CHUNKS % NT == 0, "chunks split evenly");

    static __device__ __forceinline__ int slot(int row, int c)
    {
        if constexpr (KM) return c ^ ((((row & 3) | ((row >> 1) & 4)) << 1) & (WIDE - 1));
        else return c ^ ((row >> 2) & 3);
    }
    // Offset of chunk c of LDS row `row` in a plane.
    static __device__ __forceinline__ int at(int row, int c) { return row * WIDE * 8 + slot(row, c) * 8; }

    // Fragment: k 8 (lane >> 4) .. + 7 of index base + (lane & 15).
    static __device__ __forceinline__ bf16x8_t frag(const uint16_t *plane, int base, int lane)
    {
        if constexpr (KM) {
            typedef __attribute__((address_space(3))) s16x4_t lds_t;
            const int i = lane & 15, col = base + 4 * (i & 3);
            s16x4_t v[2];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int k = 8 * (lane >> 4) + 4 * h + (i >> 2);
                v[h] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_t *)(plane + at(k, col >> 3) + (col & 7)));
            }
            return __builtin_bit_cast(bf16x8_t, __builtin_shufflevector(v[0], v[1], 0, 1, 2, 3, 4, 5, 6, 7));
        } else {
            return ld_frag(plane + at(base + (lane & 15), lane >> 4));
        }
    }
};

template <class T, class S>
__device__ __forceinline__ void put_eight(uint16_t *buf, int at, const Eight<T> &e)
{
    if constexpr (sizeof(T) == 4) {
        u32x4_t p[3];
        split8_nearest(e, p);
#pragma unroll
        for (int q = 0; q < 3; ++q) *reinterpret_cast<u32x4_t *>(buf + q * S::PLANE + at) = p[q];
    } else {
        *reinterpret_cast<u32x4_t *>(buf + at) = e.v[0];
    }
}

// What a tile multiplies: addresses of its operands' chunks.
struct Place {
    int64_t e, m0, m_end, n0, K;     // expert; rows and their end; first column; inner extent
    int64_t r0;                      // dW: the expert's first row
};

// Row of the bank behind tile column c of a gated forward product: alternating
// blocks of 16 gate and 16 up rows, so that both of an output meet in one lane.
__device__ __forceinline__ int64_t gated_row(int64_t F, int64_t n0, int c)
{
    const int64_t f = lmin((n0 >> 1) + ((c >> 5) << 4) + (c & 15), F - 1);
    return (c & 16) ? F + f : f;
}

template <class T, class TL, int OP, bool GATED>
__device__ __forceinline__ void load_a(const ExpertProduct &g, const Place &t, int64_t k0, int chunk, Eight<T> &out)
{
    const T *const A = (const T *)g.A;
    if constexpr (OP == BACK_W) {
        constexpr int WIDE = TL::BM / 8;
        const int64_t k = k0 + chunk / WIDE, c = t.m0 + chunk % WIDE * 8;
        out.load(A + (t.r0 + k) * g.lda + c, k < t.K ? g.M - c : 0);
    } else {
        const int64_t m = lmin(t.m0 + chunk / 4, t.m_end - 1), k = k0 + chunk % 4 * 8;
        out.load(A + m * g.lda + k, t.K - k);
    }
}

template <class T, class TL, int OP, bool GATED>
__device__ __forceinline__ void load_b(const ExpertProduct &g, const Place &t, int64_t k0, int chunk, Eight<T> &out)
{
    const T *const B = (const T *)g.B + (OP == BACK_W ? 0 : t.e * g.bank);
    if constexpr (OP == FORWARD) {
        const int c = chunk / 4;
        const int64_t n = GATED ? gated_row(g.N >> 1, t.n0, c) : lmin(t.n0 + c, g.N - 1), k = k0 + chunk % 4 * 8;
        out.load(B + n * g.ldb + k, t.K - k);
    } else {
        constexpr int WIDE = TL::BN / 8;
        const int64_t k = k0 + chunk / WIDE, c = t.n0 + chunk % WIDE * 8;
        const int64_t row = OP == BACK_W ? t.r0 + k : g.map.row(k);
        out.load(B + row * g.ldb + c, k < t.K && row >= 0 ? g.N - c : 0);
    }
}

// Four results, columns n.. of a row, `left` of them there.
template <class T>
__device__ __forceinline__ void store4(T *p, const float (&f)[4], int64_t left)
{
    if (left >= 4) {
        if constexpr (sizeof(T) == 4) {
            *reinterpret_cast<u32x4_any *>(p) = u32x4_t{f2u(f[0]), f2u(f[1]), f2u(f[2]), f2u(f[3])};
        } else {
            typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
            *reinterpret_cast<u32x2_any *>(p) = u32x2{pack2(f[0], f[1]), pack2(f[2], f[3])};
        }
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (e < left) p[e] = Elem<T>::store(f[e]);
    }
}

template <class T, class TL, int OP, int GATE>
__global__ __launch_bounds__(TL::NT) void expert_kernel(ExpertProduct g)
{
    constexpr int PL = Parts<T>::PLANES, NT = TL::NT;
    constexpr bool GATED = GATE >= 0;
    typedef Stage<TL::BM, OP == BACK_W, PL, NT> SA;
    typedef Stage<TL::BN, OP != FORWARD, PL, NT> SB;
    __shared__ __attribute__((aligned(16))) uint16_t lds[2][SA::ELEMS + SB::ELEMS];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wm = wave / TL::WAVES_N, wn = wave % TL::WAVES_N;

    Place t;
    int tm, tn;
    if constexpr (OP == BACK_W) {
        const int per = g.tiles_m * g.tiles_n;
        const int v = (int)blockIdx.x % per;
        t.e = (int)blockIdx.x / per;
        tm = v / g.tiles_n;
        tn = v % g.tiles_n;
        t.m0 = (int64_t)tm * TL::BM;
        t.m_end = g.M;
        t.r0 = expert_start(g.offsets, t.e, g.P);
        t.K = expert_end(g.offsets, t.e, g.n, g.P) - t.r0;
    } else {
        const int segments = (int)g.n + 1;
        const int rows = all_tiles<TL::BM>(g.offsets, g.n, g.P, segments, lane), T_ = rows * g.tiles_n;
        if ((int)blockIdx.x >= T_) return;
        tile_of_index((int)blockIdx.x, T_, rows, g.tiles_n, imin(rows, 8), tm, tn);
        const RowTile r = find_tile<TL::BM>(g.offsets, g.n, g.P, segments, tm, lane);
        if (r.segment < 0) return;
        t.e = r.segment;
        t.m0 = r.row;
        t.m_end = r.end;
        t.r0 = 0;
        t.K = t.e < g.n ? g.K : 0;                       // rows of no expert: zeros
    }
    t.n0 = (int64_t)tn * TL::BN;

    constexpr int BANDS = PL;
    f32x4_t acc[BANDS][TL::NI][TL::MI];
#pragma unroll
    for (int b = 0; b < BANDS; ++b)
#pragma unroll
        for (int j = 0; j < TL::NI; ++j)
#pragma unroll
            for (int i = 0; i < TL::MI; ++i) acc[b][j][i] = f32x4_t{};

    const int steps = (int)((t.K + BK - 1) / BK);
    Eight<T> a[SA::MINE], b[SB::MINE];
    auto load = [&](int kt) {
#pragma unroll
        for (int c = 0; c < SA::MINE; ++c) load_a<T, TL, OP, GATED>(g, t, (int64_t)kt * BK, (int)threadIdx.x + c * NT, a[c]);
#pragma unroll
        for (int c = 0; c < SB::MINE; ++c) load_b<T, TL, OP, GATED>(g, t, (int64_t)kt * BK, (int)threadIdx.x + c * NT, b[c]);
    };
    auto put = [&](uint16_t *buf) {
#pragma unroll
        for (int c = 0; c < SA::MINE; ++c) {
            const int chunk = (int)threadIdx.x + c * NT;
            put_eight<T, SA>(buf, SA::at(chunk / SA::WIDE, chunk % SA::WIDE), a[c]);
        }
#pragma unroll
        for (int c = 0; c < SB::MINE; ++c) {
            const int chunk = (int)threadIdx.x + c * NT;
            put_eight<T, SB>(buf + SA::ELEMS, SB::at(chunk / SB::WIDE, chunk % SB::WIDE), b[c]);
        }
    };
    if (steps > 0) {
        load(0);
        put(lds[0]);
        if (steps > 1) load(1);
    }
    __syncthreads();
    for (int kt = 0; kt < steps; ++kt) {
        const uint16_t *const buf = lds[kt & 1];
        bf16x8_t fa[PL][TL::MI], fb[PL][TL::NI];
#pragma unroll
        for (int q = 0; q < PL; ++q) {
#pragma unroll
            for (int i = 0; i < TL::MI; ++i) fa[q][i] = SA::frag(buf + q * SA::PLANE, wm * TL::TM + i * 16, lane);
#pragma unroll
            for (int j = 0; j < TL::NI; ++j)
                fb[q][j] = SB::frag(buf + SA::ELEMS + q * SB::PLANE, wn * TL::TN + j * 16, lane);
        }
#pragma unroll
        for (int band = BANDS - 1; band >= 0; --band)
#pragma unroll
            for (int p = 0; p <= band; ++p)
#pragma unroll
                for (int i = 0; i < TL::MI; ++i)
#pragma unroll
                    for (int j = 0; j < TL::NI; ++j)
                        acc[band][j][i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(fb[band - p][j], fa[p][i],
                                                                                  acc[band][j][i], 0, 0, 0);
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
                v[q] = acc[0][j][i][q];
                if constexpr (GATED) u[q] = acc[0][j + 1][i][q];
                if constexpr (BANDS == 3) {
                    v[q] += __builtin_fmaf(acc[2][j][i][q], 0x1p-16f, acc[1][j][i][q] * 0x1p-8f);
                    if constexpr (GATED) u[q] += __builtin_fmaf(acc[2][j + 1][i][q], 0x1p-16f, acc[1][j + 1][i][q] * 0x1p-8f);
                }
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

template <class T, class TL, int OP, int GATE>
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
    if (blocks * TL::NT >= (int64_t)1 << 32) return hipErrorInvalidValue;   // more work-items than a launch can have
    hipLaunchKernelGGL((expert_kernel<T, TL, OP, GATE>), dim3((unsigned)blocks), dim3(TL::NT), 0, stream, g);
    return hipGetLastError();
}

// 128 x 128 tiles where they fill the CUs, else 64 x 64.
template <class T, int OP, int GATE>
hipError_t launch_op(const ExpertProduct &g, hipStream_t stream)
{
    const int64_t tm = OP == BACK_W ? g.n * ((g.M + 127) / 128) : g.P / 128, tn = (g.N + 127) / 128;
    if (tm * tn >= g.num_cus) return launch_tile<T, Tile128, OP, GATE>(g, stream);
    return launch_tile<T, Tile64, OP, GATE>(g, stream);
}

template <class T>
hipError_t launch_forward(const ExpertProduct &g, hipStream_t stream)
{
    switch (g.gate) {
    case kSilu: return launch_op<T, FORWARD, kSilu>(g, stream);
    case kGelu: return launch_op<T, FORWARD, kGelu>(g, stream);
    case kGeluTanh: return launch_op<T, FORWARD, kGeluTanh>(g, stream);
    case kSigmoid: return launch_op<T, FORWARD, kSigmoid>(g, stream);
    case kRelu: return launch_op<T, FORWARD, kRelu>(g, stream);
    default: return launch_op<T, FORWARD, -1>(g, stream);
    }
}

}  // namespace

hipError_t launch_expert_forward(int dtype, const ExpertProduct &g, hipStream_t stream)
{
    if (g.P == 0 || g.N == 0) return hipSuccess;
    if (dtype == kBF16 && expert_lies(kForward, g)) return launch_expert_bf16(kForward, g, stream);
    return dtype == kF32 ? launch_forward<float>(g, stream) : launch_forward<uint16_t>(g, stream);
}

hipError_t launch_expert_dx(int dtype, const ExpertProduct &g, hipStream_t stream)
{
    if (g.P == 0 || g.N == 0) return hipSuccess;
    if (dtype == kBF16 && expert_lies(kBackX, g)) return launch_expert_bf16(kBackX, g, stream);
    return dtype == kF32 ? launch_op<float, BACK_X, -1>(g, stream) : launch_op<uint16_t, BACK_X, -1>(g, stream);
}

hipError_t launch_expert_dw(int dtype, const ExpertProduct &g, hipStream_t stream)
{
    if (g.n == 0 || g.M == 0 || g.N == 0) return hipSuccess;
    if (dtype == kBF16 && expert_lies(kBackW, g)) return launch_expert_bf16(kBackW, g, stream);
    return dtype == kF32 ? launch_op<float, BACK_W, -1>(g, stream) : launch_op<uint16_t, BACK_W, -1>(g, stream);
}

}  // namespace sgemm_emu_dev
