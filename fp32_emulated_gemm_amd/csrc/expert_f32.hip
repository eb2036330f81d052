// expert_f32.hip -- the experts' FP32 products.
//
// Each operand is split into three BF16 parts as it is staged, x = x0 + 2^-8 x1 +
// 2^-16 x2, every stage rounded to nearest even.  With 2^e <= |x| < 2^(e+1) the first
// rounding leaves at most 2^(e-8), so |x1| <= 2^e <= |x|, and the second 2^(e-9) of
// that, so |x2| <= 2^(e-1) <= |x| / 2.  The products x1 w2 and x2 w1, of weight 2^-24,
// are each at most |x w| / 2 (x2 w2 is 2^-10 of them): together at most 2^-24 |x w|,
// an FP32 product's own rounding, and a tenth of it on average.  They are left out:
// six products on the BF16 matrix cores in three bands of one weight each, summed in
// FP32 and added smallest first.
//
// One workgroup per output tile, in K steps of 32.  A step's operands are loaded two
// steps ahead, and split and written to the other LDS buffer among the MFMAs of the
// step before: vector instructions, the split's for the most part, take 1.25 times the
// MFMAs' cycles (dX below), so neither may wait for the other.  Loads go through descriptors that end with the
// last element, so nothing is read behind it, whatever K and the alignment; where K
// ends inside a step, what a row's pieces hold behind it is cleared.
//
// Operands whose k are rows (W in dX, dZ and X in dW) keep that layout in LDS and are
// read by ds_read_b64_tr_b16, four k of a column at a time: nothing is transposed in
// memory, and an expert's rows may start anywhere.
//
// What bounds it is the split beside the MFMAs: 2048^3 in one expert runs at 146 TFLOP/s
// (the platform's FP32 product: 124; 154 at 8192^3).  12288 x 256 -> 1024 over eight
// experts, gated, with Z: 85 us; dX 66, dW 67 and 11 for its pieces' sums.  There vector
// instructions and MFMAs take 29 and 23 % of the SIMDs' cycles in dX, 35 and 18 % in the
// forward pass (its gate and Z besides), and waves wait in a quarter to a third of theirs.
#include <type_traits>

#include "expert_stage.hpp"

namespace sgemm_emu_dev {

namespace {

constexpr int PL = 3;                        // BF16 parts, and bands

// One operand's pieces of 16 bytes in this thread: where they lie.
template <class S, bool KM>
struct Pieces {
    const float *p[KM ? 1 : S::MINE];        // !KM: first row of the wave's eight, at k = 0
    uint32_t bytes[KM ? 1 : S::MINE];        // to the last element of the last of them
    uint32_t off[KM ? 1 : S::MINE];          // KM: the next piece lies a fixed number of rows on
};

constexpr int64_t MOST_BYTES = 0xFFFFFFF0ll;

// make_rsrc for a size that fits.
__device__ __forceinline__ rsrc_t make_rsrc32(const void *base, uint32_t bytes)
{
    const uint64_t p = (uint64_t)(uintptr_t)base;
    void *const ub = (void *)(uintptr_t)(((uint64_t)(uint32_t)__builtin_amdgcn_readfirstlane((uint32_t)(p >> 32)) << 32) |
                                         (uint32_t)__builtin_amdgcn_readfirstlane((uint32_t)p));
    return __builtin_amdgcn_make_buffer_rsrc(ub, (short)0, (int)__builtin_amdgcn_readfirstlane(bytes), RSRC_WORD3);
}

template <class TL, int OP, int GATE>
__global__ __launch_bounds__(TL::NT, TL::PER_CU) void expert_f32_kernel(ExpertProduct g)
{
    constexpr int NT = TL::NT;
    constexpr bool GATED = GATE >= 0, A_KM = OP == kBackW, B_KM = OP != kForward;
    typedef Stage<float, TL::BM, A_KM, PL, NT> SA;
    typedef Stage<float, TL::BN, B_KM, PL, NT> SB;
    __shared__ __attribute__((aligned(16))) uint16_t lds[2][SA::ELEMS + SB::ELEMS];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wm = wave / TL::WAVES_N, wn = wave % TL::WAVES_N;

    int64_t e, m0, m_end, K, r0 = 0;
    int tm, tn;
    int chunk = 0;
    if constexpr (OP == kBackW) {
        const int per = g.tiles_m * g.tiles_n;
        chunk = workgroup() / per;
        if (chunk >= weight_chunks(g)) return;
        tile_at(xcd_order(workgroup() - chunk * per, per), g.tiles_m, g.tiles_n, imin(g.tiles_m, 8), tm, tn);
        m0 = (int64_t)tm * TL::BM;
        m_end = g.M;
        const RowTile r = weight_rows(g, chunk, lane);
        if (r.segment < 0) return;
        e = r.segment;
        r0 = r.row;
        K = r.end - r0;
    } else {
        RowTiles<TL::BM> row_tiles(g.offsets, g.n, g.P, (int)g.n + 1, lane);
        const int rows = row_tiles.total, tiles = rows * g.tiles_n;
        if (workgroup() >= tiles) return;
        tile_at(xcd_order(workgroup(), tiles), rows, g.tiles_n, imin(rows, 8), tm, tn);
        const RowTile r = row_tiles.find(tm);
        if (r.segment < 0) return;
        e = r.segment;
        m0 = r.row;
        m_end = r.end;
        K = e < g.n ? g.K : 0;                             // rows of no expert: zeros
    }
    const int64_t n0 = (int64_t)tn * TL::BN;
    const bool there = OP == kBackW || e < g.n;
    const float *const A = (const float *)g.A;
    const float *const B = (const float *)g.B + (OP == kBackW || !there ? 0 : e * g.bank);
    const int steps = (int)((K + BK - 1) / BK);

    Pieces<SA, A_KM> pa;
    Pieces<SB, B_KM> pb;
    // Eight threads take a row's 32 k, a wave eight rows.
    auto rows_of = [&](auto &q, const float *from, int64_t ld, int c, auto row) {
        const int piece = (int)threadIdx.x + c * NT, r = piece / 8, first8 = (wave * 64 + c * NT) / 8;
        int64_t first = row(first8), last = row(first8 + 7);
        q.p[c] = from + first * ld;
        q.bytes[c] = (uint32_t)lmin(((last - first) * ld + K) * 4, MOST_BYTES);
        q.off[c] = (uint32_t)(((row(r) - first) * ld + piece % 8 * 4) * 4);
    };
    if constexpr (A_KM) {
        pa.off[0] = (uint32_t)(((int)threadIdx.x / SA::ROW * g.lda + (int)threadIdx.x % SA::ROW * 4) * 4);
    } else {
#pragma unroll
        for (int c = 0; c < SA::MINE; ++c) rows_of(pa, A, g.lda, c, [&](int r) { return lmin(m0 + r, m_end - 1); });
    }
    if constexpr (B_KM) {
        pb.off[0] = (uint32_t)(((int)threadIdx.x / SB::ROW * g.ldb + (int)threadIdx.x % SB::ROW * 4) * 4);
    } else {
#pragma unroll
        for (int c = 0; c < SB::MINE; ++c)
            rows_of(pb, B, g.ldb, c, [&](int r) { return GATED ? gated_row(g.N >> 1, n0, r) : lmin(n0 + r, g.N - 1); });
    }
    // Bytes of `rows` rows of ld elements, from column c0 of cols on, to the last
    // element.  The rows span less than 2^32 bytes, and nothing here branches: a branch
    // would part the step's split from its MFMAs.
    auto extent = [](int rows, int64_t ld, int64_t cols, int64_t c0) {
        const uint32_t last = (uint32_t)(cols - c0) * 4u, before = (uint32_t)(rows - 1) * (uint32_t)(ld * 4);
        return rows > 0 ? last + before : 0u;
    };
    auto rows_left = [](int64_t left) { return (int)(left < BK ? left : BK); };

    struct Set {
        u32x4_t a[SA::MINE], b[SB::MINE];
    };
    auto load = [&](Set &s, int kt) {
        const int64_t k0 = (int64_t)kt * BK;
        if constexpr (A_KM) {
            const rsrc_t r = make_rsrc32(A + (r0 + k0) * g.lda + m0, extent(rows_left(K - k0), g.lda, g.M, m0));
#pragma unroll
            for (int c = 0; c < SA::MINE; ++c) s.a[c] = bload_u32x4(r, pa.off[0] + (uint32_t)(c * (NT / SA::ROW) * g.lda * 4), 0);
        } else {
#pragma unroll
            for (int c = 0; c < SA::MINE; ++c) s.a[c] = bload_u32x4(make_rsrc32(pa.p[c], pa.bytes[c]), pa.off[c] + (uint32_t)(k0 * 4), 0);
        }
        if constexpr (B_KM) {
            // dX: a step lies in one half of dZ's columns (h is a multiple of BK, or K itself)
            const bool up = OP == kBackX && k0 >= g.map.h;
            const int64_t in = up ? k0 - g.map.h : k0, row = OP == kBackW ? r0 + k0 : up ? g.map.F + in : in;
            // a step past the last (loaded ahead, never used) has no rows: without a gate the
            // rows behind W's last would seem to be an up half
            const int64_t left = OP == kBackW ? K - k0 : lmin(g.map.F - in, K - k0);
            const rsrc_t r = make_rsrc32(B + row * g.ldb + n0, extent(rows_left(left), g.ldb, g.N, n0));
#pragma unroll
            for (int c = 0; c < SB::MINE; ++c) s.b[c] = bload_u32x4(r, pb.off[0] + (uint32_t)(c * (NT / SB::ROW) * g.ldb * 4), 0);
        } else {
#pragma unroll
            for (int c = 0; c < SB::MINE; ++c) s.b[c] = bload_u32x4(make_rsrc32(pb.p[c], pb.bytes[c]), pb.off[c] + (uint32_t)(k0 * 4), 0);
        }
    };
    // What a row's pieces hold behind K, in the step where it ends.
    auto clear_tail = [&](Set &s, int kt) {
        const int left = (int)(K - (int64_t)kt * BK);
        if (left >= BK) return;
        const int c0 = (int)threadIdx.x % 8 * 4;
        if constexpr (!A_KM) {
#pragma unroll
            for (int c = 0; c < SA::MINE; ++c)
#pragma unroll
                for (int q = 0; q < 4; ++q) s.a[c][q] = c0 + q < left ? s.a[c][q] : 0u;
        }
        if constexpr (!B_KM) {
#pragma unroll
            for (int c = 0; c < SB::MINE; ++c)
#pragma unroll
                for (int q = 0; q < 4; ++q) s.b[c][q] = c0 + q < left ? s.b[c][q] : 0u;
        }
    };
    auto put = [&](uint16_t *buf, const Set &s) {
#pragma unroll
        for (int c = 0; c < SA::MINE; ++c) put_piece<float, SA>(buf, SA::piece((int)threadIdx.x, c), s.a[c]);
#pragma unroll
        for (int c = 0; c < SB::MINE; ++c) put_piece<float, SB>(buf + SA::ELEMS, SB::piece((int)threadIdx.x, c), s.b[c]);
    };

    f32x4_t acc[PL][TL::NI][TL::MI];
#pragma unroll
    for (int b = 0; b < PL; ++b)
#pragma unroll
        for (int j = 0; j < TL::NI; ++j)
#pragma unroll
            for (int i = 0; i < TL::MI; ++i) acc[b][j][i] = f32x4_t{};

    // Step kt: its operands lie in `buf`; `next` takes those of kt + 1 from `s`, which
    // then loads those of kt + 3.  MORE: 0 for the last step, 2 where kt + 1 is the
    // last, which may end inside K.  The planes' fragments are read in turn, two planes
    // held at a time; a band's products need no order among them.
    auto step = [&](int kt, const uint16_t *buf, uint16_t *next, Set &s, auto more) {
        constexpr int MORE = decltype(more)::value;
        bf16x8_t fa[2][TL::MI], fb[2][TL::NI];
        auto read = [&](int into, int q) {
#pragma unroll
            for (int i = 0; i < TL::MI; ++i) fa[into][i] = SA::frag(buf + q * SA::PLANE, wm * TL::TM + i * 16, lane);
#pragma unroll
            for (int j = 0; j < TL::NI; ++j)
                fb[into][j] = SB::frag(buf + SA::ELEMS + q * SB::PLANE, wn * TL::TN + j * 16, lane);
        };
        auto multiply = [&](int band, int x, int y) {
#pragma unroll
            for (int i = 0; i < TL::MI; ++i)
#pragma unroll
                for (int j = 0; j < TL::NI; ++j)
                    acc[band][j][i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(fb[y][j], fa[x][i], acc[band][j][i], 0, 0, 0);
        };
        read(0, 0);
        read(1, 1);
        multiply(0, 0, 0);
        multiply(1, 0, 1);
        multiply(1, 1, 0);
        multiply(2, 1, 1);
        read(1, 2);
        if constexpr (MORE == 2) clear_tail(s, kt + 1);
        if constexpr (MORE != 0) put(next, s);   // whose readers passed the last barrier
        if constexpr (MORE == 1) load(s, kt + 3);   // past the last step: nothing inside the descriptors that is used
        multiply(2, 0, 1);
        multiply(2, 1, 0);
        if constexpr (MORE == 1) {
            constexpr int MFMAS = 6 * TL::MI * TL::NI, PUTS = SA::MINE + SB::MINE, EACH = MFMAS / PUTS;
#pragma unroll
            for (int q = 0; q < PUTS; ++q) {
#pragma unroll
                for (int i = 0; i < EACH; ++i) {
                    __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);                       // an MFMA
                    __builtin_amdgcn_sched_group_barrier(0x002, (56 + EACH - 1) / EACH, 0);  // vector instructions
                }
                __builtin_amdgcn_sched_group_barrier(0x200, 3, 0);                           // a piece's three parts
            }
        }
        lds_barrier();
    };
    if (steps > 0) {
        constexpr auto MAIN = std::integral_constant<int, 1>();
        Set s0, s1;
        load(s0, 0);
        load(s1, 1);
        if (steps == 1) clear_tail(s0, 0);
        put(lds[0], s0);
        load(s0, 2);
        lds_barrier();
        int kt = 0;
        for (; kt + 3 < steps; kt += 2) {
            step(kt, lds[0], lds[1], s1, MAIN);
            step(kt + 1, lds[1], lds[0], s0, MAIN);
        }
        int at = 0;
        if (kt + 2 < steps) {
            step(kt, lds[0], lds[1], s1, MAIN);
            s1 = s0;
            at = 1;
            ++kt;
        }
        if (kt + 1 < steps) {
            step(kt, lds[at], lds[at ^ 1], s1, std::integral_constant<int, 2>());
            at ^= 1;
            ++kt;
        }
        step(kt, lds[at], nullptr, s1, std::integral_constant<int, 0>());
    }

    // acc[..][j][i][q]: row 16 i + (lane & 15), column 16 j + 4 (lane >> 4) + q of the wave's block
    const int mlane = lane & 15, quad = 4 * (lane >> 4);
    auto total = [&](int j, int i, int q) {
        return acc[0][j][i][q] + __builtin_fmaf(acc[2][j][i][q], 0x1p-16f, acc[1][j][i][q] * 0x1p-8f);
    };
    const float *const bias = OP == kForward && there && g.bias != nullptr ? (const float *)g.bias + e * g.N : nullptr;
    const int64_t F = GATED ? g.N >> 1 : g.N;
#pragma unroll
    for (int j = 0; j < TL::NI; j += GATED ? 2 : 1) {
        const int64_t n = GATED ? ((n0 + wn * TL::TN) >> 1) + j * 8 + quad : n0 + wn * TL::TN + j * 16 + quad;
        float b[4] = {0, 0, 0, 0}, bu[4] = {0, 0, 0, 0};
        if (bias != nullptr) {
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const int64_t at = lmin(n + q, F - 1);
                b[q] = bias[at];
                if constexpr (GATED) bu[q] = bias[F + at];
            }
        }
#pragma unroll
        for (int i = 0; i < TL::MI; ++i) {
            int64_t m = m0 + wm * TL::TM + i * 16 + mlane;
            bool in = m < m_end && n < F;
            float *row = (float *)g.C;
            int64_t ld = g.ldc;
            if constexpr (OP == kBackW) {
                if (g.partials != nullptr) {
                    row = g.partials + chunk * g.M * g.N;
                    ld = g.N;
                } else {
                    m = g.map.row(m);
                    in = in && m >= 0;
                    row += e * g.bank;
                }
            }
            if (!in) continue;
            row += m * ld + n;
            float v[4];
#pragma unroll
            for (int q = 0; q < 4; ++q) v[q] = total(j, i, q) + b[q];
            if constexpr (GATED) {
                float u[4];
#pragma unroll
                for (int q = 0; q < 4; ++q) u[q] = total(j + 1, i, q) + bu[q];
                if (g.Z != nullptr && there) {
                    float *const z = g.Z + m * g.ldz + n;
                    *reinterpret_cast<f32x4_t *>(z) = f32x4_t{v[0], v[1], v[2], v[3]};
                    *reinterpret_cast<f32x4_t *>(z + g.ldz / 2) = f32x4_t{u[0], u[1], u[2], u[3]};
                }
#pragma unroll
                for (int q = 0; q < 4; ++q) v[q] = there ? gate_act<GATE>(v[q]) * u[q] : 0.0f;
            }
            store4<float>(row, v, F - n);
        }
    }
}

struct Tile128 : Tile<2, 4, 64, 32> { static constexpr int PER_CU = 1; };
struct Tile64 : Tile<2, 2, 32, 32> { static constexpr int PER_CU = 3; };

template <class TL, int OP, int GATE>
hipError_t launch_tile(ExpertProduct g, hipStream_t stream)
{
    g.tiles_m = (int)((g.M + TL::BM - 1) / TL::BM);        // dW only: elsewhere from the offsets
    g.tiles_n = (int)((g.N + TL::BN - 1) / TL::BN);
    const int64_t segments = g.n + 1;
    const int64_t rows = OP == kBackW ? weight_chunks(g) * g.tiles_m : g.P / TL::BM + (segments < g.P ? segments : g.P);
    const int64_t blocks = rows * g.tiles_n;
    if (!grid_ok(blocks)) return hipErrorInvalidValue;
    hipLaunchKernelGGL((expert_f32_kernel<TL, OP, GATE>), grid_of(blocks), dim3(TL::NT), 0, stream, g);
    return hipGetLastError();
}

// 128 x 128 tiles where they fill half of the CUs, else 64 x 64 (dX of 12288 x 1024 -> 256,
// 208 tiles: 62 us against 90).
template <int OP, int GATE>
hipError_t launch_op(const ExpertProduct &g, hipStream_t stream)
{
    const int64_t tm = OP == kBackW ? weight_chunks(g) * ((g.M + 127) / 128) : g.P / 128, tn = (g.N + 127) / 128;
    if (2 * tm * tn >= g.num_cus) return launch_tile<Tile128, OP, GATE>(g, stream);
    return launch_tile<Tile64, OP, GATE>(g, stream);
}

}  // namespace

hipError_t launch_expert_f32(int op, const ExpertProduct &g, hipStream_t stream)
{
    if (op == kBackX) return launch_op<kBackX, -1>(g, stream);
    if (op == kBackW) return launch_op<kBackW, -1>(g, stream);
    switch (g.gate) {
    case kSilu: return launch_op<kForward, kSilu>(g, stream);
    case kGelu: return launch_op<kForward, kGelu>(g, stream);
    case kGeluTanh: return launch_op<kForward, kGeluTanh>(g, stream);
    case kSigmoid: return launch_op<kForward, kSigmoid>(g, stream);
    case kRelu: return launch_op<kForward, kRelu>(g, stream);
    default: return launch_op<kForward, -1>(g, stream);
    }
}

}  // namespace sgemm_emu_dev
