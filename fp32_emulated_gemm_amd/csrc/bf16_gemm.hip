// bf16_gemm.hip -- bfloat16 products C = A B^T on the BF16 matrix cores, with
// the gated product or the low-rank adapters' part in the epilogue.
//
// A bfloat16 value is its own first component: one product takes the place of
// the nine of the FP32 emulation, accumulated in FP32 and rounded once.
//
// One workgroup per BM x BN output tile.  K advances in steps of 64, two MFMA
// slices; both operands' tiles of a step (128-byte rows, so that a copy takes
// whole cache lines; the 16-byte slot of k group kg of row r at slot
// kg ^ ((r >> 1) & 7), which keeps the 128-bit fragment reads of 16 rows on
// distinct banks) are copied global -> LDS by buffer loads with LDS destination
// into a ring of buffers.  A step enters with its first slice's fragments in
// registers: it reads the second slice's under the first slice's MFMAs, passes
// one LDS-only barrier, behind which its buffer is free for the copies of the
// step a ring ahead, and reads the next step's first slice under its second
// slice's MFMAs.
// v_mfma_f32_16x16x32_bf16 rather than 32x32x16: an accumulator is read and
// written once per 32 products instead of 16, and this load runs at the chip's
// power limit.
//
// The MFMAs take B's rows as their first operand, so a lane's accumulator
// registers run along N for one row of C (its column in the MFMA's result):
// gate and up rows of a gated product are dealt to the tile in alternating
// blocks of 16, which puts act(gate) and up of one output into one lane, and
// the adapters' part selects its rows per lane.
// The result goes through LDS (the ring's space) and leaves in 128-bit stores.
//
// Bound by the matrix cores at the power limit: 8192 x 4096 -> 2 x 8192 gated 816-830
// us, 1.34 PFLOP/s (the platform's library 1.34 on the plain product); 8192 x 4096 x
// 4096 with adapters of rank 16 230 us, 1.19, of which about 13 us are the start and
// the end of a tile.
#include "bf16_tile.hpp"
#include "ops.hpp"

namespace sgemm_emu_dev {

namespace {

enum { EPI_PLAIN = 0, EPI_GATED = 1, EPI_ADAPTER = 2, EPI_PARTIAL = 3 };

// Row of B behind tile row c (see the file's head).
template <int EPI>
__device__ __forceinline__ int64_t b_row(const Bf16Gemm &g, int64_t n0, int c)
{
    if constexpr (EPI == EPI_GATED) return gated_row(g.N >> 1, n0, c);
    else return lmin(n0 + c, g.N - 1);
}

// The accumulators' start: the adapters' part, up[i][n][:] . S[m][:] for the
// rows m of adapter i, zeros for rows without one.  S comes in two BF16 parts (16
// significant bits; the rest lies 2^-8 below the output's own rounding), up is
// exact: 16 ranks' high and low parts are the 32 k of one MFMA.
// A wave whose rows share one adapter (the inside of a request) multiplies them
// all at once.  Elsewhere each block of 16 rows takes its adapters one after
// another (in order of their first row), and a lane keeps the products of its
// own row's: zero times Inf or NaN in one adapter's weights never reaches
// another's rows.
template <class T>
__device__ __forceinline__ void start_adapters(f32x4_t (&acc)[T::NI][T::MI], const Bf16Gemm &g, int64_t m0w,
                                               int64_t n0w, int lane)
{
    int id[T::MI];
#pragma unroll
    for (int i = 0; i < T::MI; ++i) {
        // rows past M count as the last one: they are dropped
        const int v = g.ids[lmin(m0w + i * 16 + (lane & 15), g.M - 1)];
        id[i] = v >= 0 && v < g.n ? v : -1;
    }
    // Rows and ranks past the matrices read zeros: their offsets lie past the
    // descriptors.
    const int r8 = 8 * ((lane >> 4) & 1);                        // first rank of this lane
    const uint32_t srow = (uint32_t)(((lane & 15) * 2 + (lane >> 5)) * g.rp + r8) * 2u;   // high or low part
    const uint32_t urow = (uint32_t)((lane & 15) * g.r + r8) * 2u;
    const uint32_t sblock = (uint32_t)g.rp * 64u, ublock = (uint32_t)g.r * 32u;           // bytes of 16 rows
    const rsrc_t rs = make_rsrc(g.S + m0w * 2 * g.rp, (g.M - m0w) * 2 * g.rp * 2);
    auto bank = [&](int me) { return make_rsrc(g.up + ((int64_t)me * g.N + n0w) * g.r, (g.N - n0w) * g.r * 2); };
    // Eight ranks from rc + r8 on; those past the rank belong to the next row of
    // up, and S's zeros would not take an Inf or NaN of it away.
    auto load_up = [&](u32x4_t (&up)[T::NI], rsrc_t ru, int64_t rc) {
        const int64_t left = g.r - (rc + r8);
#pragma unroll
        for (int j = 0; j < T::NI; ++j) {
            up[j] = bload_u32x4(ru, left > 0 ? urow + j * ublock + (uint32_t)rc * 2u : OUT_OF_RANGE, 0);
            if ((g.r & 7) != 0) {
#pragma unroll
                for (int e = 0; e < 4; ++e) up[j][e] = 2 * e < left ? up[j][e] : 0u;
            }
        }
    };
    const int first = __builtin_amdgcn_readfirstlane(id[0]);
    bool same = true;
#pragma unroll
    for (int i = 0; i < T::MI; ++i) same = same && id[i] == first;
    if (__all(same)) {
        if (first < 0) return;
        const rsrc_t ru = bank(first);
        for (int64_t rc = 0; rc < g.rp; rc += 16) {
            u32x4_t up[T::NI], sv[T::MI];
            load_up(up, ru, rc);
#pragma unroll
            for (int i = 0; i < T::MI; ++i) sv[i] = bload_u32x4(rs, srow + i * sblock + (uint32_t)rc * 2u, 0);
#pragma unroll
            for (int i = 0; i < T::MI; ++i)
#pragma unroll
                for (int j = 0; j < T::NI; ++j)
                    acc[j][i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                        __builtin_bit_cast(bf16x8_t, up[j]), __builtin_bit_cast(bf16x8_t, sv[i]), acc[j][i], 0, 0, 0);
        }
        return;
    }
#pragma unroll
    for (int i = 0; i < T::MI; ++i) {
        f32x4_t mine[T::NI];
#pragma unroll
        for (int j = 0; j < T::NI; ++j) mine[j] = f32x4_t{};
        uint32_t todo = (uint32_t)__ballot(id[i] >= 0) & 0xFFFFu;
        while (todo != 0) {
            const int me = __builtin_amdgcn_readlane(id[i], __builtin_ctz(todo));
            todo &= ~(uint32_t)__ballot(id[i] == me);
            const rsrc_t ru = bank(me);
            f32x4_t t[T::NI];
#pragma unroll
            for (int j = 0; j < T::NI; ++j) t[j] = f32x4_t{};
            for (int64_t rc = 0; rc < g.rp; rc += 16) {
                u32x4_t up[T::NI];
                load_up(up, ru, rc);
                const u32x4_t sv = bload_u32x4(rs, srow + i * sblock + (uint32_t)rc * 2u, 0);
#pragma unroll
                for (int j = 0; j < T::NI; ++j)
                    t[j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, up[j]),
                                                                   __builtin_bit_cast(bf16x8_t, sv), t[j], 0, 0, 0);
            }
#pragma unroll
            for (int j = 0; j < T::NI; ++j)
#pragma unroll
                for (int q = 0; q < 4; ++q) mine[j][q] = id[i] == me ? t[j][q] : mine[j][q];
        }
#pragma unroll
        for (int j = 0; j < T::NI; ++j) acc[j][i] = mine[j];
    }
}

template <class T, int EPI, int GATE, bool KTAIL>
__device__ __forceinline__ void gemm_tile(const Bf16Gemm &g, uint16_t *lds)
{
    typedef __attribute__((address_space(3))) void lds_void_t;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wm = wave / T::WAVES_N, wn = wave % T::WAVES_N;

    int tm, tn;
    tile_of_index((int)blockIdx.x, (int)gridDim.x, g.tiles_m, g.tiles_n, g.group_m, tm, tn);
    const int64_t m0 = g.m_base + (int64_t)tm * T::BM, n0 = g.n_base + (int64_t)tn * T::BN;
    const int64_t kb = (int64_t)blockIdx.y * g.k_per_split, ke = lmin(kb + g.k_per_split, g.K);
    const int nk = (int)((ke - kb + KS - 1) / KS);

    // Copies: lane -> (row, 16-byte slot) of an 8-row block.  A lane's offset from
    // its block's first row is fixed; k advances in the scalar offset, so a copy
    // costs no vector arithmetic.  Copies past the last step repeat it (nobody
    // reads them), so every access lies inside the operand; in the last step of a
    // K that is not a multiple of KS the lanes past K read zeros.
    const int srow = lane >> 3;
    rsrc_t ra[T::A_COPIES], rb[T::B_COPIES];
    uint32_t aoff[T::A_COPIES], boff[T::B_COPIES], aend[T::A_COPIES], bend[T::B_COPIES];
    const int64_t klast = (ke - kb) - (int64_t)(nk - 1) * KS;        // k of the last step
#pragma unroll
    for (int d = 0; d < T::A_COPIES; ++d) {
        const int r = (wave * T::A_COPIES + d) * 8, kg = kslot(r + srow, lane & 7) * 8;
        const int64_t first = lmin(m0 + r, g.M - 1), mine = lmin(m0 + r + srow, g.M - 1);
        ra[d] = make_rsrc(g.A + first * g.lda + kb, 0xFFFFFFF0ll);
        aoff[d] = (uint32_t)(((mine - first) * g.lda + kg) * 2);
        aend[d] = kg < klast ? aoff[d] : OUT_OF_RANGE;
    }
#pragma unroll
    for (int d = 0; d < T::B_COPIES; ++d) {
        const int r = (wave * T::B_COPIES + d) * 8, kg = kslot(r + srow, lane & 7) * 8;
        const int64_t first = b_row<EPI>(g, n0, r), mine = b_row<EPI>(g, n0, r + srow);
        rb[d] = make_rsrc(g.B + first * g.ldb + kb, 0xFFFFFFF0ll);
        boff[d] = (uint32_t)(((mine - first) * g.ldb + kg) * 2);
        bend[d] = kg < klast ? boff[d] : OUT_OF_RANGE;
    }
    auto stage = [&](int kt) {
        uint16_t *const buf = lds + (kt % T::RING) * T::STAGE;
        const bool end = KTAIL && kt >= nk - 1;
        const int soff = (kt < nk ? kt : nk - 1) * (KS * 2);
#pragma unroll
        for (int d = 0; d < T::A_COPIES; ++d)
            __builtin_amdgcn_raw_ptr_buffer_load_lds(
                ra[d], (lds_void_t *)(buf + (wave * T::A_COPIES + d) * 8 * KS), 16, (int)(end ? aend[d] : aoff[d]),
                soff, 0, 0);
#pragma unroll
        for (int d = 0; d < T::B_COPIES; ++d)
            __builtin_amdgcn_raw_ptr_buffer_load_lds(
                rb[d], (lds_void_t *)(buf + T::BM * KS + (wave * T::B_COPIES + d) * 8 * KS), 16,
                (int)(end ? bend[d] : boff[d]), soff, 0, 0);
    };

    f32x4_t acc[T::NI][T::MI];
#pragma unroll
    for (int j = 0; j < T::NI; ++j)
#pragma unroll
        for (int i = 0; i < T::MI; ++i) acc[j][i] = f32x4_t{};

    // acc[j][i][q]: row m0w + 16 i + (lane & 15), column n0w + 16 j + 4 (lane >> 4) + q
    const int64_t m0w = m0 + wm * T::TM, n0w = n0 + wn * T::TN;
    constexpr int COPIES = T::A_COPIES + T::B_COPIES;
    if (nk > 0) {
#pragma unroll
        for (int q = 0; q < T::RING; ++q) stage(q);
    }
    // The adapters' part first, while the copies are under way: behind the loop it
    // would take the registers that the loop needs.
    if constexpr (EPI == EPI_ADAPTER) start_adapters<T>(acc, g, m0w, n0w, lane);
    if (nk > 0) {
        Frag<T> f0, f1;
        wait_vmem_at_most<(T::RING - 1) * COPIES>();
        lds_barrier();
        read_frag<T>(f0, lds, 0, wm, wn, lane);
        for (int kt = 0; kt < nk; ++kt) {
            const uint16_t *const buf = lds + (kt % T::RING) * T::STAGE, *const next = lds + ((kt + 1) % T::RING) * T::STAGE;
            constexpr int NM = T::MI * T::NI, NR = T::MI + T::NI;
            read_frag<T>(f1, buf, 1, wm, wn, lane);
            mfma_slice<T>(acc, f0);
            spread<NM, NR, 0x100>();
            step_barrier<(T::RING - 2) * COPIES>();   // step kt + 1 has landed, buf's readers are done
            read_frag<T>(f0, next, 0, wm, wn, lane);
            stage(kt + T::RING);
            mfma_slice<T>(acc, f1);
            spread<NM, NR, 0x100, COPIES, 0x020>();
            __builtin_amdgcn_sched_barrier(0);
        }
    }
    wait_vmem_at_most<0>();                  // no copy may land in the epilogue's space
    lds_barrier();

    const int mlane = lane & 15, quad = 4 * (lane >> 4);
    if constexpr (EPI == EPI_PARTIAL) {
        float *const part = g.partials + (int64_t)blockIdx.y * g.M * g.N;
        const bool vec = g.N % 4 == 0;
#pragma unroll
        for (int i = 0; i < T::MI; ++i) {
            const int64_t m = m0w + i * 16 + mlane;
            if (m >= g.M) continue;
#pragma unroll
            for (int j = 0; j < T::NI; ++j) {
                const int64_t n = n0w + j * 16 + quad;
                float *const p = part + m * g.N + n;
                if (vec && n + 4 <= g.N) {
                    *reinterpret_cast<f32x4_t *>(p) = acc[j][i];
                } else {
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (n + e < g.N) p[e] = acc[j][i][e];
                }
            }
        }
        return;
    }
    uint16_t *const out = lds + wave * T::EPI_WAVE;
    if constexpr (EPI == EPI_GATED) {
        // blocks 2 p are gate rows, 2 p + 1 the up rows of the same 16 outputs
        const int64_t F = g.N >> 1, f0w = n0w >> 1;
#pragma unroll
        for (int p = 0; p < T::NI / 2; ++p) {
            float bg[4] = {0, 0, 0, 0}, bu[4] = {0, 0, 0, 0};
            if (g.bias != nullptr) {
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const int64_t f = lmin(f0w + p * 16 + quad + q, F - 1);
                    bg[q] = bf2f(g.bias[f]);
                    bu[q] = bf2f(g.bias[F + f]);
                }
            }
#pragma unroll
            for (int i = 0; i < T::MI; ++i) {
                f32x4_t zg, zu;
                float h[4];
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    zg[q] = acc[2 * p][i][q] + bg[q];
                    zu[q] = acc[2 * p + 1][i][q] + bu[q];
                    h[q] = gate_act<GATE>(zg[q]) * zu[q];
                }
                put4<T>(out, i * 16 + mlane, p * 16 + quad, h[0], h[1], h[2], h[3]);
                if (g.Z != nullptr) {
                    // pre-activations stay in 32 bits: a lane's four are 16 bytes of a row,
                    // whose padding to a multiple of 8 always takes them
                    const int64_t m = m0w + i * 16 + mlane, f = f0w + p * 16 + quad;
                    if (m < g.M && f < F) {
                        float *const z = g.Z + m * g.ldz + f;
                        *reinterpret_cast<f32x4_t *>(z) = zg;
                        *reinterpret_cast<f32x4_t *>(z + g.ldz / 2) = zu;
                    }
                }
            }
        }
        wave_fence();
        flush_block<T, T::TN / 2>(out, g.C, g.ldc, g.M, F, m0w, f0w, lane);
    } else {
#pragma unroll
        for (int j = 0; j < T::NI; ++j) {
            float b[4] = {0, 0, 0, 0};
            if (g.bias != nullptr) {
#pragma unroll
                for (int q = 0; q < 4; ++q) b[q] = bf2f(g.bias[lmin(n0w + j * 16 + quad + q, g.N - 1)]);
            }
#pragma unroll
            for (int i = 0; i < T::MI; ++i)
                put4<T>(out, i * 16 + mlane, j * 16 + quad, acc[j][i][0] + b[0], acc[j][i][1] + b[1],
                        acc[j][i][2] + b[2], acc[j][i][3] + b[3]);
        }
        wave_fence();
        flush_block<T, T::TN>(out, g.C, g.ldc, g.M, g.N, m0w, n0w, lane);
    }
}

template <class T, int EPI, int GATE, bool KTAIL>
__global__ __launch_bounds__(T::NT, T::PER_CU) void bf16_gemm_kernel(Bf16Gemm g)
{
    __shared__ __attribute__((aligned(16))) uint16_t lds[T::LDS];
    gemm_tile<T, EPI, GATE, KTAIL>(g, lds);
}

// C = bf16(sum of the K slices' products, in slice order, + bias).
__global__ __launch_bounds__(256) void bf16_sum_slices_kernel(Bf16Gemm g)
{
    const int64_t plane = g.M * g.N, c = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (c >= g.N) return;
    for (int64_t m = blockIdx.y; m < g.M; m += gridDim.y) {
        float v = 0.0f;
        for (int s = 0; s < g.splits; ++s) v += g.partials[s * plane + m * g.N + c];
        if (g.bias != nullptr) v += bf2f(g.bias[c]);
        g.C[m * g.ldc + c] = f2bf(v);
    }
}

// ---------------------------------------------------------------- tiles

// The part of a product that one launch covers: tiles from row m_base, column
// n_base (multiples of the tile) to row m_end, column n_end.
struct Part {
    int64_t m_base, n_base, m_end, n_end;
};

template <class T, int EPI, int GATE>
void launch_tile(Bf16Gemm g, const Part &p, hipStream_t stream)
{
    g.m_base = p.m_base;
    g.n_base = p.n_base;
    g.tiles_m = (int)((p.m_end - p.m_base + T::BM - 1) / T::BM);
    // a gated tile holds BN / 2 outputs of F = N / 2
    g.tiles_n = (int)((p.n_end - p.n_base + T::BN - 1) / T::BN);
    g.group_m = g.tiles_m < 8 ? g.tiles_m : 8;
    const dim3 grid((unsigned)((int64_t)g.tiles_m * g.tiles_n), (unsigned)g.splits);
    // K slices begin at multiples of KS, so only the last can end inside a step
    if (g.K % KS == 0) hipLaunchKernelGGL((bf16_gemm_kernel<T, EPI, GATE, false>), grid, dim3(T::NT), 0, stream, g);
    else hipLaunchKernelGGL((bf16_gemm_kernel<T, EPI, GATE, true>), grid, dim3(T::NT), 0, stream, g);
}

template <class T>
hipError_t launch_epi(const Bf16Gemm &g, const Part &p, hipStream_t stream)
{
    if (g.splits > 1) {
        launch_tile<T, EPI_PARTIAL, 0>(g, p, stream);
        const dim3 grid((unsigned)((g.N + 255) / 256), (unsigned)(g.M < 16384 ? g.M : 16384));
        hipLaunchKernelGGL(bf16_sum_slices_kernel, grid, dim3(256), 0, stream, g);
        return hipGetLastError();
    }
    switch (g.gate) {
    case kSilu: launch_tile<T, EPI_GATED, kSilu>(g, p, stream); break;
    case kGelu: launch_tile<T, EPI_GATED, kGelu>(g, p, stream); break;
    case kGeluTanh: launch_tile<T, EPI_GATED, kGeluTanh>(g, p, stream); break;
    case kSigmoid: launch_tile<T, EPI_GATED, kSigmoid>(g, p, stream); break;
    case kRelu: launch_tile<T, EPI_GATED, kRelu>(g, p, stream); break;
    default:
        if (g.ids != nullptr) launch_tile<T, EPI_ADAPTER, 0>(g, p, stream);
        else launch_tile<T, EPI_PLAIN, 0>(g, p, stream);
    }
    return hipGetLastError();
}

enum { TILE_64, TILE_128_DEEP, TILE_128, TILE_256, TILES };

hipError_t launch_part(int tile, const Bf16Gemm &g, const Part &p, hipStream_t stream)
{
    switch (tile) {
    case TILE_256: return launch_epi<Tile256>(g, p, stream);
    case TILE_128: return launch_epi<Tile128>(g, p, stream);
    case TILE_128_DEEP: return launch_epi<Tile128Deep>(g, p, stream);
    default: return launch_epi<Tile64>(g, p, stream);
    }
}

int64_t tiles_of(int64_t M, int64_t N, int64_t t) { return ((M + t - 1) / t) * ((N + t - 1) / t); }

// Expected time of `rounds` of tiles over K, in tenths of a us: per K step of 64
// and per round, as measured on 256 CUs (128 .. 10922 x 288 .. 10240 x 256 ..
// 8192).  A round is one workgroup per CU, or two for TILE_64 and TILE_128; 64 x 64
// tiles with a CU each take 0.22 us a step.
//   1024 x 4096 x 4096: 64: 51 us, 128 deep: 34, 128: 47, 256: 74
//   2048 x 4096 x 4096:     97             67       60       81
//   8192 x 2048 x 8192:    358            245      219      183
//    512 x 4096 x 4096:     26             30       44       73
int64_t tile_cost(int tile, int64_t M, int64_t N, int64_t K, int64_t splits, int num_cus)
{
    static const struct { int size, per_cu, step, fixed; } t[TILES] = {
        {64, 2, 38, 20}, {128, 1, 43, 35}, {128, 2, 82, 50}, {256, 1, 138, 100}};
    const int64_t steps = (K + KS * splits - 1) / (KS * splits), tiles = tiles_of(M, N, t[tile].size) * splits;
    const int64_t slots = (int64_t)num_cus * t[tile].per_cu;
    const int64_t step = tile == TILE_64 && tiles <= num_cus ? 22 : t[tile].step;
    return (tiles + slots - 1) / slots * (steps * step + t[tile].fixed * 10) / 10;
}

int best_tile(int64_t M, int64_t N, int64_t K, int64_t splits, int num_cus, int64_t *cost)
{
    int best = TILE_64;
    *cost = tile_cost(TILE_64, M, N, K, splits, num_cus);
    for (int t = TILE_64 + 1; t < TILES; ++t) {
        const int64_t c = tile_cost(t, M, N, K, splits, num_cus);
        if (c < *cost) { *cost = c; best = t; }
    }
    return best;
}

// How a product is run: one tile, over K slices where there are few tiles; or
// whole rounds of 256 x 256 tiles and the rows (or columns) left over as a second
// launch of smaller tiles, which spares a last round that few tiles fill
// (10922 x 2048 x 8192: 317 us as 344 tiles, 283 as 256 and 352 small ones).
struct TilePlan {
    int tile;
    int64_t splits;
    Part main;
    int tail_tile;           // -1: none
    Part tail;
};

TilePlan tile_plan(int64_t M, int64_t N, int64_t K, bool plain, int num_cus)
{
    const Part whole{0, 0, M, N};
    TilePlan p{0, 1, whole, -1, whole};
    int64_t cost = 0;
    p.tile = best_tile(M, N, K, 1, num_cus, &cost);
    const int64_t tm = (M + 255) / 256, tn = (N + 255) / 256, rounds = tm * tn / num_cus;
    if (rounds > 0) {
        for (int along_n = 0; along_n < 2; ++along_n) {
            const int64_t lines = rounds * num_cus / (along_n ? tm : tn), at = 256 * lines;
            if (lines == 0 || at >= (along_n ? N : M)) continue;
            const Part a = along_n ? Part{0, 0, M, at} : Part{0, 0, at, N},
                       b = along_n ? Part{0, at, M, N} : Part{at, 0, M, N};
            int64_t rest = 0;
            const int t = best_tile(b.m_end - b.m_base, b.n_end - b.n_base, K, 1, num_cus, &rest);
            const int64_t c = tile_cost(TILE_256, a.m_end, a.n_end, K, 1, num_cus) + rest + 30;
            if (c < cost) {
                cost = c;
                p.tile = TILE_256;
                p.main = a;
                p.tail_tile = t;
                p.tail = b;
            }
        }
    }
    // the slices' sums pass through memory twice, at about 4 TB/s
    for (int64_t s = 2; plain && s <= 16 && K / s >= 512; ++s) {
        int64_t c = 0;
        const int t = best_tile(M, N, K, s, num_cus, &c);
        c += 50 + (8 * s + 2) * M * N / 400000;
        if (c < cost) {
            cost = c;
            p = TilePlan{t, s, whole, -1, whole};
        }
    }
    return p;
}

}  // namespace

int64_t bf16_gemm_partial_floats(int64_t M, int64_t N, int64_t K, bool plain, int num_cus)
{
    const TilePlan p = tile_plan(M, N, K, plain, num_cus);
    return p.splits > 1 ? p.splits * M * N : 0;
}

hipError_t launch_bf16_gemm(const Bf16Gemm &args, int num_cus, hipStream_t stream)
{
    Bf16Gemm g = args;
    if (g.M == 0 || g.N == 0) return hipSuccess;
    if (g.K == 0) {                          // nothing is read: every copy is past the end of K
        g.A = g.B = nullptr;
        g.lda = g.ldb = 8;
    }
    if (g.ids != nullptr && (g.r % 2 != 0 || !aligned(g.up, 4))) return hipErrorInvalidValue;
    if (g.K % 8 != 0 || g.lda % 8 != 0 || g.ldb % 8 != 0 || !aligned(g.A, 16) || !aligned(g.B, 16))
        return hipErrorInvalidValue;
    const bool plain = g.gate < 0 && g.ids == nullptr;
    const TilePlan p = tile_plan(g.M, g.N, g.K, plain && g.partials != nullptr, num_cus);
    g.splits = (int)p.splits;
    g.k_per_split = round_up((g.K + p.splits - 1) / p.splits, KS);
    const hipError_t e = launch_part(p.tile, g, p.main, stream);
    return e != hipSuccess || p.tail_tile < 0 ? e : launch_part(p.tail_tile, g, p.tail, stream);
}

}  // namespace sgemm_emu_dev
