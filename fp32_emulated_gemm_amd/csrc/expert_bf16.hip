// expert_bf16.hip -- the experts' bfloat16 products on operands that lie in 16-byte
// pieces: the tiles, ring and steps of bf16_gemm.hip (see there), on row tiles found
// from the offsets, with operands of either layout.
//
// An operand whose k are rows (W in dX, dZ and X in dW) is copied to LDS row piece by
// row piece like the other kind and read by ds_read_b64_tr_b16, four k of a column at
// a time.  A wave's read takes 32 bytes of each of 16 rows; 16-byte chunks of a row
// are permuted by its number so that the 8 rows of half a wave lie on all banks.
// Rows past an expert's last are not copied: their lanes' offsets lie past the
// descriptor and read zeros.
//
// The matrix cores bound it at the clock that the card's power allows: 32768 x 4096 ->
// 2048 over 16 experts takes 550 us, 1.0 PFLOP/s (the library's 8192^3 product on the
// same card: 1.13).  16382 x 2048 -> 2 x 1365: gated with Z 284 us, 645 TFLOP/s and 179 MB
// of Z; dX 234, 780; dW 226, 810.
#include "bf16_tile.hpp"
#include "expert_device.hpp"

namespace sgemm_emu_dev {

namespace {

typedef short s16x4_t __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) s16x4_t lds_s16x4_t;

// An operand's tile: R outputs' rows or columns by KS of k.
template <int R, bool KM, int WAVES>
struct Operand {
    static constexpr int COPIES = R / 8 / WAVES;           // per wave and step, 1 KB each
    static constexpr int WIDE = KM ? R / 8 : KS / 8;       // 16-byte chunks of an LDS row
    static constexpr int ROWS = 64 / WIDE;                 // LDS rows of a copy

    // Where chunk c of LDS row `row` lies.
    static __device__ __forceinline__ int slot(int row, int c)
    {
        if constexpr (!KM) return kslot(row, c);
        else if constexpr (WIDE == 8) return c ^ ((((row >> 1) & 1) | ((row >> 2) & 2)) << 1);
        else return c ^ (((row & 3) | ((row >> 1) & 4)) << 1);
    }
    // Fragment of a slice of 32 k: k 8 (lane >> 4) .. + 7 of index base + (lane & 15).
    static __device__ __forceinline__ bf16x8_t frag(const uint16_t *buf, int slice, int base, int lane)
    {
        if constexpr (KM) {
            const int i = lane & 15, col = base + 4 * (i & 3);
            s16x4_t v[2];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int k = slice * 32 + 8 * (lane >> 4) + 4 * h + (i >> 2);
                v[h] = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                    (lds_s16x4_t *)(buf + (k * WIDE + slot(k, col >> 3)) * 8 + (col & 7)));
            }
            return __builtin_bit_cast(bf16x8_t, __builtin_shufflevector(v[0], v[1], 0, 1, 2, 3, 4, 5, 6, 7));
        } else {
            const int row = base + (lane & 15);
            return ld_frag(buf + (row * WIDE + slot(row, slice * 4 + (lane >> 4))) * 8);
        }
    }
    static constexpr int READS = KM ? 2 : 1;               // LDS instructions of a fragment

    const uint16_t *p[KM ? 1 : COPIES];                    // !KM: first row of a copy
    uint32_t off[COPIES], end[COPIES];
    int row[COPIES];                                       // KM: k of the lane's row in a step

    // !KM: rows of the tile by `row_of` (clamped, wave-uniform but for the lane's own).
    template <class F>
    __device__ __forceinline__ void rows(const uint16_t *from, int64_t ld, int64_t klast, int wave, int lane, F row_of)
    {
#pragma unroll
        for (int d = 0; d < COPIES; ++d) {
            const int q = (wave * COPIES + d) * 8, kg = kslot(q + (lane >> 3), lane & 7) * 8;
            const int64_t first = row_of(q), mine = row_of(q + (lane >> 3));
            p[d] = from + first * ld;
            off[d] = (uint32_t)(((mine - first) * ld + kg) * 2);
            end[d] = kg < klast ? off[d] : OUT_OF_RANGE;
        }
    }
    // KM: columns c0.. of `cols`.
    __device__ __forceinline__ void columns(int64_t ld, int64_t c0, int64_t cols, int wave, int lane)
    {
#pragma unroll
        for (int d = 0; d < COPIES; ++d) {
            row[d] = (wave * COPIES + d) * ROWS + lane / WIDE;
            const int c = slot(row[d], lane % WIDE) * 8;
            off[d] = c0 + c < cols ? (uint32_t)((row[d] * ld + c) * 2) : OUT_OF_RANGE;
        }
    }
};

// A copy of 16 bytes a lane from `at` + off to LDS, as the builtin's, written out: the
// compiler does not know how the transposing reads relate to copies in flight and
// puts a wait for all of them before each group of reads, half a step too early.
// Here the steps' own waits (step_barrier) order them.  The wait states are those
// between a vector write of a scalar register, or a write of m0, and its use.  m0 is
// listed so that no value of the compiler's own is kept in it across a copy; its
// warning is that it saves none there either, which nothing here needs.
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
__device__ __forceinline__ void copy_untracked(uint32_t lds, const uint16_t *at, uint32_t off)
{
    const uint64_t p = (uint64_t)(uintptr_t)at;
    const u32x4_t r = {(uint32_t)__builtin_amdgcn_readfirstlane((uint32_t)p),
                       (uint32_t)__builtin_amdgcn_readfirstlane((uint32_t)(p >> 32)), 0xFFFFFFF0u, (uint32_t)RSRC_WORD3};
    asm volatile("s_mov_b32 m0, %0\n\t"
                 "s_nop 4\n\t"
                 "buffer_load_dwordx4 %1, %2, 0 offen lds" ::"s"(__builtin_amdgcn_readfirstlane(lds)), "v"(off), "s"(r)
                 : "memory", "m0");
}
#pragma clang diagnostic pop

// Which of a product's 256 x 256 tiles a launch covers: ALL (tiles of any size);
// WHOLE, all of them or, where the last round would fill less than half of the CUs,
// the rounds before it; REST, what WHOLE leaves, in quarters, two to a CU.  How many
// there are is known on the device only.
enum { ALL, WHOLE, REST };
__device__ __forceinline__ int whole_rounds(int tiles, int slots)
{
    const int rest = tiles % slots;
    return 2 * rest > slots ? tiles : tiles - rest;
}

template <class T, int OP, int GATE, int PART>
__global__ __launch_bounds__(T::NT, T::PER_CU) void expert_bf16_kernel(ExpertProduct g)
{
    constexpr bool GATED = GATE >= 0, A_KM = OP == kBackW, B_KM = OP != kForward;
    typedef Operand<T::BM, A_KM, T::WAVES> OA;
    typedef Operand<T::BN, B_KM, T::WAVES> OB;
    __shared__ __attribute__((aligned(16))) uint16_t lds[T::LDS];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wm = wave / T::WAVES_N, wn = wave % T::WAVES_N;

    // Tile `index` of REST's 256 x 256 tiles or this launch's own, in the order of
    // tile_of_index; of the former, this workgroup takes a quarter.
    constexpr bool QUARTER = PART == REST;
    constexpr int SIZE_M = QUARTER ? 256 : T::BM;
    int64_t e, m0, m_end, K, r0 = 0;
    int rows, tiles, tm, tn, chunk = 0;
    RowTiles<SIZE_M> row_tiles(g.offsets, g.n, g.P, OP == kBackW ? 0 : (int)g.n + 1, lane);
    if constexpr (OP == kBackW) {
        rows = g.tiles_m;
        tiles = (int)weight_chunks(g) * rows * g.tiles_n;
    } else {
        rows = row_tiles.total;
        tiles = rows * g.tiles_n;
    }
    int index = QUARTER ? (int)blockIdx.x >> 2 : workgroup();
    if constexpr (PART == ALL) {
        if (index >= tiles) return;
        if constexpr (OP != kBackW) index = xcd_order(index, tiles);
    } else {
        const int whole = whole_rounds(tiles, g.num_cus);
        if (index >= (QUARTER ? tiles - whole : whole)) return;
        index = QUARTER ? whole + index : OP == kBackW ? index : xcd_order(index, whole);
    }
    if constexpr (OP == kBackW) {
        const int per = rows * g.tiles_n;
        chunk = index / per;
        // each expert's tiles over all XCDs: their lengths differ from expert to expert
        tile_at(xcd_order(index - chunk * per, per), rows, g.tiles_n, imin(rows, 8), tm, tn);
        m0 = (int64_t)tm * SIZE_M;
        m_end = g.M;
        const RowTile r = weight_rows(g, chunk, lane);
        if (r.segment < 0) return;
        e = r.segment;
        r0 = r.row;
        K = r.end - r0;
    } else {
        tile_at(index, rows, g.tiles_n, imin(rows, 8), tm, tn);
        const RowTile r = row_tiles.find(tm);
        if (r.segment < 0) return;
        e = r.segment;
        m0 = r.row;
        m_end = r.end;
        K = e < g.n ? g.K : 0;                             // rows of no expert: zeros
    }
    int64_t n0 = (int64_t)tn * (QUARTER ? 256 : T::BN);
    if constexpr (QUARTER) {
        static_assert(T::BM == 128 && T::BN == 128, "quarters of 256 x 256");
        m0 += (blockIdx.x & 2) * 64;
        n0 += (blockIdx.x & 1) * 128;
        if (m0 >= m_end || n0 >= (GATED ? round_up(g.N, 32) : g.N)) return;
    }
    const bool there = OP == kBackW || e < g.n;
    const uint16_t *const A = (const uint16_t *)g.A;
    const uint16_t *const B = (const uint16_t *)g.B + (OP == kBackW || !there ? 0 : e * g.bank);
    const int nk = (int)((K + KS - 1) / KS);
    const int64_t klast = K - (int64_t)(nk - 1) * KS;

    OA oa;
    OB ob;
    if constexpr (A_KM) oa.columns(g.lda, m0, g.M, wave, lane);
    else oa.rows(A, g.lda, klast, wave, lane, [&](int c) { return lmin(m0 + c, m_end - 1); });
    if constexpr (B_KM) ob.columns(g.ldb, n0, g.N, wave, lane);
    else ob.rows(B, g.ldb, klast, wave, lane, [&](int c) { return GATED ? gated_row(g.N >> 1, n0, c) : lmin(n0 + c, g.N - 1); });

    // One copy of 1 KB: by a lane's offset from `at`, `soff` bytes further.
    auto copy = [&](uint16_t *buf, int q, const uint16_t *at, uint32_t off, int soff) {
        typedef __attribute__((address_space(3))) void lds_void_t;
        if constexpr (OP == kForward) {
            __builtin_amdgcn_raw_ptr_buffer_load_lds(make_rsrc(at, 0xFFFFFFF0ll), (lds_void_t *)(buf + q * 512), 16, (int)off,
                                                     soff, 0, 0);
        } else {
            copy_untracked((uint32_t)(uintptr_t)(lds_void_t *)(buf + q * 512), at, off);
        }
    };
    // Copies past the last step repeat it (nobody reads them).
    auto stage = [&](int kt) {
        uint16_t *const buf = lds + (kt % T::RING) * T::STAGE, *const bufb = buf + T::BM * KS;
        const int k = imin(kt, nk - 1);
        const bool last = k == nk - 1;
        const int64_t k0 = (int64_t)k * KS;
        const int left = (int)lmin(K - k0, KS);
#pragma unroll
        for (int d = 0; d < OA::COPIES; ++d) {
            const int q = wave * OA::COPIES + d;
            if constexpr (A_KM) copy(buf, q, A + (r0 + k0) * g.lda + m0, oa.row[d] < left ? oa.off[d] : OUT_OF_RANGE, 0);
            else copy(buf, q, OP == kForward ? oa.p[d] : oa.p[d] + k0, last ? oa.end[d] : oa.off[d], k * (KS * 2));
        }
        // dX: a step lies in one half of dZ's columns (h is a multiple of KS, or K itself)
        const bool up = OP == kBackX && k0 >= g.map.h;
        const int64_t in = up ? k0 - g.map.h : k0, row = OP == kBackW ? r0 + k0 : up ? g.map.F + in : in;
        const int rows = OP == kBackW ? left : (int)lmin(g.map.F - in, KS);
#pragma unroll
        for (int d = 0; d < OB::COPIES; ++d) {
            const int q = wave * OB::COPIES + d;
            if constexpr (B_KM) copy(bufb, q, B + row * g.ldb + n0, ob.row[d] < rows ? ob.off[d] : OUT_OF_RANGE, 0);
            else copy(bufb, q, ob.p[d], last ? ob.end[d] : ob.off[d], k * (KS * 2));
        }
    };
    auto read = [&](Frag<T> &f, const uint16_t *buf, int slice) {
#pragma unroll
        for (int j = 0; j < T::NI; ++j) f.b[j] = OB::frag(buf + T::BM * KS, slice, wn * T::TN + j * 16, lane);
#pragma unroll
        for (int i = 0; i < T::MI; ++i) f.a[i] = OA::frag(buf, slice, wm * T::TM + i * 16, lane);
    };

    f32x4_t acc[T::NI][T::MI];
#pragma unroll
    for (int j = 0; j < T::NI; ++j)
#pragma unroll
        for (int i = 0; i < T::MI; ++i) acc[j][i] = f32x4_t{};

    constexpr int COPIES = OA::COPIES + OB::COPIES;
    if (nk > 0) {
#pragma unroll
        for (int q = 0; q < T::RING; ++q) stage(q);
        Frag<T> f0, f1;
        wait_vmem_at_most<(T::RING - 1) * COPIES>();
        lds_barrier();
        read(f0, lds, 0);
        for (int kt = 0; kt < nk; ++kt) {
            const uint16_t *const buf = lds + (kt % T::RING) * T::STAGE, *const next = lds + ((kt + 1) % T::RING) * T::STAGE;
            constexpr int NM = T::MI * T::NI, NR = T::MI * OA::READS + T::NI * OB::READS;
            read(f1, buf, 1);
            mfma_slice<T>(acc, f0);
            spread<NM, NR, 0x100>();
            step_barrier<(T::RING - 2) * COPIES>();        // step kt + 1 has landed, buf's readers are done
            read(f0, next, 0);
            stage(kt + T::RING);
            mfma_slice<T>(acc, f1);
            spread<NM, NR, 0x100, COPIES, 0x020>();
            __builtin_amdgcn_sched_barrier(0);
        }
    }
    wait_vmem_at_most<0>();                                // no copy may land in the epilogue's space
    lds_barrier();

    // acc[j][i][q]: row m0w + 16 i + (lane & 15), column n0w + 16 j + 4 (lane >> 4) + q
    const int64_t m0w = m0 + wm * T::TM, n0w = n0 + wn * T::TN;
    const int mlane = lane & 15, quad = 4 * (lane >> 4);
    if constexpr (OP == kBackW && PART == ALL) {
        if (g.partials != nullptr) {
#pragma unroll
            for (int i = 0; i < T::MI; ++i) {
                const int64_t m = m0w + i * 16 + mlane;
                if (m >= g.M) continue;
#pragma unroll
                for (int j = 0; j < T::NI; ++j) {
                    const int64_t n = n0w + j * 16 + quad;   // N is a multiple of 8: four lie inside or outside
                    if (n < g.N) *reinterpret_cast<f32x4_t *>(g.partials + (chunk * g.M + m) * g.N + n) = acc[j][i];
                }
            }
            return;
        }
    }
    uint16_t *const out = lds + wave * T::EPI_WAVE;
    const uint16_t *const bias = OP == kForward && there && g.bias != nullptr ? (const uint16_t *)g.bias + e * g.N : nullptr;
    if constexpr (GATED) {
        const int64_t F = g.N >> 1, f0w = n0w >> 1;
#pragma unroll
        for (int p = 0; p < T::NI / 2; ++p) {
            float bg[4] = {0, 0, 0, 0}, bu[4] = {0, 0, 0, 0};
            if (bias != nullptr) {
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const int64_t f = lmin(f0w + p * 16 + quad + q, F - 1);
                    bg[q] = bf2f(bias[f]);
                    bu[q] = bf2f(bias[F + f]);
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
                    h[q] = there ? gate_act<GATE>(zg[q]) * zu[q] : 0.0f;
                }
                put4<T>(out, i * 16 + mlane, p * 16 + quad, h[0], h[1], h[2], h[3]);
                if (g.Z != nullptr && there) {
                    const int64_t m = m0w + i * 16 + mlane, f = f0w + p * 16 + quad;
                    if (m < m_end && f < F) {
                        float *const z = g.Z + m * g.ldz + f;
                        *reinterpret_cast<f32x4_t *>(z) = zg;
                        *reinterpret_cast<f32x4_t *>(z + g.ldz / 2) = zu;
                    }
                }
            }
        }
        wave_fence();
        flush_block<T, T::TN / 2>(out, (uint16_t *)g.C, g.ldc, m_end, F, m0w, f0w, lane);
    } else {
#pragma unroll
        for (int j = 0; j < T::NI; ++j) {
            float b[4] = {0, 0, 0, 0};
            if (bias != nullptr) {
#pragma unroll
                for (int q = 0; q < 4; ++q) b[q] = bf2f(bias[lmin(n0w + j * 16 + quad + q, g.N - 1)]);
            }
#pragma unroll
            for (int i = 0; i < T::MI; ++i)
                put4<T>(out, i * 16 + mlane, j * 16 + quad, acc[j][i][0] + b[0], acc[j][i][1] + b[1],
                        acc[j][i][2] + b[2], acc[j][i][3] + b[3]);
        }
        wave_fence();
        uint16_t *C = (uint16_t *)g.C;
        if constexpr (OP == kBackW) {
            // a wave's rows lie in one half of dZ's columns (h is a multiple of its rows, or M itself)
            const bool up = m0w >= g.map.h;
            const int64_t in = up ? m0w - g.map.h : m0w, first = up ? g.map.F : 0;
            C += e * g.bank + first * g.ldc;
            if (!up || g.map.h < g.M) flush_block<T, T::TN>(out, C, g.ldc, g.map.F, g.N, in, n0w, lane);
        } else {
            flush_block<T, T::TN>(out, C, g.ldc, m_end, g.N, m0w, n0w, lane);
        }
    }
}

template <class T, int OP, int GATE, int PART>
hipError_t launch_part(ExpertProduct g, hipStream_t stream)
{
    constexpr int BM = PART == REST ? 256 : T::BM, BN = PART == REST ? 256 : T::BN;
    g.tiles_m = (int)((g.M + BM - 1) / BM);                // dW only: elsewhere from the offsets
    g.tiles_n = (int)((g.N + BN - 1) / BN);
    const int64_t segments = g.n + 1, rows = OP == kBackW ? weight_chunks(g) * g.tiles_m : g.P / BM + (segments < g.P ? segments : g.P);
    int64_t blocks = rows * g.tiles_n;
    if (PART == REST) blocks = 4 * (g.num_cus / 2 < blocks ? g.num_cus / 2 : blocks);
    if (!grid_ok(blocks)) return hipErrorInvalidValue;
    hipLaunchKernelGGL((expert_bf16_kernel<T, OP, GATE, PART>), grid_of(blocks), dim3(T::NT), 0, stream, g);
    return hipGetLastError();
}

enum { TILE_64, TILE_128, TILE_256, TILES };

// The tile with the least expected time, from the rounds of tiles over the CUs and
// the times of a step and of a tile's ends on 256 CUs, in tenths of a us, as in
// bf16_gemm.hip.  An expert's last row tile is half filled on average.
int best_tile(int op, const ExpertProduct &g)
{
    if (op == kBackW && g.partials != nullptr) return TILE_128;
    static const struct { int size, per_cu, step, fixed, keep; } t[TILES] = {
        {64, 2, 38, 20, 60}, {128, 2, 82, 50, 210}, {256, 1, 138, 100, 280}};
    const int64_t steps = ((op == kBackW ? g.P / g.n : g.K) + KS - 1) / KS;
    // kept pre-activations leave at a tile's end: 16382 x 2048 -> 2 x 1365 takes 250 us in
    // three whole rounds of 256 x 256 tiles and 38 for the rest, 310 in six of 128 x 128
    auto round = [&](int i, int64_t step) { return steps * step + (t[i].fixed + (g.Z != nullptr ? t[i].keep : 0)) * 10; };
    int best = TILE_64;
    int64_t least = INT64_MAX;
    for (int i = 0; i < TILES; ++i) {
        const int64_t s = t[i].size, slots = (int64_t)g.num_cus * t[i].per_cu;
        const int64_t rows = op == kBackW ? g.n * ((g.M + s - 1) / s) : g.P / s + (g.n + 1) / 2;
        const int64_t tiles = (rows > 0 ? rows : 1) * ((g.N + s - 1) / s), rest = tiles % slots;
        const int64_t one = round(i, i == TILE_64 && tiles <= g.num_cus ? 22 : t[i].step);
        int64_t c = (tiles + slots - 1) / slots * one;
        if (i == TILE_256 && 2 * rest <= slots) c = tiles / slots * one + (rest > 0 ? round(TILE_128, t[TILE_128].step) : 0) + 300;
        if (c < least) {
            least = c;
            best = i;
        }
    }
    return best;
}

template <int OP, int GATE>
hipError_t launch_op(const ExpertProduct &g, hipStream_t stream)
{
    switch (best_tile(OP, g)) {
    case TILE_256: {
        const hipError_t e = launch_part<Tile256, OP, GATE, WHOLE>(g, stream);
        return e != hipSuccess ? e : launch_part<Tile128, OP, GATE, REST>(g, stream);
    }
    case TILE_128: return launch_part<Tile128, OP, GATE, ALL>(g, stream);
    default: return launch_part<Tile64, OP, GATE, ALL>(g, stream);
    }
}

}  // namespace

bool expert_lies(int op, const ExpertProduct &g)
{
    const bool rows = g.lda % 8 == 0 && g.ldb % 8 == 0 && aligned(g.A, 16) && aligned(g.B, 16);
    // chunks of eight lie inside or outside; a bank's experts begin at pieces
    if (op == kForward) return rows && g.K % 8 == 0;
    if (op == kBackX) return rows && g.K % 8 == 0 && g.N % 8 == 0 && g.bank % 8 == 0;
    return rows && g.M % 8 == 0 && g.N % 8 == 0;
}

hipError_t launch_expert_bf16(int op, const ExpertProduct &g, hipStream_t stream)
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
