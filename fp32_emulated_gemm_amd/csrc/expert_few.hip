// expert_few.hip -- the experts' forward products with few rows: single tokens.
//
// A tile of expert_f32.hip or expert_bf16.hip takes its K steps one behind the other,
// which with few tiles is all the time there is.  Here a workgroup takes 16 rows of an
// expert and 16 outputs, and its waves take the blocks of 128 columns in turn: both
// operands go from memory into MFMA fragments, nothing is shared but the sums at the
// end.  FP32 operands come in three parts and six products, as in expert_f32.hip.
// What bounds it: the loads' latency, then W's way in; one row of 4096 x 4096 takes 20 us
// in FP32, 9 in bfloat16, 3.3 and 3.7 TB/s of W.
#include "expert_rows.hpp"

namespace sgemm_emu_dev {

namespace {

constexpr int KB = 128, WAVES = 8, NT = 64 * WAVES;

// GATED: a second tile of W holds the up projection's rows of the same outputs.
template <class T, bool GATED, bool LIES>
__global__ __launch_bounds__(NT) void expert_few_kernel(ExpertProduct g)
{
    constexpr int NB = GATED ? 2 : 1, BANDS = sizeof(T) == 4 ? 3 : 1;
    __shared__ __attribute__((aligned(16))) f32x4_t sums[WAVES][NB][64];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const RowTile t = RowTiles<16>(g.offsets, g.n, g.P, (int)g.n + 1, lane).find(workgroup() / g.tiles_n);
    if (t.segment < 0) return;
    const int64_t F = GATED ? g.N / 2 : g.N, n0 = (int64_t)(workgroup() % g.tiles_n) * 16;
    const int here = (int)lmin(t.end - t.row, 16);
    T *const C = (T *)g.C;
    if (t.segment >= g.n) {                                // rows of no expert
        for (int o = threadIdx.x; o < 16 * here; o += NT)
            if (n0 + o % 16 < F) C[(t.row + o / 16) * g.ldc + n0 + o % 16] = Elem<T>::store(0.0f);
        return;
    }
    const T *const W = (const T *)g.B + t.segment * g.bank;
    const int64_t blocks = (g.K + KB - 1) / KB;
    f32x4_t acc[NB][BANDS];
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int q = 0; q < BANDS; ++q) acc[b][q] = f32x4_t{};
    for (int64_t kb = wave; kb < blocks; kb += WAVES) {
        RowBlock<T> x, w[NB];
        x.template load<LIES>((const T *)g.A, g.lda, t.row + (lane & 15), t.end, kb * KB, g.K, lane);
#pragma unroll
        for (int b = 0; b < NB; ++b)
            w[b].template load<LIES>(W + b * F * g.ldb, g.ldb, n0 + (lane & 15), F, kb * KB, g.K, lane);
#pragma unroll
        for (int d = 0; d < 4; ++d) {
            u32x4_t xp[BANDS], wp[BANDS];
            x.parts(d, xp);
#pragma unroll
            for (int b = 0; b < NB; ++b) {
                w[b].parts(d, wp);
                // parts i and j add to band i + j; those beyond the last are left out
#pragma unroll
                for (int i = 0; i < BANDS; ++i)
#pragma unroll
                    for (int j = 0; i + j < BANDS; ++j)
                        acc[b][i + j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                            __builtin_bit_cast(bf16x8_t, wp[j]), __builtin_bit_cast(bf16x8_t, xp[i]), acc[b][i + j], 0, 0, 0);
            }
        }
    }
#pragma unroll
    for (int b = 0; b < NB; ++b) {
        f32x4_t v = acc[b][0];
        if constexpr (BANDS == 3) {
#pragma unroll
            for (int q = 0; q < 4; ++q) v[q] += __builtin_fmaf(acc[b][2][q], 0x1p-16f, acc[b][1][q] * 0x1p-8f);
        }
        sums[wave][b][lane] = v;
    }
    __syncthreads();
    // sums[..][b][l][q]: output 4 (l >> 4) + q, row l & 15
    const T *const bias = g.bias != nullptr ? (const T *)g.bias + t.segment * g.N : nullptr;
    auto total = [&](int b, int n, int m) {
        float v = 0.0f;
#pragma unroll
        for (int i = 0; i < WAVES; ++i) v += sums[i][b][(n >> 2) * 16 + m][n & 3];
        return v;
    };
    for (int o = threadIdx.x; o < 16 * here; o += NT) {
        const int n = o % 16, m = o / 16;
        const int64_t f = n0 + n;
        if (f >= F) continue;
        float v = total(0, n, m);
        if (bias != nullptr) v += Elem<T>::load(bias + f);
        if constexpr (GATED) {
            float u = total(1, n, m);
            if (bias != nullptr) u += Elem<T>::load(bias + F + f);
            if (g.Z != nullptr) {
                float *const z = g.Z + (t.row + m) * g.ldz + f;
                z[0] = v;
                z[g.ldz / 2] = u;
            }
            v = gate_value(g.gate, v) * u;
        }
        C[(t.row + m) * g.ldc + f] = Elem<T>::store(v);
    }
}

template <class T, bool LIES>
void launch(const ExpertProduct &g, dim3 grid, hipStream_t stream)
{
    if (g.gate >= 0) hipLaunchKernelGGL((expert_few_kernel<T, true, LIES>), grid, dim3(NT), 0, stream, g);
    else hipLaunchKernelGGL((expert_few_kernel<T, false, LIES>), grid, dim3(NT), 0, stream, g);
}

int64_t row_tiles(const ExpertProduct &g) { return g.P / 16 + (g.n + 1 < g.P ? g.n + 1 : g.P); }

}  // namespace

// Up to 1024 rows, where this kernel's time for a block of columns is below the tiles':
// hundredths of a us, at least those of one workgroup or tile alone, beyond that in
// proportion to how many a CU has, with the rows evenly among the experts (beyond 256
// rows: tiles as if one expert had all, where they are fewest).  Times on
// 4096 x 4096, here and in 64 x 64 tiles: FP32 1 row 20 and 104 us, 64 rows 73 and 105,
// 128 rows 132 and 108; bfloat16 1 row 9 and 18, 16 rows 11 and 18, 64 rows 32 and 18.
// 512 rows of 128 x 2720: FP32 19 and 70, bfloat16 7 and 13.  bfloat16 rows that do not
// lie in pieces, 1024 x 1001 over 8 experts: 1 row 5 and 13, 128 rows 12 and 17, 256 20 and 17.
bool expert_few(int dtype, const ExpertProduct &g)
{
    if (g.P > 1024 || g.n == 0) return false;
    const bool lies = dtype == kF32 || expert_lies(kForward, g);
    const int64_t with = g.n < g.P ? g.n : g.P, each = (g.P + with - 1) / with, cus = g.num_cus;
    const int64_t here = with * ((each + 15) / 16) * ((g.N + 15) / 16);
    const int64_t rows = g.P <= 256 ? with * ((each + 63) / 64) : (g.P + 63) / 64;
    const int64_t tiles = rows * ((g.N + 63) / 64);
    auto most = [](int64_t a, int64_t b) { return a > b ? a : b; };
    if (dtype == kF32) return 50 * most(cus, here) < most(320 * cus, 270 * tiles);
    if (lies) return 20 * most(cus, here) < most(44 * cus, 68 * tiles);
    return 50 * most(cus, here) < 120 * most(cus, tiles);
}

hipError_t launch_expert_few(int dtype, const ExpertProduct &args, hipStream_t stream)
{
    ExpertProduct g = args;
    g.tiles_n = (int)(((g.gate >= 0 ? g.N / 2 : g.N) + 15) / 16);
    const int64_t blocks = row_tiles(g) * g.tiles_n;
    if (!grid_ok(blocks)) return hipErrorInvalidValue;
    const dim3 grid = grid_of(blocks);
    const bool lies = g.lda % 2 == 0 && g.ldb % 2 == 0 && g.bank % 2 == 0 && aligned(g.A, 4) && aligned(g.B, 4) &&
                      (g.gate < 0 || (g.N / 2 * g.ldb) % 2 == 0);
    if (dtype == kF32) launch<float, true>(g, grid, stream);
    else if (lies) launch<uint16_t, true>(g, grid, stream);
    else launch<uint16_t, false>(g, grid, stream);
    return hipGetLastError();
}

}  // namespace sgemm_emu_dev
