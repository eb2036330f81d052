// gemm.hip -- BF16x9 emulated SGEMM: the split-K reduction, the stream-K and
// small-tile cost models, the native FP32 kernel, and the dispatch of the
// kernels in gemm_kernels.hpp.
#include "gemm_kernels.hpp"

namespace sgemm_emu_dev {

// ---------------------------------------------------------------- split-K reduction

// C = act(sum over K slices of the slices' recombined results + bias), per
// element, adding the slices in slice order.
// Workgroups walk rows, threads walk a row's columns (no per-element division).
__global__ __launch_bounds__(256) void splitk_reduce_kernel(GemmArgs g)
{
    const int64_t plane = g.M * g.ldp;
    for (int64_t r = blockIdx.x; r < g.M; r += gridDim.x) {
        for (int64_t c = threadIdx.x; c < g.N; c += blockDim.x) {
            const float *p = g.partials + r * g.ldp + c;
            float v = p[0];
            for (int sl = 1; sl < g.splits; ++sl) v += p[(int64_t)sl * plane];
            v = v + (g.bias ? g.bias[c] : -0.0f);
            if (g.act == 1) v = gelu_erf(v);
            g.C[r * g.ldc + c] = v;
        }
    }
}

// Domains of a stream-K grid of G workgroups over T tiles of ppt K pairs.
// Workgroup w runs on XCD w % 8 (the dispatcher deals workgroups to the XCDs
// in turn), so 8 domains, domain d holding workgroups w = d (mod 8) and tile
// block d of the stream-K order, keep each block's A and B panels in one L2.
// Taken when every workgroup still gets two K pairs and the largest block is
// within 10 % of an even share of the tiles; otherwise one domain.
int64_t streamk_domains(int64_t T, int64_t ppt, int64_t G)
{
    if (G % 8 != 0 || T < 8) return 1;
    if (T / 8 * ppt < 2 * (G / 8)) return 1;
    if ((T + 7) / 8 * 80 > T * 11) return 1;
    return 8;
}

// Stream-K against the persistent kernel, in K-pair times per CU: the
// persistent kernel needs ceil(T / G) whole tiles of ppt pairs; stream-K needs
// ceil(T ppt / G) pairs plus the publication, wait and sum of the cut tiles,
// which measured about kStreamkFixPairs pair times (6144 x 256 x 1024,
// 3072 x 1536 x 1024, 8192 x 640 x 1024, 6144 x 768 x 512, 2560^2 x 1024 and
// 4096 x 2048 x 512 on 256 CUs: stream-K 21-24 % faster on grids of 1.1-1.3
// waves of tiles with K = 1024, even at 1.56 waves, 11 % slower at 2 full
// waves).  Stream-K is taken where the model expects it 10 % faster.
constexpr int64_t kStreamkFixPairs = 6;
constexpr int64_t kStreamkMaxPieces = 8;               // per tile: the last piece adds the others' slots one by one

int gemm_streamk_grid(int64_t M, int64_t N, int64_t K, int num_cus)
{
#ifdef SGEMM_EMU_SERIAL_LDS
    (void)M; (void)N; (void)K; (void)num_cus;
    return 0;                                          // the debug build has no stream-K
#endif
    const int64_t tiles = ((M + 127) / 128) * ((N + 127) / 128);
    if (K % (2 * BK) != 0 || tiles == 0) return 0;
    const int64_t ppt = K / (2 * BK), units = tiles * ppt;
    const int64_t G0 = num_cus > 8 ? num_cus & ~7 : 8;
    int64_t G = G0;
    if (units < 2 * G) G = units / 2;                  // at least two K pairs per workgroup
    if (G > kStreamkMaxPieces * tiles) G = kStreamkMaxPieces * tiles;
    if (G < 2) return 0;
    const int64_t t_persistent = (tiles + G0 - 1) / G0 * ppt;
    const int64_t t_streamk = (units + G - 1) / G + kStreamkFixPairs;
    if (t_streamk * 10 >= t_persistent * 9) return 0;
    if (units * G >= ((int64_t)1 << 32)) return 0;     // the kernel's index arithmetic is 32-bit
    return (int)G;
}

int gemm_streamk_pieces(int64_t M, int64_t N, int64_t K, int grid)
{
    if (grid <= 0) return 1;
    const int64_t tiles = ((M + 127) / 128) * ((N + 127) / 128), ppt = K / (2 * BK);
    const int64_t D = streamk_domains(tiles, ppt, grid), G = grid / D;
    int64_t most = 1;
    for (int64_t d = 0; d < D; ++d) {
        const int64_t Td = (d + 1) * tiles / D - d * tiles / D, P = Td * ppt;
        for (int64_t t = 0; t < Td; ++t) {
            const int64_t first = ((t * ppt + 1) * G - 1) / P, last = (((t + 1) * ppt) * G - 1) / P;
            if (last - first + 1 > most) most = last - first + 1;
        }
    }
    return (int)most;
}

// FP32 B on a partly filled grid: the one-pass kernel on 64 x 64 tiles (B
// split inside each tile, nothing in a workspace, LDS for two workgroups per
// CU) against what 128 x 128 tiles would run -- one pass per tile (the kernel
// that splits B itself, or the N x K plane kernel after a split of B), or,
// where `streamk` allows it, stream-K on split planes.  Costs in K-pair times
// of a 128 x 128 tile on one CU, in twentieths: a 64 x 64 tile's K pair
// measured half of that on a CU of its own and 0.65 beside a second one
// (512^3, 768^3, 1024^3, 1024 x 1024 x 512, 2048 x 512 x 512,
// 1280 / 1536 / 2048 x 1024 x 1024, 4096 x 512 x 1024, 6144 x 256 x 1024 and
// 512 x 512 x 4096 on 256 CUs); stream-K as in gemm_streamk_grid.  Taken where
// the model expects the 64 x 64 tiles 10 % faster: measured 7-90 % faster
// there, and where it declines (256^2 x 1024, 512^2 x 2048 and x 4096,
// 1024^2 x 2048, 2560 x 1024 x 512, 3072 x 1024 x 1024, 3072 x 1536 x 1024)
// the other path was 3-150 % faster.  Four 64 x 64 tiles cost 1.3 times one
// 128 x 128 tile once the grid fills the CUs, so full grids never take them.
bool gemm_tile64_pays(int64_t M, int64_t N, int64_t K, int num_cus, bool streamk)
{
    const int64_t kpad = (K + 2 * BK - 1) / (2 * BK) * (2 * BK), ppt = kpad / (2 * BK);
    const int64_t tiles = ((M + 127) / 128) * ((N + 127) / 128);
    const int64_t G0 = num_cus > 8 ? num_cus & ~7 : 8;
    int64_t t_other = (tiles + G0 - 1) / G0 * ppt;
    const int G = streamk ? gemm_streamk_grid(M, N, kpad, num_cus) : 0;
    if (G > 0) t_other = (tiles * ppt + G - 1) / G + kStreamkFixPairs;
    const int64_t tiles64 = ((M + 63) / 64) * ((N + 63) / 64);
    const int64_t t_tile64 = ppt * (tiles64 <= G0 ? 10 : 13 * ((tiles64 + 2 * G0 - 1) / (2 * G0)));
    return t_tile64 * 10 <= 20 * t_other * 9;
}

// ---------------------------------------------------------------- native FP32 (performant strategy)
//
// The pages' "performant" strategy uses the emulation only where it expects
// a speed-up over the platform's native FP32 GEMM (NVIDIA blog, section
// "BF16x9 on NVIDIA Blackwell GPUs", Fig. 4; discuss.pytorch.kr summary,
// "PyTorch에서 직접 써 보려면").  This is the library's own native path: the
// FP32 matrix instruction v_mfma_f32_32x32x2_f32, one FP32 accumulator per
// output, no split.
//
// One workgroup per (tile, K slice); waves as in Cfg, each (MI x 32) x (NI x 32)
// of accumulators.  K advances in steps of NBK k (32, or 16 with element
// loads), double-buffered in LDS and loaded NLA steps ahead into registers:
//   * A rows hold NBK k values plus 4 of padding (144 or 80 bytes): 16
//     consecutive rows read with 128-bit loads touch 64 distinct banks;
//   * B rows (one k each) hold the tile's BN columns plus 4 of padding, so
//     the two half-waves reading k and k + 8 land on disjoint banks.
// Within each 16 k of a step, half-wave h (lanes 32h..32h+31) feeds
// k = 8h + kk to the kk-th MFMA: the instruction's two k rows come from k and
// k + 8, so each lane reads its eight A values of the 16 with two 128-bit
// loads.  Every k < K is multiplied in exactly once, in an order the bound
// allows.

// K per step and register stages: with 128-bit loads 32 k and two stages
// ahead (against 16 k and four: 768^3 37.4 -> 43.0 TFLOP/s, 1024^3 68.0 ->
// 77.3, 1024 x 1024 x 512 59.4 -> 66.9, 6144 x 256 x 1024 71.9 -> 76.6, the
// larger grids unchanged); with element loads 16 k and four stages (32 k
// measured 10.2 -> 8.0 TFLOP/s on 333 x 444 x 555).
template <bool VEC>
struct NativeSteps {
    static constexpr int NBK = VEC ? 32 : 16;   // k per step
    static constexpr int NLA = VEC ? 2 : 4;     // steps loaded ahead (register stages)
};

template <class C, int NBK>
struct NativeLayout {
    static constexpr int NAP = NBK + 4;                   // A row pitch in LDS (floats)
    static constexpr int BNP = C::BN + 4;                 // B row pitch in LDS (floats)
    static constexpr int A_FLOATS = C::BM * NAP;
    static constexpr int B_FLOATS = NBK * BNP;
    static constexpr int STAGE = A_FLOATS + B_FLOATS;
    static constexpr int A_VECS = C::BM * (NBK / 4) / C::NT;   // 16-byte A chunks per thread and step
    static constexpr int B_VECS = NBK * (C::BN / 4) / C::NT;   // 16-byte B chunks per thread and step
    static_assert(C::BM * (NBK / 4) % C::NT == 0 && NBK * (C::BN / 4) % C::NT == 0, "loader mapping");
};

template <class C, int NBK>
struct NativeStage {
    float a[NativeLayout<C, NBK>::A_VECS][4];
    float b[NativeLayout<C, NBK>::B_VECS][4];
};

// Thread -> A chunk (row, 4-wide k group): 16 consecutive lanes take 16 rows of
// one k group (conflict-free 128-bit LDS writes at the 80-byte pitch); a wave
// covers 16 rows x 4 k groups, the waves run through the tile's row blocks.
template <class C>
__device__ __forceinline__ void native_a_chunk(int q, int &row, int &kg)
{
    constexpr int ROW_BLOCKS = C::BM / 16;
    const int lane = q & 63, blk = q >> 6;
    row = (blk % ROW_BLOCKS) * 16 + (lane & 15);
    kg = (lane >> 4) + 4 * (blk / ROW_BLOCKS);
}

// Load one step (k0 .. k0 + 15) of A and B into registers.  VEC: 128-bit
// loads (16-byte aligned operands, leading dimensions and K / N multiples of
// 4), else one dword at a time.  A past K reads the next row's values and is
// masked by the caller; B rows past K and A, B beyond the operands read zero
// or values whose outputs are never stored.
template <class C, bool VEC, int NBK>
__device__ __forceinline__ void native_load(NativeStage<C, NBK> &st, const GemmArgs &g, int64_t m0, int64_t n0,
                                            int64_t k0)
{
    using L = NativeLayout<C, NBK>;
    const int tid = threadIdx.x;
    {
        const int64_t rows = lmin((int64_t)C::BM, g.M - m0);
        const rsrc_t ra = make_rsrc(g.A + m0 * g.lda + k0, ((rows - 1) * g.lda + (g.K - k0)) * 4);
#pragma unroll
        for (int c = 0; c < L::A_VECS; ++c) {
            int row, kg;
            native_a_chunk<C>(c * C::NT + tid, row, kg);
            const int64_t r = lmin((int64_t)row, rows - 1);
            const uint32_t off = (uint32_t)((r * g.lda + kg * 4) * 4);
            if (VEC) {
                const u32x4_t v = bload_u32x4(ra, off, 0);
#pragma unroll
                for (int e = 0; e < 4; ++e) st.a[c][e] = __uint_as_float(v[e]);
            } else {
#pragma unroll
                for (int e = 0; e < 4; ++e) st.a[c][e] = bload_f32(ra, off + 4 * e, 0);
            }
        }
    }
    {
        // base at row k0; the descriptor ends at element (K-1, N-1)
        const rsrc_t rb = make_rsrc(g.B + k0 * g.ldb, ((g.K - 1 - k0) * g.ldb + g.N) * 4);
#pragma unroll
        for (int c = 0; c < L::B_VECS; ++c) {
            const int q = c * C::NT + tid, col = (q % (C::BN / 4)) * 4, k = q / (C::BN / 4);
            const int64_t n = lmin(n0 + col, (g.N - 1) & ~(int64_t)3);
            const uint32_t off = (uint32_t)(((int64_t)k * g.ldb + (VEC ? n : n0 + col)) * 4);
            if (VEC) {
                const u32x4_t v = bload_u32x4(rb, off, 0);
#pragma unroll
                for (int e = 0; e < 4; ++e) st.b[c][e] = __uint_as_float(v[e]);
            } else {
#pragma unroll
                for (int e = 0; e < 4; ++e) st.b[c][e] = bload_f32(rb, off + 4 * e, 0);
            }
        }
    }
}

template <class C, int NBK>
__device__ __forceinline__ void native_store(const NativeStage<C, NBK> &st, float *buf, int64_t kvalid)
{
    using L = NativeLayout<C, NBK>;
    const int tid = threadIdx.x;
#pragma unroll
    for (int c = 0; c < L::A_VECS; ++c) {
        int row, kg;
        native_a_chunk<C>(c * C::NT + tid, row, kg);
        float x[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) x[e] = (kg * 4 + e < kvalid) ? st.a[c][e] : 0.0f;
        *reinterpret_cast<u32x4_t *>(buf + row * L::NAP + kg * 4) =
            u32x4_t{__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3])};
    }
#pragma unroll
    for (int c = 0; c < L::B_VECS; ++c) {
        const int q = c * C::NT + tid, col = (q % (C::BN / 4)) * 4, k = q / (C::BN / 4);
        *reinterpret_cast<u32x4_t *>(buf + L::A_FLOATS + k * L::BNP + col) =
            u32x4_t{__float_as_uint(st.b[c][0]), __float_as_uint(st.b[c][1]), __float_as_uint(st.b[c][2]),
                    __float_as_uint(st.b[c][3])};
    }
}

template <class C, int NBK>
__device__ __forceinline__ void native_step(Acc<C, 1> &acc, const float *buf, int wm, int wn, int lane)
{
    using L = NativeLayout<C, NBK>;
    const int h = lane >> 5, r = lane & 31;
#pragma unroll
    for (int kb = 0; kb < NBK; kb += 16) {
        float a[C::MI][8];
#pragma unroll
        for (int i = 0; i < C::MI; ++i) {
            const float *p = buf + (wm * C::WTM + i * 32 + r) * L::NAP + kb + 8 * h;
            const u32x4_t v0 = *reinterpret_cast<const u32x4_t *>(p);
            const u32x4_t v1 = *reinterpret_cast<const u32x4_t *>(p + 4);
#pragma unroll
            for (int e = 0; e < 4; ++e) { a[i][e] = __uint_as_float(v0[e]); a[i][4 + e] = __uint_as_float(v1[e]); }
        }
#pragma unroll
        for (int kk = 0; kk < 8; ++kk) {
            float b[C::NI];
#pragma unroll
            for (int j = 0; j < C::NI; ++j)
                b[j] = buf[L::A_FLOATS + (kb + 8 * h + kk) * L::BNP + wn * C::WTN + j * 32 + r];
#pragma unroll
            for (int i = 0; i < C::MI; ++i)
#pragma unroll
                for (int j = 0; j < C::NI; ++j)
                    acc.v[i][j][0] = __builtin_amdgcn_mfma_f32_32x32x2f32(a[i][kk], b[j], acc.v[i][j][0], 0, 0, 0);
        }
    }
}

template <class C, bool VEC>
__global__ __launch_bounds__(C::NT, 2) void gemm_f32_native_kernel(GemmArgs g)
{
    constexpr int NBK = NativeSteps<VEC>::NBK, NLA = NativeSteps<VEC>::NLA;
    using L = NativeLayout<C, NBK>;
    __shared__ __attribute__((aligned(16))) float lds[2 * L::STAGE];
    int tm, tn;
    tile_of_index((int)blockIdx.x, (int)gridDim.x, g.tiles_m, g.tiles_n, g.group_m, tm, tn);
    const int64_t m0 = (int64_t)tm * C::BM, n0 = (int64_t)tn * C::BN;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int wm = wave / C::WAVES_N, wn = wave % C::WAVES_N;
    // K slice of this workgroup (split-K): steps [s0, s1)
    const int64_t nsteps = (g.K + NBK - 1) / NBK;
    const int64_t per = (nsteps + g.splits - 1) / g.splits;
    const int64_t s0 = (int64_t)blockIdx.y * per, s1 = lmin(nsteps, s0 + per);

    Acc<C, 1> acc;
#pragma unroll
    for (int i = 0; i < C::MI; ++i)
#pragma unroll
        for (int j = 0; j < C::NI; ++j) acc.v[i][j][0] = f32x16_t{};

    if (s0 < s1) {
        // A ring of NLA register stages: the loads of step t + NLA go out while
        // step t is computed, so each step's loads have NLA - 1 steps of MFMA
        // work to arrive before they are written to LDS (one step of lead
        // leaves these short K steps waiting on memory latency).
        // The loads and LDS writes are unconditional, so every wait for a
        // stage counts only the NLA - 1 stages loaded after it: a load past
        // the slice re-reads its last step and is never stored for use, and
        // the LDS write after the last step goes to a buffer no step reads.
        NativeStage<C, NBK> st[NLA];
#pragma unroll
        for (int r = 0; r < NLA; ++r)
            native_load<C, VEC, NBK>(st[r], g, m0, n0, lmin(s0 + r, s1 - 1) * NBK);
        native_store<C, NBK>(st[0], lds, g.K - s0 * NBK);
        __syncthreads();
        for (int64_t s = s0; s < s1; s += NLA) {
#pragma unroll
            for (int r = 0; r < NLA; ++r) {
                const int64_t t = s + r;          // the step computed now; its data is in LDS
                if (t >= s1) break;
                const float *cur = lds + ((t - s0) & 1) * L::STAGE;
                float *nxt = lds + ((t - s0 + 1) & 1) * L::STAGE;
                native_load<C, VEC, NBK>(st[r], g, m0, n0, lmin(t + NLA, s1 - 1) * NBK);
                native_step<C, NBK>(acc, cur, wm, wn, lane);
                native_store<C, NBK>(st[(r + 1) % NLA], nxt, g.K - (t + 1) * NBK);
                __syncthreads();
            }
        }
    }
    float bias[C::NI];
    load_bias<C>(bias, g, n0, wn, lane);
    if (g.splits > 1) store_c_act<C, 1, -1>(acc, bias, g, m0, n0, wm, wn, lane, (int)blockIdx.y);
    else store_c<C, 1>(acc, bias, g, m0, n0, wm, wn, lane);
}

using CfgN128 = Cfg<2, 2, 64, 64>;    // 4 waves, 128 x 128 tile
using CfgN64 = Cfg<2, 2, 32, 32>;     // 4 waves, 64 x 64 tile

bool native_vec(const float *A, int64_t lda, const float *B, int64_t ldb, int64_t K, int64_t N)
{
    return aligned(A, 16) && aligned(B, 16) && lda % 4 == 0 && ldb % 4 == 0 && K % 4 == 0 && N % 4 == 0;
}

template <class C>
static hipError_t launch_native_cfg(const GemmArgs &args, int splits, hipStream_t stream)
{
    GemmArgs g = args;
    g.tiles_m = (int)((g.M + C::BM - 1) / C::BM);
    g.tiles_n = (int)((g.N + C::BN - 1) / C::BN);
    g.group_m = group_rows(g.tiles_n, g.num_cus);
    g.splits = splits;
    const bool vec = native_vec(g.A, g.lda, g.B, g.ldb, g.K, g.N);
    const dim3 grid((unsigned)((int64_t)g.tiles_m * g.tiles_n), (unsigned)splits), block(C::NT);
    GemmArgs gk = g;
    if (splits > 1) gk.done = nullptr;          // the reduction is the last kernel
    if (vec) launch_last(gemm_f32_native_kernel<C, true>, grid, block, stream, gk);
    else launch_last(gemm_f32_native_kernel<C, false>, grid, block, stream, gk);
    if (splits > 1) {
        const int64_t blocks = g.M < (int64_t)g.num_cus * 8 ? g.M : (int64_t)g.num_cus * 8;   // rows
        launch_last(splitk_reduce_kernel, dim3((unsigned)blocks), dim3(256), stream, g);
    }
    return hipGetLastError();
}

NativePlan native_plan(int64_t M, int64_t N, int64_t K, int num_cus, bool vec)
{
    const int NBK = vec ? NativeSteps<true>::NBK : NativeSteps<false>::NBK;
    NativePlan p{};
    const int64_t t128 = ((M + 127) / 128) * ((N + 127) / 128);
    if (t128 >= num_cus) {
        p.tile = 128;
        p.splits = 1;
        return p;
    }
    const int64_t t64 = ((M + 63) / 64) * ((N + 63) / 64);
    p.tile = 64;
    p.splits = 1;
    // small grids: K slices of at least 8 steps until about one workgroup per
    // CU (the slices' sum costs a second launch), and on to two per CU where a
    // slice would still be longer than 64 steps.  Measured against two per CU
    // throughout: 1024 x 1024 x 512 45.7 -> 62.2 TFLOP/s, 2048 x 512 x 512
    // 45.2 -> 63.5, 1024^3 65.3 -> 71.0, 1024 x 512 x 4096 unchanged at 82.6
    // (it keeps four slices), with 16-k steps; the same counts of the 32-k
    // steps are what the figures above NativeSteps were measured with.
    const int64_t nsteps = (K + NBK - 1) / NBK;
    auto grow = [&](int64_t per_cu) {
        while (p.splits < 16 && t64 * (p.splits + 1) <= per_cu * (int64_t)num_cus && nsteps / (p.splits + 1) >= 8)
            ++p.splits;
    };
    grow(1);
    if (nsteps / p.splits > 64) grow(2);
    return p;
}

hipError_t launch_native(const GemmArgs &args, const NativePlan &plan, hipStream_t stream)
{
    if (plan.splits > 1 && args.partials == nullptr) return hipErrorInvalidValue;
    if (plan.tile == 128) return launch_native_cfg<CfgN128>(args, plan.splits, stream);
    return launch_native_cfg<CfgN64>(args, plan.splits, stream);
}

// ---------------------------------------------------------------- K == 0

__global__ __launch_bounds__(256) void zero_kernel(float *__restrict__ C, int64_t ldc, int64_t M, int64_t N,
                                                   const float *__restrict__ bias, int act)
{
    for (int64_t r = blockIdx.x; r < M; r += gridDim.x) {
        for (int64_t c = threadIdx.x; c < N; c += blockDim.x) {
            float v = bias ? 0.0f + bias[c] : 0.0f;
            if (act == 1) v = gelu_erf(v);
            C[r * ldc + c] = v;
        }
    }
}

hipError_t launch_zero(int64_t M, int64_t N, float *C, int64_t ldc, const float *bias, int act, int num_cus,
                       hipStream_t stream)
{
    const int64_t blocks = M < (int64_t)num_cus * 8 ? M : (int64_t)num_cus * 8;   // rows
    hipLaunchKernelGGL(zero_kernel, dim3((unsigned)blocks), dim3(256), 0, stream, C, ldc, M, N, bias, act);
    return hipGetLastError();
}

// ---------------------------------------------------------------- dispatch

// Tile-rows per group.  An XCD runs about num_cus / 8 consecutive tiles at
// once.  A narrow tile grid (at least 4 whole tile-rows in that window) runs
// row by row (groups of one row), so the column tiles that read an A row
// panel are neighbours and run together; wider grids use groups of 8 rows,
// which share both A and B panels.
int group_rows(int tiles_n, int num_cus)
{
    const int per_xcd = num_cus >= 8 ? num_cus / 8 : 1;
    return tiles_n * 4 <= per_xcd ? 1 : 8;
}

template <class C, int NB, bool AVEC, int BSRC, bool RNE>
static void launch_cfg_b(const GemmArgs &g, int bvec, hipStream_t stream)
{
    const dim3 grid((unsigned)((int64_t)g.tiles_m * g.tiles_n)), block(C::NT);
    if constexpr (BSRC == B_FP32) {
        // FP32 B loads element by element; only A has a vector path
        hipLaunchKernelGGL((gemm_bf16x9_kernel<C, NB, AVEC, BSRC, 0, RNE>), grid, block, 0, stream, g);
    } else {
        if (bvec == 1) hipLaunchKernelGGL((gemm_bf16x9_kernel<C, NB, AVEC, BSRC, 1, RNE>), grid, block, 0, stream, g);
        else if (BSRC == B_PLANES_NK && bvec == 2)
            hipLaunchKernelGGL((gemm_bf16x9_kernel<C, NB, AVEC, BSRC, BSRC == B_PLANES_NK ? 2 : 0, RNE>), grid, block, 0,
                               stream, g);
        else hipLaunchKernelGGL((gemm_bf16x9_kernel<C, NB, AVEC, BSRC, 0, RNE>), grid, block, 0, stream, g);
    }
}

// bvec: B's load width -- 1: 128-bit (N x K planes) or 32-bit (K x N planes);
// 2: 32-bit for N x K planes; 0: element loads.
template <class C, int NB, int BSRC, bool RNE>
static void launch_cfg(const GemmArgs &g, bool avec, int bvec, hipStream_t stream)
{
    if (avec) launch_cfg_b<C, NB, true, BSRC, RNE>(g, bvec, stream);
    else launch_cfg_b<C, NB, false, BSRC, RNE>(g, bvec, stream);
}

template <class C, int BSRC, bool RNE = false>
static void launch_nb(const GemmArgs &g, int nbands, bool avec, int bvec, hipStream_t stream)
{
    switch (nbands) {
    case 1: launch_cfg<C, 1, BSRC, RNE>(g, avec, bvec, stream); break;
    case 2: launch_cfg<C, 2, BSRC, RNE>(g, avec, bvec, stream); break;
    case 3: launch_cfg<C, 3, BSRC, RNE>(g, avec, bvec, stream); break;
    case 4: launch_cfg<C, 4, BSRC, RNE>(g, avec, bvec, stream); break;
    default: launch_cfg<C, 5, BSRC, RNE>(g, avec, bvec, stream); break;
    }
}

template <class C, int NB, bool RNE, bool KTAIL>
static void launch_dma_nb(const GemmArgs &g, bool avec, hipStream_t stream)
{
    // One resident workgroup per CU (LDS-limited); a multiple of 8 keeps each
    // workgroup on one XCD for all of its tiles.
    const dim3 block(C::NT);
#ifdef SGEMM_EMU_SERIAL_LDS
    {
        const dim3 grid((unsigned)((int64_t)g.tiles_m * g.tiles_n));
        if (avec) launch_last(gemm_bf16x9_serial_kernel<C, NB, true, RNE, KTAIL>, grid, block, stream, g);
        else launch_last(gemm_bf16x9_serial_kernel<C, NB, false, RNE, KTAIL>, grid, block, stream, g);
        return;
    }
#endif
    if (g.sk_grid > 0) {
        // small tile grid: stream-K over sk_grid workgroups
        GemmArgs s = g;
        s.sk_domains = streamk_domains((int64_t)g.tiles_m * g.tiles_n, g.K / (2 * BK), g.sk_grid);
        s.group_m = kStreamkGroupRows;
        const dim3 grid((unsigned)g.sk_grid);
        if (avec) launch_last(gemm_bf16x9_streamk_kernel<C, NB, true, RNE, KTAIL>, grid, block, stream, s);
        else launch_last(gemm_bf16x9_streamk_kernel<C, NB, false, RNE, KTAIL>, grid, block, stream, s);
        return;
    }
    const int64_t units = (int64_t)g.tiles_m * g.tiles_n;
    int64_t slots = (int64_t)(g.num_cus > 8 ? g.num_cus & ~7 : 8);
    const dim3 grid((unsigned)(units < slots ? units : slots));
    if (avec) launch_last(gemm_bf16x9_dma_kernel<C, NB, true, RNE, KTAIL>, grid, block, stream, g);
    else launch_last(gemm_bf16x9_dma_kernel<C, NB, false, RNE, KTAIL>, grid, block, stream, g);
}

template <class C, bool RNE, bool KTAIL>
static hipError_t launch_dma(const GemmArgs &args, int nbands, hipStream_t stream)
{
    GemmArgs g = args;
    g.tiles_m = (int)((g.M + C::BM - 1) / C::BM);
    g.tiles_n = (int)((g.N + C::BN - 1) / C::BN);
    g.group_m = group_rows(g.tiles_n, g.num_cus);
    // no 128-bit A load may straddle the end of A's rows (see launch_with)
    const bool avec = aligned(g.A, 16) && (g.lda % 4 == 0) && (g.ka % 4 == 0);
    switch (nbands) {
    case 1: launch_dma_nb<C, 1, RNE, KTAIL>(g, avec, stream); break;
    case 2: launch_dma_nb<C, 2, RNE, KTAIL>(g, avec, stream); break;
    case 3: launch_dma_nb<C, 3, RNE, KTAIL>(g, avec, stream); break;
    case 4: launch_dma_nb<C, 4, RNE, KTAIL>(g, avec, stream); break;
    default: launch_dma_nb<C, 5, RNE, KTAIL>(g, avec, stream); break;
    }
    return hipGetLastError();
}

template <class C, int NB>
static void launch_planes_nb(const GemmArgs &g, hipStream_t stream)
{
    const int64_t units = (int64_t)g.tiles_m * g.tiles_n;
    int64_t slots = (int64_t)(g.num_cus > 8 ? g.num_cus & ~7 : 8);
    const dim3 grid((unsigned)(units < slots ? units : slots)), block(C::NT);
    launch_last(gemm_bf16x9_planes_kernel<C, NB>, grid, block, stream, g);
}

hipError_t launch_gemm_planes(const GemmArgs &args, int nbands, hipStream_t stream)
{
    using C = Cfg8S;
    if (args.K % (2 * BK) != 0 || args.lda % 8 != 0 || args.ldb % 8 != 0 || !aligned(args.A0, 16) ||
        !aligned(args.A1, 16) || !aligned(args.A2, 16) || !aligned(args.B0, 16) || !aligned(args.B1, 16) ||
        !aligned(args.B2, 16))
        return hipErrorInvalidValue;
    GemmArgs g = args;
    g.tiles_m = (int)((g.M + C::BM - 1) / C::BM);
    g.tiles_n = (int)((g.N + C::BN - 1) / C::BN);
    g.group_m = group_rows(g.tiles_n, g.num_cus);
    switch (nbands) {
    case 1: launch_planes_nb<C, 1>(g, stream); break;
    case 2: launch_planes_nb<C, 2>(g, stream); break;
    case 3: launch_planes_nb<C, 3>(g, stream); break;
    case 4: launch_planes_nb<C, 4>(g, stream); break;
    default: launch_planes_nb<C, 5>(g, stream); break;
    }
    return hipGetLastError();
}

template <class C>
static GemmArgs tiled(const GemmArgs &args)
{
    GemmArgs g = args;
    g.tiles_m = (int)((g.M + C::BM - 1) / C::BM);
    g.tiles_n = (int)((g.N + C::BN - 1) / C::BN);
    g.group_m = group_rows(g.tiles_n, g.num_cus);
    return g;
}

// 128-bit loads along k need every 4 (A) or 8 (N x K planes) elements to lie
// entirely below or entirely above K, so that no vector load straddles the
// end of its descriptor's range.
static bool a_vec(const GemmArgs &g)
{
    return aligned(g.A, 16) && (g.lda % 4 == 0) && (g.K % 4 == 0);
}

// Load width of N x K planes: 128-bit loads need every 8 elements of a row to
// lie entirely below or above K (16-byte aligned planes, ldb and K multiples of
// 8); 32-bit loads need pairs (4-byte aligned planes, ldb and K even); else
// element loads.
static int nk_bvec(const GemmArgs &g)
{
    if (aligned(g.B0, 16) && aligned(g.B1, 16) && aligned(g.B2, 16) && g.ldb % 8 == 0 && g.K % 8 == 0) return 1;
    if (aligned(g.B0, 4) && aligned(g.B1, 4) && aligned(g.B2, 4) && g.ldb % 2 == 0 && g.K % 2 == 0) return 2;
    return 0;
}

// Load width of K x N planes: 32-bit loads (a column pair) need 4-byte
// aligned planes and ldb, N even; else element loads.
static int kn_bvec(const GemmArgs &g)
{
    return aligned(g.B0, 4) && aligned(g.B1, 4) && aligned(g.B2, 4) && g.ldb % 2 == 0 && g.N % 2 == 0 ? 1 : 0;
}

template <class C>
static hipError_t launch_with(const GemmArgs &args, int nbands, BSource bsrc, hipStream_t stream, bool rne)
{
    const GemmArgs g = tiled<C>(args);
    const bool avec = a_vec(g);
    int bvec = 0;
    if (bsrc == B_PLANES_NK)
        bvec = nk_bvec(g);
    else if (bsrc == B_PLANES_KN)
        bvec = kn_bvec(g);
    if (rne) {
        if (bsrc != B_FP32) return hipErrorInvalidValue;
        launch_nb<C, B_FP32, true>(g, nbands, avec, false, stream);
        return hipGetLastError();
    }
    switch (bsrc) {
    case B_FP32: launch_nb<C, B_FP32>(g, nbands, avec, false, stream); break;
    case B_PLANES_NK: launch_nb<C, B_PLANES_NK>(g, nbands, avec, bvec, stream); break;
    default: launch_nb<C, B_PLANES_KN>(g, nbands, avec, bvec, stream); break;
    }
    return hipGetLastError();
}

template <class C>
static hipError_t launch_tile64_cfg(const GemmArgs &args, int nbands, BSource bsrc, hipStream_t stream, bool rne)
{
    const GemmArgs g = tiled<C>(args);
    if (bsrc == B_PLANES_NK) {
        if (rne) return hipErrorInvalidValue;
        launch_nb<C, B_PLANES_NK>(g, nbands, a_vec(g), nk_bvec(g), stream);
    } else if (bsrc == B_PLANES_KN) {
        if (rne) return hipErrorInvalidValue;
        launch_nb<C, B_PLANES_KN>(g, nbands, a_vec(g), kn_bvec(g), stream);
    } else if (bsrc == B_FP32) {
        if (rne) launch_nb<C, B_FP32, true>(g, nbands, a_vec(g), false, stream);
        else launch_nb<C, B_FP32>(g, nbands, a_vec(g), false, stream);
    } else {
        return hipErrorInvalidValue;
    }
    return hipGetLastError();
}

// Where every CU holds at most one 64 x 64 tile, the split's arithmetic spread
// two VALU instructions per MFMA measured faster than four (1024^3 67.7 -> 72.1
// TFLOP/s on FP32 B, 1024 x 1024 x 512 64.2 -> 68.1, 768^3 37.1 -> 39.2; N x K
// and K x N planes up to 4 % faster); with two tiles per CU four stay faster
// (6144 x 256 x 1024 88.1 against 86.5, 1200 x 1300 x 900 80.5 against 77.3).
// Scheduling only: the same bits.
hipError_t launch_gemm_tile64(const GemmArgs &args, int nbands, BSource bsrc, hipStream_t stream, bool rne)
{
    const int64_t tiles64 = ((args.M + 63) / 64) * ((args.N + 63) / 64);
    const int64_t G0 = args.num_cus > 8 ? args.num_cus & ~7 : 8;
    if (tiles64 <= G0) return launch_tile64_cfg<Cfg64S1>(args, nbands, bsrc, stream, rne);
    return launch_tile64_cfg<Cfg64S>(args, nbands, bsrc, stream, rne);
}

bool gemm_uses_dma(int64_t K, int64_t ldb, const void *B0, const void *B1, const void *B2)
{
    return K % (2 * BK) == 0 && ldb % 8 == 0 && aligned(B0, 16) && aligned(B1, 16) && aligned(B2, 16);
}

// Configuration per B source, chosen by measurement on MI355X: the explicit
// MFMA / split interleaving pays off where the kernel splits FP32 B or copies
// N x K planes; with K x N planes the compiler's own schedule is faster.
bool launch_done_attached(const GemmArgs &args, BSource bsrc)
{
    return bsrc == B_PLANES_NK && gemm_uses_dma(args.K, args.ldb, args.B0, args.B1, args.B2);
}

hipError_t launch_gemm(const GemmArgs &args, int nbands, BSource bsrc, hipStream_t stream, bool rne)
{
    if (bsrc == B_PLANES_KN) return launch_with<Cfg8>(args, nbands, bsrc, stream, rne);
    if (bsrc == B_PLANES_NK && gemm_uses_dma(args.K, args.ldb, args.B0, args.B1, args.B2)) {
        // A K tail (only with B planes zero-padded to the kernel's K) masks A past its K
        if (args.ka != args.K) {
            if (rne) return hipErrorInvalidValue;
            return launch_dma<Cfg8S, false, true>(args, nbands, stream);
        }
        return rne ? launch_dma<Cfg8S, true, false>(args, nbands, stream)
                   : launch_dma<Cfg8S, false, false>(args, nbands, stream);
    }
    return launch_with<Cfg8S>(args, nbands, bsrc, stream, rne);
}

}  // namespace sgemm_emu_dev
