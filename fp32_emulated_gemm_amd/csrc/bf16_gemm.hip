// bf16_gemm.hip -- bfloat16 products C = A B^T on the BF16 matrix cores, with
// the gated product or the low-rank adapters' part in the epilogue.
//
// A bfloat16 value is its own first component: one product takes the place of
// the nine of the FP32 emulation, accumulated in FP32 and rounded once.
//
// One workgroup per BM x BN output tile.  K advances in steps of 32; both
// operands' tiles of a step (64-byte rows, the 16-byte slot of k group kg of
// row r at slot kg ^ ((r >> 2) & 3), which keeps the 128-bit fragment reads of
// 16 consecutive rows on distinct banks) are copied global -> LDS by buffer
// loads with LDS destination, three steps ahead, into a ring of four buffers.
// One LDS-only barrier per step: the copies of step kt + 3 overwrite the buffer
// of step kt - 1, whose last fragments every wave read before the barrier of
// step kt - 1.  After a step's barrier the next step's first fragments are
// read while the step's last MFMAs run.
//
// The MFMAs take B's rows as their first operand, so a lane's accumulator
// registers run along N for one row of C (its column in the MFMA's result):
// gate and up rows of a gated product are dealt to the tile in alternating
// blocks of 16, which puts act(gate) and up of one output into one lane, and
// the adapters' part of the epilogue selects its rows per lane.
// The result goes through LDS (the ring's space) and leaves in 128-bit stores.
#include "ops_device.hpp"
#include "ops.hpp"

namespace sgemm_emu_dev {

namespace {

enum { EPI_PLAIN = 0, EPI_GATED = 1, EPI_ADAPTER = 2, EPI_PARTIAL = 3 };

constexpr int KS = 32;                       // K step
constexpr int RING = 4;

template <int WAVES_M_, int WAVES_N_, int TM_, int TN_>
struct Tile {
    static constexpr int WAVES_M = WAVES_M_, WAVES_N = WAVES_N_, WAVES = WAVES_M * WAVES_N, NT = 64 * WAVES;
    static constexpr int TM = TM_, TN = TN_;                       // one wave's part
    static constexpr int BM = WAVES_M * TM, BN = WAVES_N * TN;
    static constexpr int MI = TM / 32, NI = TN / 32;
    static constexpr int A_COPIES = BM / 16 / WAVES, B_COPIES = BN / 16 / WAVES;   // 16-row copies per wave and step
    static constexpr int STAGE = (BM + BN) * KS;                   // BF16 elements of one ring buffer
    static constexpr int PITCH = TN + 8;                           // epilogue rows: an odd number of 16-byte slots
    static constexpr int EPI_WAVE = TM * PITCH;
    static constexpr int LDS = RING * STAGE > WAVES * EPI_WAVE ? RING * STAGE : WAVES * EPI_WAVE;
    static_assert(BM % (16 * WAVES) == 0 && BN % (16 * WAVES) == 0, "tile rows split into 16-row copies");
};

using Tile256 = Tile<2, 4, 128, 64>;         // 8 waves, one workgroup per CU
using Tile128 = Tile<2, 2, 64, 64>;          // 4 waves, two workgroups per CU
using Tile64 = Tile<2, 2, 32, 32>;           // 4 waves

constexpr uint32_t OUT_OF_RANGE = 0xFFFFFFF0u;   // past every descriptor: reads zeros

// Row of B behind tile row c (see the file's head): block c / 16 is gate rows
// for an even block, up rows for an odd one.
template <int EPI>
__device__ __forceinline__ int64_t b_row(const Bf16Gemm &g, int64_t n0, int c)
{
    if constexpr (EPI == EPI_GATED) {
        const int64_t F = g.N >> 1, f = lmin((n0 >> 1) + ((c >> 5) << 4) + (c & 15), F - 1);
        return (c & 16) ? F + f : f;
    } else {
        return lmin(n0 + c, g.N - 1);
    }
}

template <class T>
struct Frag {
    bf16x8_t a[T::MI], b[T::NI];
};

template <class T>
__device__ __forceinline__ void read_frag(Frag<T> &f, const uint16_t *buf, int slice, int wm, int wn, int lane)
{
    const int kg = slice * 2 + (lane >> 5);
#pragma unroll
    for (int j = 0; j < T::NI; ++j) {
        const int row = wn * T::TN + j * 32 + (lane & 31);
        f.b[j] = ld_frag(buf + T::BM * KS + row * KS + bslot(row, kg) * 8);
    }
#pragma unroll
    for (int i = 0; i < T::MI; ++i) {
        const int row = wm * T::TM + i * 32 + (lane & 31);
        f.a[i] = ld_frag(buf + row * KS + bslot(row, kg) * 8);
    }
}

template <class T, int FIRST, int LAST>
__device__ __forceinline__ void mfma_part(f32x16_t (&acc)[T::NI][T::MI], const Frag<T> &f)
{
    int n = 0;
#pragma unroll
    for (int i = 0; i < T::MI; ++i)
#pragma unroll
        for (int j = 0; j < T::NI; ++j) {
            if (n >= FIRST && n < LAST)
                acc[j][i] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(f.b[j], f.a[i], acc[j][i], 0, 0, 0);
            ++n;
        }
}

// Add the adapters' part: acc[n][m] += up[i][n][:] . S[m][:] for the rows m of
// adapter i, one adapter of the wave's rows after another (in order of their
// first row).  S comes in two BF16 parts (16 significant bits; the rest lies
// 2^-8 below the output's own rounding), up is exact.  A lane keeps its old
// value unless its row belongs to the adapter: zero times Inf or NaN in one
// adapter's weights never reaches another's rows.
template <class T>
__device__ __forceinline__ void add_adapters(f32x16_t (&acc)[T::NI][T::MI], const Bf16Gemm &g, int64_t m0w,
                                             int64_t n0w, int lane)
{
    int id[T::MI];
    const uint16_t *srow[T::MI], *urow[T::NI];
    uint32_t todo[T::MI];
#pragma unroll
    for (int i = 0; i < T::MI; ++i) {
        const int64_t m = m0w + i * 32 + (lane & 31);
        srow[i] = g.S + lmin(m, g.M - 1) * 2 * g.rp + 8 * (lane >> 5);
        const int v = m < g.M ? g.ids[m] : -1;
        id[i] = v >= 0 && v < g.n ? v : -1;
        todo[i] = (uint32_t)__ballot(id[i] >= 0);
    }
#pragma unroll
    for (int j = 0; j < T::NI; ++j)
        urow[j] = g.up + lmin(n0w + j * 32 + (lane & 31), g.N - 1) * g.r + 8 * (lane >> 5);
    const bool vec = g.r % 8 == 0 && ((uintptr_t)g.up % 16) == 0;
    for (;;) {
        int me = -1;
#pragma unroll
        for (int i = T::MI - 1; i >= 0; --i)
            if (todo[i] != 0) me = __builtin_amdgcn_readlane(id[i], __builtin_ctz(todo[i]));
        if (me < 0) break;
        bool own[T::MI];
#pragma unroll
        for (int i = 0; i < T::MI; ++i) {
            own[i] = id[i] == me;
            todo[i] &= ~(uint32_t)__ballot(own[i]);
        }
        const int64_t bank = (int64_t)me * g.N * g.r;
        for (int64_t rc = 0; rc < g.rp; rc += 16) {
            u32x4_t up[T::NI], hi[T::MI], lo[T::MI];
#pragma unroll
            for (int j = 0; j < T::NI; ++j) {
                const uint16_t *p = urow[j] + bank + rc;
                const int64_t r0 = rc + 8 * (lane >> 5);
                up[j] = u32x4_t{0, 0, 0, 0};
                if (vec) {
                    if (r0 < g.r) up[j] = *reinterpret_cast<const u32x4_t *>(p);
                } else {
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        if (r0 + e < g.r) up[j][e >> 1] |= (uint32_t)p[e] << (16 * (e & 1));
                }
            }
#pragma unroll
            for (int i = 0; i < T::MI; ++i) {
                hi[i] = *reinterpret_cast<const u32x4_t *>(srow[i] + rc);
                lo[i] = *reinterpret_cast<const u32x4_t *>(srow[i] + g.rp + rc);
            }
#pragma unroll
            for (int i = 0; i < T::MI; ++i)
#pragma unroll
                for (int j = 0; j < T::NI; ++j) {
                    const bf16x8_t u = __builtin_bit_cast(bf16x8_t, up[j]);
                    f32x16_t t = __builtin_amdgcn_mfma_f32_32x32x16_bf16(u, __builtin_bit_cast(bf16x8_t, lo[i]),
                                                                         acc[j][i], 0, 0, 0);
                    t = __builtin_amdgcn_mfma_f32_32x32x16_bf16(u, __builtin_bit_cast(bf16x8_t, hi[i]), t, 0, 0, 0);
#pragma unroll
                    for (int q = 0; q < 16; ++q) acc[j][i][q] = own[i] ? t[q] : acc[j][i][q];
                }
        }
    }
}

// One wave's TM x W block of BF16 results in LDS (rows of PITCH elements) ->
// rows m0w.., columns c0.. of a matrix of `cols` columns: 128-bit stores where
// the matrix allows them, else a row's elements by consecutive lanes.
template <class T, int W>
__device__ __forceinline__ void flush_block(const uint16_t *buf, uint16_t *out, int64_t ld, int64_t M, int64_t cols,
                                            int64_t m0w, int64_t c0, int lane)
{
    if (((uintptr_t)out % 16) == 0 && ld % 8 == 0 && c0 + W <= cols) {
        constexpr int PER_ROW = W / 8, ROWS = 64 / PER_ROW;        // lanes per row, rows per pass
#pragma unroll 4
        for (int p = 0; p < T::TM / ROWS; ++p) {
            const int row = p * ROWS + lane / PER_ROW, c = (lane % PER_ROW) * 8;
            const u32x4_t v = *reinterpret_cast<const u32x4_t *>(buf + row * T::PITCH + c);
            if (m0w + row < M) *reinterpret_cast<u32x4_t *>(out + (m0w + row) * ld + c0 + c) = v;
        }
    } else {
        constexpr int ROWS = 64 / W;
        const int c = lane % W;
#pragma unroll 8
        for (int p = 0; p < T::TM / ROWS; ++p) {
            const int row = p * ROWS + lane / W;
            const uint16_t v = buf[row * T::PITCH + c];
            if (m0w + row < M && c0 + c < cols) out[(m0w + row) * ld + c0 + c] = v;
        }
    }
}

// LDS accesses of one wave complete in order; this keeps the compiler from
// reordering them across lanes' hand-offs.
__device__ __forceinline__ void wave_fence()
{
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
}

template <class T>
__device__ __forceinline__ void put4(uint16_t *buf, int row, int col, float v0, float v1, float v2, float v3)
{
    typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
    *reinterpret_cast<u32x2 *>(buf + row * T::PITCH + col) = u32x2{pack2(v0, v1), pack2(v2, v3)};
}

template <class T, int EPI, int GATE>
__device__ __forceinline__ void gemm_tile(const Bf16Gemm &g, uint16_t *lds)
{
    typedef __attribute__((address_space(3))) void lds_void_t;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wm = wave / T::WAVES_N, wn = wave % T::WAVES_N;

    int tm, tn;
    tile_of_index((int)blockIdx.x, (int)gridDim.x, g.tiles_m, g.tiles_n, g.group_m, tm, tn);
    const int64_t m0 = (int64_t)tm * T::BM, n0 = (int64_t)tn * T::BN;
    const int64_t kb = (int64_t)blockIdx.y * g.k_per_split, ke = lmin(kb + g.k_per_split, g.K);
    const int nk = (int)((ke - kb + KS - 1) / KS);

    // Copies: lane -> (row, 16-byte slot) of a 16-row block.  The rows' offsets
    // are relative to a per-copy base; k past the end reads zeros.
    const int srow = lane >> 2;
    rsrc_t ra[T::A_COPIES], rb[T::B_COPIES];
    uint32_t aoff[T::A_COPIES], boff[T::B_COPIES];
    int akg[T::A_COPIES], bkg[T::B_COPIES];
#pragma unroll
    for (int d = 0; d < T::A_COPIES; ++d) {
        const int r = (wave * T::A_COPIES + d) * 16;
        const int64_t first = lmin(m0 + r, g.M - 1), mine = lmin(m0 + r + srow, g.M - 1);
        ra[d] = make_rsrc(g.A + first * g.lda, 0xFFFFFFF0ll);
        akg[d] = bslot(r + srow, lane & 3) * 8;
        aoff[d] = (uint32_t)((mine - first) * g.lda * 2);
    }
#pragma unroll
    for (int d = 0; d < T::B_COPIES; ++d) {
        const int r = (wave * T::B_COPIES + d) * 16;
        const int64_t first = b_row<EPI>(g, n0, r), mine = b_row<EPI>(g, n0, r + srow);
        rb[d] = make_rsrc(g.B + first * g.ldb, 0xFFFFFFF0ll);
        bkg[d] = bslot(r + srow, lane & 3) * 8;
        boff[d] = (uint32_t)((mine - first) * g.ldb * 2);
    }
    auto stage = [&](int kt) {
        uint16_t *const buf = lds + (kt & (RING - 1)) * T::STAGE;
        const int64_t k0 = kb + (int64_t)kt * KS;
#pragma unroll
        for (int d = 0; d < T::A_COPIES; ++d) {
            const int64_t k = k0 + akg[d];
            const uint32_t off = k < ke ? aoff[d] + (uint32_t)(k * 2) : OUT_OF_RANGE;
            __builtin_amdgcn_raw_ptr_buffer_load_lds(
                ra[d], (lds_void_t *)(buf + (wave * T::A_COPIES + d) * 16 * KS), 16, (int)off, 0, 0, 0);
        }
#pragma unroll
        for (int d = 0; d < T::B_COPIES; ++d) {
            const int64_t k = k0 + bkg[d];
            const uint32_t off = k < ke ? boff[d] + (uint32_t)(k * 2) : OUT_OF_RANGE;
            __builtin_amdgcn_raw_ptr_buffer_load_lds(
                rb[d], (lds_void_t *)(buf + T::BM * KS + (wave * T::B_COPIES + d) * 16 * KS), 16, (int)off, 0, 0, 0);
        }
    };

    f32x16_t acc[T::NI][T::MI];
#pragma unroll
    for (int j = 0; j < T::NI; ++j)
#pragma unroll
        for (int i = 0; i < T::MI; ++i) acc[j][i] = f32x16_t{};

    constexpr int COPIES = T::A_COPIES + T::B_COPIES, NM = T::MI * T::NI, TAIL = NM / 2;
    Frag<T> f0, f1;
    stage(0);
    stage(1);
    stage(2);
    wait_vmem_at_most<2 * COPIES>();
    lds_barrier();
    read_frag<T>(f0, lds, 0, wm, wn, lane);
    for (int kt = 0; kt < nk; ++kt) {
        const uint16_t *const buf = lds + (kt & (RING - 1)) * T::STAGE;
        stage(kt + 3);
        read_frag<T>(f1, buf, 1, wm, wn, lane);
        mfma_part<T, 0, NM>(acc, f0);
        mfma_part<T, 0, NM - TAIL>(acc, f1);
        wait_vmem_at_most<2 * COPIES>();     // step kt + 1 has landed; kt + 2 and kt + 3 may be in flight
        lds_barrier();
        read_frag<T>(f0, lds + ((kt + 1) & (RING - 1)) * T::STAGE, 0, wm, wn, lane);
        mfma_part<T, NM - TAIL, NM>(acc, f1);
    }
    wait_vmem_at_most<0>();                  // no copy may land in the epilogue's space
    lds_barrier();

    const int64_t m0w = m0 + wm * T::TM, n0w = n0 + wn * T::TN;
    const int mlane = lane & 31, half = lane >> 5;
    if constexpr (EPI == EPI_PARTIAL) {
        float *const part = g.partials + (int64_t)blockIdx.y * g.M * g.N;
        const bool vec = g.N % 4 == 0;
#pragma unroll
        for (int i = 0; i < T::MI; ++i) {
            const int64_t m = m0w + i * 32 + mlane;
            if (m >= g.M) continue;
#pragma unroll
            for (int j = 0; j < T::NI; ++j)
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const int64_t n = n0w + j * 32 + 8 * q + 4 * half;
                    float *const p = part + m * g.N + n;
                    const f32x4_t v = {acc[j][i][4 * q], acc[j][i][4 * q + 1], acc[j][i][4 * q + 2],
                                       acc[j][i][4 * q + 3]};
                    if (vec && n + 4 <= g.N) {
                        *reinterpret_cast<f32x4_t *>(p) = v;
                    } else {
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            if (n + e < g.N) p[e] = v[e];
                    }
                }
        }
        return;
    }
    if constexpr (EPI == EPI_ADAPTER) add_adapters<T>(acc, g, m0w, n0w, lane);

    uint16_t *const out = lds + wave * T::EPI_WAVE;
    if constexpr (EPI == EPI_GATED) {
        const int64_t F = g.N >> 1, f0w = n0w >> 1;
        if (g.bias != nullptr) {
#pragma unroll
            for (int j = 0; j < T::NI; ++j)
#pragma unroll
                for (int q = 0; q < 16; ++q) {
                    const int n = 8 * (q >> 2) + 4 * half + (q & 3);             // row of the 32-row block
                    const int64_t f = lmin(f0w + j * 16 + (n & 15), F - 1);
                    const float b = bf2f(g.bias[n < 16 ? f : F + f]);
#pragma unroll
                    for (int i = 0; i < T::MI; ++i) acc[j][i][q] += b;
                }
        }
        constexpr int W = T::TN / 2;
        if (g.Z != nullptr) {
            // pre-activations stay in 32 bits: a lane's four are 16 bytes of a row
#pragma unroll
            for (int i = 0; i < T::MI; ++i) {
                const int64_t m = m0w + i * 32 + mlane;
                if (m >= g.M) continue;
#pragma unroll
                for (int j = 0; j < T::NI; ++j)
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const int64_t f = f0w + j * 16 + 8 * (q & 1) + 4 * half;
                        // rows are padded to a multiple of 8, so four always fit
                        if (f < F)
                            *reinterpret_cast<f32x4_t *>(g.Z + m * g.ldz + (q >> 1) * (g.ldz / 2) + f) =
                                f32x4_t{acc[j][i][4 * q], acc[j][i][4 * q + 1], acc[j][i][4 * q + 2],
                                        acc[j][i][4 * q + 3]};
                    }
            }
        }
#pragma unroll
        for (int i = 0; i < T::MI; ++i)
#pragma unroll
            for (int j = 0; j < T::NI; ++j)
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    float h[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) h[e] = gate_act<GATE>(acc[j][i][4 * q + e]) * acc[j][i][8 + 4 * q + e];
                    put4<T>(out, i * 32 + mlane, j * 16 + 8 * q + 4 * half, h[0], h[1], h[2], h[3]);
                }
        wave_fence();
        flush_block<T, W>(out, g.C, g.ldc, g.M, F, m0w, f0w, lane);
    } else {
        if (g.bias != nullptr) {
#pragma unroll
            for (int j = 0; j < T::NI; ++j)
#pragma unroll
                for (int q = 0; q < 16; ++q) {
                    const float b = bf2f(g.bias[lmin(n0w + j * 32 + 8 * (q >> 2) + 4 * half + (q & 3), g.N - 1)]);
#pragma unroll
                    for (int i = 0; i < T::MI; ++i) acc[j][i][q] += b;
                }
        }
#pragma unroll
        for (int i = 0; i < T::MI; ++i)
#pragma unroll
            for (int j = 0; j < T::NI; ++j)
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const f32x16_t &v = acc[j][i];
                    put4<T>(out, i * 32 + mlane, j * 32 + 8 * q + 4 * half, v[4 * q], v[4 * q + 1], v[4 * q + 2],
                            v[4 * q + 3]);
                }
        wave_fence();
        flush_block<T, T::TN>(out, g.C, g.ldc, g.M, g.N, m0w, n0w, lane);
    }
}

template <class T, int EPI, int GATE>
__global__ __launch_bounds__(T::NT, T::BM == 256 ? 1 : 2) void bf16_gemm_kernel(Bf16Gemm g)
{
    __shared__ __attribute__((aligned(16))) uint16_t lds[T::LDS];
    gemm_tile<T, EPI, GATE>(g, lds);
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

template <class T, int EPI, int GATE>
void launch_tile(Bf16Gemm g, hipStream_t stream)
{
    g.tiles_m = (int)((g.M + T::BM - 1) / T::BM);
    // a gated tile holds BN / 2 outputs of F = N / 2
    g.tiles_n = (int)((g.N + T::BN - 1) / T::BN);
    g.group_m = g.tiles_m < 8 ? g.tiles_m : 8;
    const dim3 grid((unsigned)((int64_t)g.tiles_m * g.tiles_n), (unsigned)g.splits);
    hipLaunchKernelGGL((bf16_gemm_kernel<T, EPI, GATE>), grid, dim3(T::NT), 0, stream, g);
}

template <class T>
hipError_t launch_epi(const Bf16Gemm &g, hipStream_t stream)
{
    if (g.splits > 1) {
        launch_tile<T, EPI_PARTIAL, 0>(g, stream);
        const dim3 grid((unsigned)((g.N + 255) / 256), (unsigned)(g.M < 16384 ? g.M : 16384));
        hipLaunchKernelGGL(bf16_sum_slices_kernel, grid, dim3(256), 0, stream, g);
        return hipGetLastError();
    }
    switch (g.gate) {
    case kSilu: launch_tile<T, EPI_GATED, kSilu>(g, stream); break;
    case kGelu: launch_tile<T, EPI_GATED, kGelu>(g, stream); break;
    case kGeluTanh: launch_tile<T, EPI_GATED, kGeluTanh>(g, stream); break;
    case kSigmoid: launch_tile<T, EPI_GATED, kSigmoid>(g, stream); break;
    case kRelu: launch_tile<T, EPI_GATED, kRelu>(g, stream); break;
    default:
        if (g.ids != nullptr) launch_tile<T, EPI_ADAPTER, 0>(g, stream);
        else launch_tile<T, EPI_PLAIN, 0>(g, stream);
    }
    return hipGetLastError();
}

struct TilePlan {
    int tile;
    int splits;
};

int64_t tiles_of(int64_t M, int64_t N, int64_t t) { return ((M + t - 1) / t) * ((N + t - 1) / t); }

// The tile and the K slices of a product.
TilePlan tile_plan(int64_t M, int64_t N, int64_t K, bool plain, int num_cus)
{
    TilePlan p{64, 1};
    if (tiles_of(M, N, 256) * 4 >= num_cus * 3) p.tile = 256;
    else if (tiles_of(M, N, 128) >= num_cus || plain) p.tile = 128;
    if (plain && p.tile == 128) {
        const int64_t t = tiles_of(M, N, 128);
        while (p.splits < 16 && t * (p.splits + 1) <= 2 * (int64_t)num_cus && K / (p.splits + 1) >= 512) ++p.splits;
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
    if (g.K == 0) {                          // nothing is read: every copy is past the end of K
        g.A = g.B = nullptr;
        g.lda = g.ldb = 8;
    }
    if (g.K % 8 != 0 || g.lda % 8 != 0 || g.ldb % 8 != 0 || !aligned(g.A, 16) || !aligned(g.B, 16))
        return hipErrorInvalidValue;
    const bool plain = g.gate < 0 && g.ids == nullptr;
    TilePlan p = tile_plan(g.M, g.N, g.K, plain, num_cus);
    if (g.partials == nullptr) p.splits = 1;
    g.splits = p.splits;
    g.k_per_split = round_up((g.K + p.splits - 1) / p.splits, KS);
    if (p.tile == 256) return launch_epi<Tile256>(g, stream);
    if (p.tile == 128) return launch_epi<Tile128>(g, stream);
    return launch_epi<Tile64>(g, stream);
}

}  // namespace sgemm_emu_dev
