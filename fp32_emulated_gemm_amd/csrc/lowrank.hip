// lowrank.hip -- few-row products and the low-rank parts of the adapters.
//
// dot_tile, shared by the few-row products and the shrink: a workgroup's eight
// waves split K, and their sums are added through LDS in wave order.  With few
// rows of X the weight passes once, and the time is its bytes' and the latency
// of the loads.
//   * Operands whose rows start at whole dwords go through LDS: steps of 512 bytes of every row are copied
//     by buffer loads with LDS destination (two whole row pieces per
//     instruction) into a ring, and each wave multiplies its 64-byte slice of the
//     rows.  Loaded straight into the MFMA's fragments (16 rows x 64 bytes per
//     instruction), a CU takes in about 20 bytes per ns whatever the loads in
//     flight: 81 us for the shrink of 8192 x 4096 bfloat16 to rank 64.
//   * Others (bfloat16 with odd rows) are loaded straight into the fragments: 40 us
//     for 48 x 1271 -> 2 x 8024 gated, 19 us with K = 1270.
// FP32 operands take the FP32 matrix instruction (FP32 products, FP32 sums): a
// lane's four consecutive k are the k of four instructions, the same for both
// operands, so their order inside a step does not matter.
#include "ops_device.hpp"
#include "ops.hpp"

namespace sgemm_emu_dev {

namespace {

constexpr int WAVES = 8;                         // of a dot_tile workgroup
constexpr int NT = 64 * WAVES;
constexpr uint32_t OUT_OF_RANGE = 0xFFFFFFF0u;   // past every descriptor: reads zeros

template <class T>
__device__ __forceinline__ f32x4_t mfma16(u32x4_t a, u32x4_t b, f32x4_t c)
{
    if constexpr (sizeof(T) == 2) {
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, a), __builtin_bit_cast(bf16x8_t, b),
                                                       c, 0, 0, 0);
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
            c = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(a[e]), __uint_as_float(b[e]), c, 0, 0, 0);
        return c;
    }
}

// B blocks of 16 rows of an operand: where each block starts, and the offsets of
// this lane's row in it as the copies take it and as the fragments do, or
// OUT_OF_RANGE for a row that reads zeros.
template <int B>
struct Rows {
    const char *p[B];
    uint32_t off[B], frag[B];
};

// The row of a block that a lane copies.
__device__ __forceinline__ int copy_row(int wave, int lane) { return 2 * wave + (lane >> 5); }

// VEC elements of a row from k on, zeros from ke on, at any element's address.
template <class T>
__device__ __forceinline__ u32x4_t load_k(const char *p, uint32_t row, int64_t k, int64_t ke)
{
    constexpr int V = Elem<T>::VEC;
    const T *const src = (const T *)(p + row) + k;
    u32x4_t v = {0, 0, 0, 0};
    if (row == OUT_OF_RANGE || k >= ke) return v;
    if (k + V <= ke) return *reinterpret_cast<const u32x4_any *>(src);
#pragma unroll
    for (int e = 0; e < V; ++e)
        if (k + e < ke) {
            if constexpr (sizeof(T) == 4) v[e] = __float_as_uint(src[e]);
            else v[e >> 1] |= (uint32_t)src[e] << (16 * (e & 1));
        }
    return v;
}

constexpr int STEP_BYTES = 512;                  // of a row, per step
template <int NB, int MB>
struct Ring {
    static constexpr int BLOCKS = NB + MB, STAGE = BLOCKS * 16 * STEP_BYTES;   // bytes
    static constexpr int STAGES = BLOCKS <= 2 ? 4 : BLOCKS == 3 || BLOCKS == 6 ? 3 : 2;
    static constexpr int SUMS = WAVES * NB * MB * 1024;
    static constexpr int BYTES = STAGES * STAGE > SUMS ? STAGES * STAGE : SUMS;
};

// acc[nb][mb] += rows of W times rows of X over this wave's share of [kb, ke).
template <class T, int NB, int MB, bool ALIGNED>
__device__ __forceinline__ void dot_tile(f32x4_t (&acc)[NB][MB], const Rows<NB> &w, const Rows<MB> &x, int64_t kb,
                                         int64_t ke, float *lds, int wave, int lane)
{
    typedef __attribute__((address_space(3))) void lds_void_t;
    constexpr int V = Elem<T>::VEC;
    if constexpr (ALIGNED) {
        // 16-byte slot s of row r of a block lies at slot s ^ r, so the fragment
        // reads of 16 rows are on distinct banks
        typedef Ring<NB, MB> R;
        constexpr int KC = STEP_BYTES / (int)sizeof(T);
        const int row = copy_row(wave, lane), k_lane = ((lane & 31) ^ row) * V;
        const int n = (int)((ke - kb + KC - 1) / KC);
        auto stage = [&](int t) {
            char *const buf = (char *)lds + (t % R::STAGES) * R::STAGE;
            const int64_t k = kb + (int64_t)t * KC + k_lane;
            const bool in = k + V <= ke;         // whole pieces only
            const uint32_t koff = (uint32_t)(k * (int64_t)sizeof(T));
#pragma unroll
            for (int b = 0; b < R::BLOCKS; ++b) {
                const uint32_t off = b < NB ? w.off[b < NB ? b : 0] : x.off[b < NB ? 0 : b - NB];
                const rsrc_t r = make_rsrc(b < NB ? w.p[b < NB ? b : 0] : x.p[b < NB ? 0 : b - NB], 0xFFFFFFF0ll);
                __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_void_t *)(buf + b * 16 * STEP_BYTES + wave * 1024), 16,
                                                         (int)(in && off != OUT_OF_RANGE ? off + koff : OUT_OF_RANGE),
                                                         0, 0, 0);
            }
        };
        __syncthreads();                         // the ring's space may still be read by its last user
        const int slot = ((wave * 4 + (lane >> 4)) ^ (lane & 15)) * 16 + (lane & 15) * STEP_BYTES;
#pragma unroll
        for (int t = 0; t < R::STAGES; ++t) stage(t);
        const int64_t whole = ke - (ke - kb) % V;
        if (whole < ke && wave == 0) {           // the elements behind the last whole piece
            const int64_t k = whole + (lane >> 4) * V;
            u32x4_t fw[NB], fx[MB];
#pragma unroll
            for (int nb = 0; nb < NB; ++nb) fw[nb] = load_k<T>(w.p[nb], w.frag[nb], k, ke);
#pragma unroll
            for (int mb = 0; mb < MB; ++mb) fx[mb] = load_k<T>(x.p[mb], x.frag[mb], k, ke);
#pragma unroll
            for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                for (int mb = 0; mb < MB; ++mb) acc[nb][mb] = mfma16<T>(fw[nb], fx[mb], acc[nb][mb]);
        }
        for (int t = 0; t < n; ++t) {
            wait_vmem_at_most<(R::STAGES - 1) * R::BLOCKS>();   // step t has landed,
            lds_barrier();                                      // everybody's
            const char *const buf = (const char *)lds + (t % R::STAGES) * R::STAGE + slot;
            u32x4_t fw[NB], fx[MB];
#pragma unroll
            for (int nb = 0; nb < NB; ++nb) fw[nb] = *reinterpret_cast<const u32x4_t *>(buf + nb * 16 * STEP_BYTES);
#pragma unroll
            for (int mb = 0; mb < MB; ++mb)
                fx[mb] = *reinterpret_cast<const u32x4_t *>(buf + (NB + mb) * 16 * STEP_BYTES);
            lds_barrier();                                      // everybody has read it: all buffers in flight again
            stage(t + R::STAGES);
#pragma unroll
            for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                for (int mb = 0; mb < MB; ++mb) acc[nb][mb] = mfma16<T>(fw[nb], fx[mb], acc[nb][mb]);
        }
        wait_vmem_at_most<0>();                  // no copy may land in what comes next
        lds_barrier();
    } else {
        constexpr int STEP = 4 * V;
        for (int64_t k0 = kb + wave * STEP; k0 < ke; k0 += WAVES * STEP) {
            const int64_t k = k0 + (lane >> 4) * V;
            u32x4_t fw[NB], fx[MB];
#pragma unroll
            for (int nb = 0; nb < NB; ++nb) fw[nb] = load_k<T>(w.p[nb], w.frag[nb], k, ke);
#pragma unroll
            for (int mb = 0; mb < MB; ++mb) fx[mb] = load_k<T>(x.p[mb], x.frag[mb], k, ke);
#pragma unroll
            for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                for (int mb = 0; mb < MB; ++mb) acc[nb][mb] = mfma16<T>(fw[nb], fx[mb], acc[nb][mb]);
        }
    }
}

template <int NB, int MB>
__device__ __forceinline__ void clear(f32x4_t (&acc)[NB][MB])
{
#pragma unroll
    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
        for (int mb = 0; mb < MB; ++mb) acc[nb][mb] = f32x4_t{};
}

template <int NB, int MB>
__device__ __forceinline__ void put_sums(float *lds, const f32x4_t (&acc)[NB][MB], int wave, int lane)
{
#pragma unroll
    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
        for (int mb = 0; mb < MB; ++mb)
            reinterpret_cast<f32x4_t *>(lds)[((wave * NB + nb) * MB + mb) * 64 + lane] = acc[nb][mb];
}

// Sum over the waves of element (n, m) of the tile put by put_sums.
template <int NB, int MB>
__device__ __forceinline__ float get_sum(const float *lds, int n, int m)
{
    const int at = ((n >> 4) * MB + (m >> 4)) * 256 + ((((n & 15) >> 2) * 16 + (m & 15)) << 2) + (n & 3);
    float v = lds[at];
#pragma unroll
    for (int w = 1; w < WAVES; ++w) v += lds[w * NB * MB * 256 + at];
    return v;
}

// Blocks b of rows r0 + 16 b .. of an operand of `rows` rows; rows past it re-read
// the last one (their results are dropped).
template <class T, int B>
__device__ __forceinline__ Rows<B> rows_at(const T *p, int64_t ld, int64_t r0, int64_t rows, int wave, int lane)
{
    Rows<B> q;
#pragma unroll
    for (int b = 0; b < B; ++b) {
        auto at = [&](int row) {
            return (uint32_t)((lmin(r0 + b * 16 + row, rows - 1) - r0) * ld * (int64_t)sizeof(T));
        };
        q.p[b] = (const char *)(p + r0 * ld);
        q.off[b] = at(copy_row(wave, lane));
        q.frag[b] = at(lane & 15);
    }
    return q;
}

// ---------------------------------------------------------------- gated, one pass
// NB / 2 blocks of 16 gate rows, then the NB / 2 blocks of up rows of the same
// outputs; the whole K in one workgroup, so that the gate runs on the sums before
// they leave.  Bound by the weight's bytes: bfloat16 4096 -> 2 x 8192 (134 MB) 34 us
// for 1 row (3.9 TB/s), 41 for 64, whose X every workgroup copies beside its rows
// of W; float32 1 x 1024 -> 2 x 4096 (34 MB) 6 us.
template <class T, int NB, int MB, int GATE, bool ALIGNED>
__global__ __launch_bounds__(NT) void few_gated_kernel(FewRows a)
{
    __shared__ __attribute__((aligned(16))) float lds[Ring<NB, MB>::BYTES / 4];
    constexpr int OUT = NB / 2 * 16;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t n0 = (int64_t)blockIdx.x * OUT, F = a.N;
    Rows<NB> w = rows_at<T, NB>((const T *)a.W, a.ldw, n0, F, wave, lane);
#pragma unroll
    for (int b = 0; b < NB / 2; ++b) {
        w.p[NB / 2 + b] = (const char *)((const T *)a.W + (F + n0) * a.ldw);
        w.off[NB / 2 + b] = w.off[b];
        w.frag[NB / 2 + b] = w.frag[b];
    }
    const Rows<MB> x = rows_at<T, MB>((const T *)a.X, a.ldx, 0, a.M, wave, lane);
    f32x4_t acc[NB][MB];
    clear<NB, MB>(acc);
    dot_tile<T, NB, MB, ALIGNED>(acc, w, x, 0, a.K, lds, wave, lane);
    put_sums<NB, MB>(lds, acc, wave, lane);
    __syncthreads();
    const T *bias = (const T *)a.bias;
    T *Y = (T *)a.Y;
    for (int o = threadIdx.x; o < OUT * 16 * MB; o += NT) {
        const int n = o % OUT, m = o / OUT;
        if (n0 + n >= F || m >= a.M) continue;
        float v = get_sum<NB, MB>(lds, n, m), u = get_sum<NB, MB>(lds, OUT + n, m);
        if (bias != nullptr) {
            v += Elem<T>::load(bias + n0 + n);
            u += Elem<T>::load(bias + F + n0 + n);
        }
        Y[m * a.ldy + n0 + n] = Elem<T>::store(gate_act<GATE>(v) * u);
    }
}

// ---------------------------------------------------------------- K slices
// partials[slice][m][n] of X W^T, 32 or 64 rows of W per workgroup, beside the
// shrink's workgroups (they come first; nothing here depends on them).  Sliced
// because so few rows a workgroup leave CUs idle otherwise; the gated product with
// few outputs comes here too.  64 rows of 64 adapters of rank 16 on bfloat16 4096 x
// 4096 (50 MB): 15 us, and 4 for the finish; 16 rows, float32 1024 x 1024: 6 and 5,
// the latency of two launches.
template <class T>
struct Tokens {
    int64_t M, N, K;
    const T *X;
    int64_t ldx;
    const T *W;
    int64_t ldw;
    float *partials;
    int64_t k_per_slice;
    int n_blocks;
    int shrink_blocks;        // workgroups of the shrink: (16-row tile, row)
    Adapters ad;
    float *S;
    int64_t rp;
};

// One workgroup per row of a 16-row tile: the first row of an adapter multiplies
// the tile's rows of that adapter, the others end.
template <class T, bool ALIGNED>
__device__ __forceinline__ void shrink_row(const Tokens<T> &a, int block, float *lds, int wave, int lane)
{
    const int64_t m0 = (int64_t)(block >> 4) * 16;
    const int mine = block & 15;
    const int64_t m = m0 + (lane & 15);
    int32_t id = -1;
    if (m < a.M) {
        id = a.ad.ids[m];
        if (id >= a.ad.n) id = -1;
    }
    if (m0 + mine >= a.M) return;
    const int32_t me = __builtin_amdgcn_readlane(id, mine);
    if (me < 0) {
        for (int64_t j = threadIdx.x; j < a.rp; j += NT) a.S[(m0 + mine) * a.rp + j] = 0.0f;
        return;
    }
    const uint32_t own = (uint32_t)(__ballot(id == me) & 0xFFFFu);
    if ((own & ((1u << mine) - 1u)) != 0) return;                    // an earlier row computes it
    Rows<1> x = rows_at<T, 1>(a.X, a.ldx, m0, a.M, wave, lane);
    if (!((own >> copy_row(wave, lane)) & 1u)) x.off[0] = OUT_OF_RANGE;
    if (!((own >> (lane & 15)) & 1u)) x.frag[0] = OUT_OF_RANGE;
    const T *down = (const T *)a.ad.down + (int64_t)me * a.ad.r * a.K;
    const float scale = a.ad.scale != nullptr ? a.ad.scale[me] : 1.0f;
    for (int64_t r0 = 0; r0 < a.rp; r0 += 16) {
        const Rows<1> w = rows_at<T, 1>(down, a.K, r0, a.ad.r, wave, lane);
        f32x4_t acc[1][1];
        clear<1, 1>(acc);
        dot_tile<T, 1, 1, ALIGNED>(acc, w, x, 0, a.K, lds, wave, lane);
        put_sums<1, 1>(lds, acc, wave, lane);
        __syncthreads();
        if (threadIdx.x < 256) {
            const int n = threadIdx.x & 15, t = threadIdx.x >> 4;
            if ((own >> t) & 1u)
                a.S[(m0 + t) * a.rp + r0 + n] = r0 + n < a.ad.r ? scale * get_sum<1, 1>(lds, n, t) : 0.0f;
        }
        __syncthreads();
    }
}

template <class T, int MB, bool ALIGNED>
__global__ __launch_bounds__(NT) void tokens_kernel(Tokens<T> a)
{
    constexpr int NB = MB > 2 ? 4 : 2;           // token_rows
    __shared__ __attribute__((aligned(16))) float lds[Ring<NB, MB>::BYTES / 4];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    int block = (int)blockIdx.x;
    if (block < a.shrink_blocks) {
        shrink_row<T, ALIGNED>(a, block, lds, wave, lane);
        return;
    }
    block -= a.shrink_blocks;
    const int64_t n0 = (int64_t)(block % a.n_blocks) * (16 * NB), slice = block / a.n_blocks;
    const int64_t kb = slice * a.k_per_slice, ke = lmin(kb + a.k_per_slice, a.K);
    const Rows<NB> w = rows_at<T, NB>(a.W, a.ldw, n0, a.N, wave, lane);
    const Rows<MB> x = rows_at<T, MB>(a.X, a.ldx, 0, a.M, wave, lane);
    f32x4_t acc[NB][MB];
    clear<NB, MB>(acc);
    dot_tile<T, NB, MB, ALIGNED>(acc, w, x, kb, ke, lds, wave, lane);
    put_sums<NB, MB>(lds, acc, wave, lane);
    __syncthreads();
    float *const part = a.partials + slice * a.M * a.N;
    for (int o = threadIdx.x; o < 16 * NB * 16 * MB; o += NT) {
        const int n = o % (16 * NB), m = o / (16 * NB);
        if (n0 + n < a.N && m < a.M) part[(int64_t)m * a.N + n0 + n] = get_sum<NB, MB>(lds, n, m);
    }
}

// Y[m][n] = sum of the slices in order + bias + up[i][n] . S[m].
template <class T>
__global__ __launch_bounds__(256) void tokens_finish_kernel(Tokens<T> a, int slices, const T *bias, T *Y, int64_t ldy)
{
    const int64_t n = (int64_t)blockIdx.x * 256 + threadIdx.x, m = blockIdx.y;
    if (n >= a.N) return;
    const int64_t plane = a.M * a.N;
    const float *p = a.partials + m * a.N + n;
    float v = 0.0f;
    for (int s = 0; s < slices; ++s) v += p[s * plane];
    if (bias != nullptr) v += Elem<T>::load(bias + n);
    if (a.shrink_blocks > 0) {
        const int32_t i = a.ad.ids[m];
        if (i >= 0 && i < a.ad.n) {
            const T *up = (const T *)a.ad.up + ((int64_t)i * a.N + n) * a.ad.r;
            const float *s = a.S + m * a.rp;
            constexpr int V = Elem<T>::VEC;
            float d = 0.0f;
            if (a.ad.r % V == 0 && ((uintptr_t)a.ad.up % 16) == 0) {
                for (int64_t j = 0; j < a.ad.r; j += V) {
                    const u32x4_t u = *reinterpret_cast<const u32x4_t *>(up + j);
#pragma unroll
                    for (int e = 0; e < V; ++e) {
                        float f;
                        if constexpr (sizeof(T) == 4) f = __uint_as_float(u[e]);
                        else f = bf2f((uint16_t)(u[e >> 1] >> (16 * (e & 1))));
                        d = __builtin_fmaf(s[j + e], f, d);
                    }
                }
            } else {
                for (int64_t j = 0; j < a.ad.r; ++j) d = __builtin_fmaf(s[j], Elem<T>::load(up + j), d);
            }
            v += d;
        }
    }
    Y[m * ldy + n] = Elem<T>::store(v);
}

// H[m][f] = act(gate) * up of the slices' sums + bias (a.N = 2F).
template <class T, int GATE>
__global__ __launch_bounds__(256) void gated_finish_kernel(Tokens<T> a, int slices, const T *bias, T *H, int64_t ldh)
{
    const int64_t f = (int64_t)blockIdx.x * 256 + threadIdx.x, m = blockIdx.y, F = a.N / 2;
    if (f >= F) return;
    const int64_t plane = a.M * a.N;
    const float *p = a.partials + m * a.N + f;
    float g = 0.0f, u = 0.0f;
    for (int s = 0; s < slices; ++s) {
        g += p[s * plane];
        u += p[s * plane + F];
    }
    if (bias != nullptr) {
        g += Elem<T>::load(bias + f);
        u += Elem<T>::load(bias + F + f);
    }
    H[m * ldh + f] = Elem<T>::store(gate_act<GATE>(g) * u);
}

// Rows that the copies to LDS take: they start at whole dwords.
template <class T>
bool rows_copied(const void *p, int64_t ld)
{
    return ld * (int64_t)sizeof(T) % 4 == 0 && aligned(p, 4);
}

// Rows of W per workgroup of a K-sliced product of M rows, and its K slices beside
// `others` workgroups of the launch, each with a step or more for every wave.  Up
// to 32 rows of X two workgroups fit a CU; with more, W and X take as many rows
// and one workgroup fills its LDS, so the launch should be one round of them
// (64 rows, 64 adapters of rank 16, bfloat16 4096 x 4096: 19 us; as two rounds of
// 32 rows of W 25).
int64_t token_rows(int64_t M) { return M > 32 ? 64 : 32; }
int token_slices(int dtype, int64_t M, int64_t N, int64_t K, int64_t others, int num_cus)
{
    const int64_t blocks = (N + token_rows(M) - 1) / token_rows(M), least = WAVES * (dtype == kF32 ? 16 : 32);
    int64_t s = ((M > 32 ? 1 : 2) * (int64_t)num_cus - others) / (blocks > 0 ? blocks : 1);
    if (s > K / least) s = K / least;
    return (int)(s < 1 ? 1 : s > 16 ? 16 : s);
}

// Workgroups of the shrink beside a few-row product.
int64_t shrink_rows(const FewRows &a) { return a.ad != nullptr ? round_up(a.M, 16) : 0; }

template <class T>
Tokens<T> make_tokens(const FewRows &a, int64_t N, int slices)
{
    Tokens<T> t{};
    t.M = a.M; t.N = N; t.K = a.K;
    t.X = (const T *)a.X; t.ldx = a.ldx;
    t.W = (const T *)a.W; t.ldw = a.ldw;
    t.partials = a.partials;
    // slices begin at whole 128-byte pairs of steps
    t.k_per_slice = round_up((a.K + slices - 1) / slices, 8 * Elem<T>::VEC);
    t.n_blocks = (int)((N + token_rows(a.M) - 1) / token_rows(a.M));
    if (a.ad != nullptr) {
        t.ad = *a.ad;
        t.S = a.S;
        t.rp = rank_pad(a.ad->r);
        t.shrink_blocks = (int)shrink_rows(a);
    }
    return t;
}

template <class T, int MB>
void launch_tokens_mb(const Tokens<T> &t, int slices, hipStream_t stream)
{
    const dim3 grid((unsigned)(t.shrink_blocks + t.n_blocks * slices)), block(NT);
    if (rows_copied<T>(t.W, t.ldw) && rows_copied<T>(t.X, t.ldx) && (t.shrink_blocks == 0 || rows_copied<T>(t.ad.down, t.K)))
        hipLaunchKernelGGL((tokens_kernel<T, MB, true>), grid, block, 0, stream, t);
    else
        hipLaunchKernelGGL((tokens_kernel<T, MB, false>), grid, block, 0, stream, t);
}

template <class T>
void launch_tokens(const Tokens<T> &t, int slices, hipStream_t stream)
{
    if (t.M <= 16) launch_tokens_mb<T, 1>(t, slices, stream);
    else if (t.M <= 32) launch_tokens_mb<T, 2>(t, slices, stream);
    else launch_tokens_mb<T, 4>(t, slices, stream);
}

template <class T, int NB, int MB, int GATE>
void launch_few_gated_al(const FewRows &a, hipStream_t stream)
{
    constexpr int OUT = NB / 2 * 16;
    const dim3 grid((unsigned)((a.N + OUT - 1) / OUT)), block(NT);
    if (rows_copied<T>(a.W, a.ldw) && rows_copied<T>(a.X, a.ldx))
        hipLaunchKernelGGL((few_gated_kernel<T, NB, MB, GATE, true>), grid, block, 0, stream, a);
    else
        hipLaunchKernelGGL((few_gated_kernel<T, NB, MB, GATE, false>), grid, block, 0, stream, a);
}

template <class T, int GATE>
void launch_few_gated(const FewRows &a, int num_cus, hipStream_t stream)
{
    if (a.partials != nullptr) {
        const int slices = token_slices(sizeof(T) == 4 ? kF32 : kBF16, a.M, 2 * a.N, a.K, 0, num_cus);
        const Tokens<T> t = make_tokens<T>(a, 2 * a.N, slices);
        launch_tokens<T>(t, slices, stream);
        hipLaunchKernelGGL((gated_finish_kernel<T, GATE>), dim3((unsigned)((a.N + 255) / 256), (unsigned)a.M), dim3(256),
                           0, stream, t, slices, (const T *)a.bias, (T *)a.Y, a.ldy);
        return;
    }
    const bool wide = a.N >= (int64_t)32 * num_cus;
    if (a.M <= 16) {
        if (wide) launch_few_gated_al<T, 4, 1, GATE>(a, stream);
        else launch_few_gated_al<T, 2, 1, GATE>(a, stream);
    } else if (a.M <= 32) {
        if (wide) launch_few_gated_al<T, 4, 2, GATE>(a, stream);
        else launch_few_gated_al<T, 2, 2, GATE>(a, stream);
    } else if (a.M <= 48) {
        if (wide) launch_few_gated_al<T, 4, 3, GATE>(a, stream);
        else launch_few_gated_al<T, 2, 3, GATE>(a, stream);
    } else {
        if (wide) launch_few_gated_al<T, 4, 4, GATE>(a, stream);
        else launch_few_gated_al<T, 2, 4, GATE>(a, stream);
    }
}

template <class T>
hipError_t launch_few_rows_t(const FewRows &a, int num_cus, hipStream_t stream)
{
    switch (a.gate) {
    case kSilu: launch_few_gated<T, kSilu>(a, num_cus, stream); break;
    case kGelu: launch_few_gated<T, kGelu>(a, num_cus, stream); break;
    case kGeluTanh: launch_few_gated<T, kGeluTanh>(a, num_cus, stream); break;
    case kSigmoid: launch_few_gated<T, kSigmoid>(a, num_cus, stream); break;
    case kRelu: launch_few_gated<T, kRelu>(a, num_cus, stream); break;
    default: {
        const int slices = token_slices(sizeof(T) == 4 ? kF32 : kBF16, a.M, a.N, a.K, shrink_rows(a), num_cus);
        const Tokens<T> t = make_tokens<T>(a, a.N, slices);
        launch_tokens<T>(t, slices, stream);
        hipLaunchKernelGGL((tokens_finish_kernel<T>), dim3((unsigned)((a.N + 255) / 256), (unsigned)a.M), dim3(256), 0,
                           stream, t, slices, (const T *)a.bias, (T *)a.Y, a.ldy);
    }
    }
    return hipGetLastError();
}

// ---------------------------------------------------------------- shrink
// S[t] = scale[i] down[i] X[t].  A workgroup takes 16 MB rows and walks the
// adapters that occur in them, in order of their first row: each pass multiplies
// all the tile's rows by that adapter's r rows and keeps the rows that belong to
// it.  Rows of one request are neighbours, so a tile of a prompt holds one or
// two adapters.  Bound by what a CU takes in, X's rows and `down`'s: bfloat16 8192 x
// 4096 to rank 16 19 us (X alone at the copy rate 13), to rank 64 37.  FP32 keeps S as floats; bfloat16 as two BF16 parts (rp high
// parts, then rp low parts per row, 16 significant bits), which is how the GEMM
// epilogue multiplies it.
template <class T>
__device__ __forceinline__ void put_s(float *S, int64_t rp, int64_t m, int64_t j, float v)
{
    if constexpr (sizeof(T) == 4) {
        S[m * rp + j] = v;
    } else {
        uint16_t *const row = (uint16_t *)S + m * 2 * rp;
        uint16_t hi, lo;
        split_hi_lo(v, hi, lo);
        row[j] = hi;
        row[rp + j] = lo;
    }
}

template <class T>
__device__ __forceinline__ float get_s(const float *S, int64_t rp, int64_t m, int64_t j)
{
    if constexpr (sizeof(T) == 4) {
        return S[m * rp + j];
    } else {
        const uint16_t *const row = (const uint16_t *)S + m * 2 * rp;
        return bf2f(row[j]) + bf2f(row[rp + j]);
    }
}

template <class T, int NB, int MB, bool AL>
__global__ __launch_bounds__(NT) void shrink_kernel(int64_t M, int64_t K, const T *X, int64_t ldx, Adapters ad,
                                                    float *S, int64_t rp)
{
    __shared__ __attribute__((aligned(16))) float lds[Ring<NB, MB>::BYTES / 4];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    constexpr int ROWS = 16 * MB;
    const int64_t m0 = (int64_t)blockIdx.x * ROWS;
    int32_t id = -1;
    if (lane < ROWS && m0 + lane < M) {
        id = ad.ids[m0 + lane];
        if (id >= ad.n) id = -1;
    }
    const Rows<MB> x = rows_at<T, MB>(X, ldx, m0, M, wave, lane);
    uint64_t todo = __ballot(id >= 0);
    const uint64_t none = __ballot(id < 0 && lane < ROWS && m0 + lane < M);
    if (none != 0)
        for (int64_t o = threadIdx.x; o < ROWS * rp; o += NT)
            if ((none >> (o / rp)) & 1) put_s<T>(S, rp, m0 + o / rp, o % rp, 0.0f);
    while (todo != 0) {
        const int32_t me = __builtin_amdgcn_readlane(id, (int)__builtin_ctzll(todo));
        const uint64_t own = __ballot(id == me);
        todo &= ~own;
        const T *down = (const T *)ad.down + (int64_t)me * ad.r * K;
        const float scale = ad.scale != nullptr ? ad.scale[me] : 1.0f;
        for (int64_t r0 = 0; r0 < rp; r0 += 16 * NB) {
            const Rows<NB> w = rows_at<T, NB>(down, K, r0, ad.r, wave, lane);
            f32x4_t acc[NB][MB];
            clear<NB, MB>(acc);
            dot_tile<T, NB, MB, AL>(acc, w, x, 0, K, lds, wave, lane);
            put_sums<NB, MB>(lds, acc, wave, lane);
            __syncthreads();
            for (int o = threadIdx.x; o < 16 * NB * ROWS; o += NT) {
                const int n = o % (16 * NB), m = o / (16 * NB);
                if (r0 + n < rp && ((own >> m) & 1))
                    put_s<T>(S, rp, m0 + m, r0 + n, r0 + n < ad.r ? scale * get_sum<NB, MB>(lds, n, m) : 0.0f);
            }
            __syncthreads();
        }
    }
}

template <class T, int NB, int MB>
void launch_shrink_mb(int64_t M, int64_t K, const T *X, int64_t ldx, const Adapters &ad, float *S, hipStream_t stream)
{
    const dim3 grid((unsigned)((M + 16 * MB - 1) / (16 * MB)));
    if (rows_copied<T>(X, ldx) && rows_copied<T>(ad.down, K))
        hipLaunchKernelGGL((shrink_kernel<T, NB, MB, true>), grid, dim3(NT), 0, stream, M, K, X, ldx, ad, S,
                           rank_pad(ad.r));
    else
        hipLaunchKernelGGL((shrink_kernel<T, NB, MB, false>), grid, dim3(NT), 0, stream, M, K, X, ldx, ad, S,
                           rank_pad(ad.r));
}

template <class T, int NB>
void launch_shrink_nb(int64_t M, int64_t K, const T *X, int64_t ldx, const Adapters &ad, float *S, int num_cus,
                      hipStream_t stream)
{
    // 16 rows per workgroup while that leaves at most two for a CU, else 32: with 32,
    // 8192 x 4096 bfloat16 to rank 16 took 24 us instead of 20.  From rank 33 on the
    // copies of `down` decide, NB + MB blocks of rows for each workgroup that a CU
    // runs: 37 us against 43 for rank 64 (float32: 91 against 103).
    auto taken = [&](int64_t mb) {
        const int64_t groups = (M + 16 * mb - 1) / (16 * mb);
        return (groups + num_cus - 1) / num_cus * (NB + mb);
    };
    const bool one = NB < 4 ? M <= (int64_t)32 * num_cus : taken(1) <= taken(2);
    if (one) launch_shrink_mb<T, NB, 1>(M, K, X, ldx, ad, S, stream);
    else launch_shrink_mb<T, NB, 2>(M, K, X, ldx, ad, S, stream);
}

template <class T>
hipError_t launch_shrink_t(int64_t M, int64_t K, const T *X, int64_t ldx, const Adapters &ad, float *S, int num_cus,
                           hipStream_t stream)
{
    if (ad.r <= 16) launch_shrink_nb<T, 1>(M, K, X, ldx, ad, S, num_cus, stream);
    else if (ad.r <= 32) launch_shrink_nb<T, 2>(M, K, X, ldx, ad, S, num_cus, stream);
    else launch_shrink_nb<T, 4>(M, K, X, ldx, ad, S, num_cus, stream);
    return hipGetLastError();
}

// ---------------------------------------------------------------- expand (FP32)
// Y[t] += up[i] S[t], one pass over Y: 12 us of 6144 x 1024, 4.2 TB/s.  A wave
// takes 32 rows x 64 columns: its part of Y is the accumulator of FP32 MFMAs over
// the rank, for one adapter of its rows after another (in order of their first
// row); a row keeps its old value unless it belongs to the adapter, so Inf and NaN
// in one adapter's weights never reach another's rows.
__global__ __launch_bounds__(256) void expand_kernel(int64_t M, int64_t N, GemmEpilogue ad, float *Y,
                                                     int64_t ldy)
{
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, half = lane >> 5;
    const int64_t m0 = ((int64_t)blockIdx.x * 2 + (wave >> 1)) * 32, n0 = ((int64_t)blockIdx.y * 2 + (wave & 1)) * 64;
    if (m0 >= M || n0 >= N) return;
    const int64_t m = m0 + (lane & 31);
    int32_t id = m < M ? ad.ids[m] : -1;
    if (id >= ad.n) id = -1;
    uint32_t todo = (uint32_t)__ballot(id >= 0);
    if (todo == 0) return;
    const float *srow = ad.S + lmin(m, M - 1) * ad.rp + 4 * half;
    int64_t col[2];
    float *y[2];
    f32x16_t acc[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        col[j] = n0 + j * 32 + (lane & 31);
        y[j] = Y + (m0 + 4 * half) * ldy + col[j];
#pragma unroll
        for (int r = 0; r < 16; ++r) {
            const int row = 8 * (r >> 2) + (r & 3);
            acc[j][r] = m0 + 4 * half + row < M && col[j] < N ? y[j][row * ldy] : 0.0f;
        }
    }
    const bool vec = ad.r % 4 == 0 && ((uintptr_t)ad.up % 16) == 0;
    while (todo != 0) {
        const int32_t me = __builtin_amdgcn_readlane(id, __builtin_ctz(todo));
        const uint32_t own = (uint32_t)__ballot(id == me) >> (4 * half);
        todo &= ~(uint32_t)__ballot(id == me);
        const float *bank = ad.up + (int64_t)me * N * ad.r + 4 * half;
        f32x16_t t[2] = {acc[0], acc[1]};
        for (int64_t q = 0; q < ad.r; q += 8) {
            // a lane's four consecutive ranks are the k of four instructions
            const f32x4_t s = *reinterpret_cast<const f32x4_t *>(srow + q);
            const int64_t k = q + 4 * half;
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const float *p = bank + lmin(col[j], N - 1) * ad.r + q;
                f32x4_t u = {0, 0, 0, 0};
                if (vec) {
                    if (k < ad.r) u = *reinterpret_cast<const f32x4_t *>(p);
                } else {
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (k + e < ad.r) u[e] = p[e];
                }
#pragma unroll
                for (int e = 0; e < 4; ++e) t[j] = __builtin_amdgcn_mfma_f32_32x32x2f32(s[e], u[e], t[j], 0, 0, 0);
            }
        }
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int r = 0; r < 16; ++r) acc[j][r] = (own >> (8 * (r >> 2) + (r & 3))) & 1 ? t[j][r] : acc[j][r];
    }
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int r = 0; r < 16; ++r) {
            const int row = 8 * (r >> 2) + (r & 3);
            if (m0 + 4 * half + row < M && col[j] < N) y[j][row * ldy] = acc[j][r];
        }
}

// ---------------------------------------------------------------- gradients of the low-rank factors
// G[i] = sum over adapter i's rows t of L[t] (x) R[t] (r x C), for one or two
// jobs (the two factors) in one launch.  The rows, grouped by adapter
// (prepare_kernel, layouts.hip), are cut into chunks of CH; workgroup (column block, chunk)
// sums the pieces of the adapters that its chunk meets, each into slot
// chunk + i of the partials (chunks and adapters both ascend along the list, so
// a piece's slot is its own), and a second kernel adds each adapter's slots in
// order.  t is the k of an FP32 MFMA, so both operands are read as they lie:
// rows of R 128 bits per lane, a lane's elements going to as many instructions.
// 8192 rows, both factors of bfloat16 4096 x 4096 at rank 16 (134 MB): 54 us and 7 for
// the second kernel, 2.5 TB/s; float32 6144 rows, 256 and 1024 columns: 11 and 6.
// Tried and slower: the next group's loads issued a step ahead (58 us, 15 in float32);
// waves side by side along the columns without the sum through LDS (48, but
// 10 for the second kernel's larger partials; float32 17 and 10).
constexpr int GRAD_WAVES = 4;

template <class T>
struct GradJob {
    const float *L;           // as put_s writes it
    const T *R;
    int64_t ldr, C;
    T *G;
    float *partials;
    int blocks;               // column blocks
    bool transposed;
};
template <class T>
struct GradJobs {
    GradJob<T> job[2];
    int64_t n, r, rp, CH;
    const int32_t *offs, *rows;
};

template <class T, int RB>
__global__ __launch_bounds__(64 * GRAD_WAVES) void lowrank_grad_kernel(GradJobs<T> a)
{
    constexpr int V = Elem<T>::VEC, U = 4;
    __shared__ __attribute__((aligned(16))) f32x4_t lds[GRAD_WAVES][RB][64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const bool second = (int)blockIdx.x >= a.job[0].blocks;
    const GradJob<T> &g = a.job[second ? 1 : 0];
    const int64_t C = g.C, c = (int64_t)(blockIdx.x - (second ? a.job[0].blocks : 0)) * (16 * V) + (lane & 15) * V;
    const int64_t r0 = (int64_t)blockIdx.z * (16 * RB);
    const int64_t total = a.offs[a.n], first = (int64_t)blockIdx.y * a.CH, end = lmin(first + a.CH, total);
    if (first >= end) return;
    // the adapter that holds position `first`: the last i with offs[i] <= first
    int64_t lo = 0, hi = a.n - 1;
    while (lo < hi) {
        const int64_t mid = (lo + hi + 1) >> 1;
        if (a.offs[mid] <= first) lo = mid;
        else hi = mid - 1;
    }
    const bool vec = c + V <= C;
    for (int64_t i = lo; i < a.n && a.offs[i] < end; ++i) {
        const int64_t pb = a.offs[i] > first ? a.offs[i] : first, pe = lmin(a.offs[i + 1], end);
        if (pb >= pe) continue;
        f32x4_t acc[RB][V];
#pragma unroll
        for (int b = 0; b < RB; ++b)
#pragma unroll
            for (int e = 0; e < V; ++e) acc[b][e] = f32x4_t{};
        // U groups of four rows at a time: their indices, then their loads
        for (int64_t p = pb + wave * 4; p < pe; p += GRAD_WAVES * 4 * U) {
            int64_t t[U];
            bool in[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int64_t q = p + u * GRAD_WAVES * 4 + (lane >> 4);
                in[u] = q < pe;
                t[u] = a.rows[in[u] ? q : pe - 1];
            }
            float l[U][RB], x[U][V];
#pragma unroll
            for (int u = 0; u < U; ++u) {
#pragma unroll
                for (int b = 0; b < RB; ++b) {
                    const int64_t rr = r0 + b * 16 + (lane & 15);
                    l[u][b] = get_s<T>(g.L, a.rp, t[u], rr < a.rp ? rr : 0);
                }
                const T *src = g.R + t[u] * g.ldr + c;
                if (vec) {
                    const u32x4_t v = *reinterpret_cast<const u32x4_any *>(src);
#pragma unroll
                    for (int e = 0; e < V; ++e) {
                        if constexpr (sizeof(T) == 4) x[u][e] = __uint_as_float(v[e]);
                        else x[u][e] = bf2f((uint16_t)(v[e >> 1] >> (16 * (e & 1))));
                    }
                } else {
#pragma unroll
                    for (int e = 0; e < V; ++e) x[u][e] = c + e < C ? Elem<T>::load(src + e) : 0.0f;
                }
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                // rows past the piece count zero times zero
#pragma unroll
                for (int b = 0; b < RB; ++b) l[u][b] = in[u] ? l[u][b] : 0.0f;
#pragma unroll
                for (int e = 0; e < V; ++e) x[u][e] = in[u] ? x[u][e] : 0.0f;
#pragma unroll
                for (int b = 0; b < RB; ++b)
#pragma unroll
                    for (int e = 0; e < V; ++e)
                        acc[b][e] = __builtin_amdgcn_mfma_f32_16x16x4f32(l[u][b], x[u][e], acc[b][e], 0, 0, 0);
            }
        }
        // waves in order; result (rank row 4 (lane >> 4) + k, column c + e)
        float *const part = g.partials + ((int64_t)blockIdx.y + i) * a.r * C;
#pragma unroll
        for (int e = 0; e < V; ++e) {
            __syncthreads();
#pragma unroll
            for (int b = 0; b < RB; ++b) lds[wave][b][lane] = acc[b][e];
            __syncthreads();
            for (int b = wave; b < RB; b += GRAD_WAVES) {
                f32x4_t v = lds[0][b][lane];
#pragma unroll
                for (int w = 1; w < GRAD_WAVES; ++w) v += lds[w][b][lane];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const int64_t rr = r0 + b * 16 + 4 * (lane >> 4) + k;
                    if (rr < a.r && c + e < C) part[rr * C + c + e] = v[k];
                }
            }
        }
    }
}

template <class T>
__global__ __launch_bounds__(256) void lowrank_grad_sum_kernel(GradJobs<T> a)
{
    const GradJob<T> &g = a.job[blockIdx.z];
    const int64_t i = blockIdx.y, o = (int64_t)blockIdx.x * 256 + threadIdx.x, C = g.C;
    if (o >= a.r * C) return;
    const int64_t pb = a.offs[i], pe = a.offs[i + 1];
    float v = 0.0f;
    if (pb < pe)
        for (int64_t ch = pb / a.CH; ch <= (pe - 1) / a.CH; ++ch) v += g.partials[(ch + i) * a.r * C + o];
    const int64_t rr = o / C, c = o % C;
    g.G[i * a.r * C + (g.transposed ? c * a.r + rr : o)] = Elem<T>::store(v);
}

// Rows per chunk: about four workgroups per CU over the column blocks.
int64_t grad_chunk(int64_t M, int64_t C0, int64_t C1, int64_t r, int vec, int num_cus)
{
    const int64_t blocks = ((C0 + 16 * vec - 1) / (16 * vec) + (C1 + 16 * vec - 1) / (16 * vec)) * ((r + 63) / 64);
    if (M == 0 || blocks == 0) return 16;
    int64_t chunks = (4 * (int64_t)num_cus + blocks - 1) / blocks;
    if (chunks > (M + 63) / 64) chunks = (M + 63) / 64;
    return round_up((M + chunks - 1) / chunks, 16);
}

template <class T>
hipError_t launch_lowrank_grad_t(const LowrankGrads &q, int num_cus, hipStream_t stream)
{
    constexpr int V = Elem<T>::VEC;
    GradJobs<T> a{};
    a.n = q.n; a.r = q.r; a.rp = rank_pad(q.r);
    a.offs = q.offs; a.rows = q.rows;
    int jobs = 0;
    int64_t most = 0, blocks = 0;
    const int64_t C0 = q.down ? q.K : 0, C1 = q.up ? q.N : 0;
    a.CH = grad_chunk(q.M, C0, C1, q.r, V, num_cus);
    const int64_t slots = (q.M + a.CH - 1) / a.CH + q.n;
    auto add = [&](const float *L, const void *R, int64_t ldr, int64_t C, void *G, float *partials, bool transposed) {
        GradJob<T> &g = a.job[jobs++];
        g.L = L; g.R = (const T *)R; g.ldr = ldr; g.C = C;
        g.G = (T *)G; g.partials = partials;
        g.blocks = (int)((C + 16 * V - 1) / (16 * V));
        g.transposed = transposed;
        blocks += g.blocks;
        if (C > most) most = C;
    };
    if (q.down) add(q.P, q.X, q.ldx, q.K, q.down, q.partials, false);
    if (q.up) add(q.S, q.dY, q.lddy, q.N, q.up, q.partials + slots * q.r * C0, true);
    if (jobs == 0) return hipSuccess;
    if (q.M > 0) {
        const unsigned chunks = (unsigned)((q.M + a.CH - 1) / a.CH);
        const dim3 block(64 * GRAD_WAVES);
        if (q.r <= 16)
            hipLaunchKernelGGL((lowrank_grad_kernel<T, 1>), dim3((unsigned)blocks, chunks, 1), block, 0, stream, a);
        else if (q.r <= 32)
            hipLaunchKernelGGL((lowrank_grad_kernel<T, 2>), dim3((unsigned)blocks, chunks, 1), block, 0, stream, a);
        else
            hipLaunchKernelGGL((lowrank_grad_kernel<T, 4>), dim3((unsigned)blocks, chunks, (unsigned)((q.r + 63) / 64)),
                               block, 0, stream, a);
    }
    hipLaunchKernelGGL((lowrank_grad_sum_kernel<T>),
                       dim3((unsigned)((q.r * most + 255) / 256), (unsigned)q.n, (unsigned)jobs), dim3(256), 0, stream,
                       a);
    return hipGetLastError();
}

}  // namespace

int64_t few_rows_partial_floats(int dtype, int64_t M, int64_t N, int64_t K, int gate, int num_cus)
{
    // without adapters there are at least as many slices
    if (gate < 0) return token_slices(dtype, M, N, K, 0, num_cus) * M * N;
    // a gated product with enough outputs for a workgroup per CU runs in one pass
    if (N >= (int64_t)16 * num_cus) return 0;
    const int s = token_slices(dtype, M, 2 * N, K, 0, num_cus);
    return s > 1 ? s * M * 2 * N : 0;
}

hipError_t launch_few_rows(int dtype, const FewRows &a, int num_cus, hipStream_t stream)
{
    return dtype == kF32 ? launch_few_rows_t<float>(a, num_cus, stream)
                         : launch_few_rows_t<uint16_t>(a, num_cus, stream);
}

hipError_t launch_shrink(int dtype, int64_t M, int64_t K, const void *X, int64_t ldx, const Adapters &ad, float *S,
                         int num_cus, hipStream_t stream)
{
    return dtype == kF32 ? launch_shrink_t<float>(M, K, (const float *)X, ldx, ad, S, num_cus, stream)
                         : launch_shrink_t<uint16_t>(M, K, (const uint16_t *)X, ldx, ad, S, num_cus, stream);
}

hipError_t launch_expand(int64_t M, int64_t N, const GemmEpilogue &ad, float *Y, int64_t ldy, hipStream_t stream)
{
    const dim3 grid((unsigned)((M + 63) / 64), (unsigned)((N + 127) / 128));
    hipLaunchKernelGGL(expand_kernel, grid, dim3(256), 0, stream, M, N, ad, Y, ldy);
    return hipGetLastError();
}

int64_t lowrank_grad_floats(int dtype, int64_t M, int64_t K, int64_t N, int64_t n, int64_t r, int num_cus)
{
    // the most slots of any choice of the two gradients
    const int vec = dtype == kF32 ? 4 : 8;
    int64_t most = 0;
    for (int which = 1; which < 4; ++which) {
        const int64_t C0 = which & 1 ? K : 0, C1 = which & 2 ? N : 0;
        const int64_t CH = grad_chunk(M, C0, C1, r, vec, num_cus);
        const int64_t floats = ((M + CH - 1) / CH + n) * r * (C0 + C1);
        if (floats > most) most = floats;
    }
    return most;
}

hipError_t launch_lowrank_grad(int dtype, const LowrankGrads &q, int num_cus, hipStream_t stream)
{
    return dtype == kF32 ? launch_lowrank_grad_t<float>(q, num_cus, stream)
                         : launch_lowrank_grad_t<uint16_t>(q, num_cus, stream);
}

}  // namespace sgemm_emu_dev
