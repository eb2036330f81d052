// lowrank.hip -- few-row products and the low-rank parts of the adapters.
//
// dot_tile, shared by the few-row product and the shrink: a workgroup's eight
// waves split K; each reads rows of both operands straight into the fragments
// of a 16 x 16 MFMA (128 bits of consecutive k per lane, four lanes of a row in
// one 64-byte segment, two segments per wave and step), and the waves' sums are
// added through LDS in wave order.  There is no reuse to stage: with few rows
// of X the weight passes once, and the time is its bytes'.
// FP32 operands take the FP32 matrix instruction (FP32 products, FP32 sums): a
// lane's four consecutive k are the k of four instructions, the same for both
// operands, so their order inside a step does not matter.
#include "ops_device.hpp"
#include "ops.hpp"

namespace sgemm_emu_dev {

namespace {

constexpr int WAVES = 8;                         // of a dot_tile workgroup

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

// VEC elements of a row from k on, zeros past K.  ALIGNED: rows are 16-byte
// aligned and K is a multiple of VEC, so a load is whole or empty.
template <class T, bool ALIGNED>
__device__ __forceinline__ u32x4_t load_k(const T *row, int64_t k, int64_t K)
{
    constexpr int V = Elem<T>::VEC;
    u32x4_t v = {0, 0, 0, 0};
    if constexpr (ALIGNED) {
        if (k < K) v = *reinterpret_cast<const u32x4_t *>(row + k);
    } else if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int e = 0; e < V; ++e)
            if (k + e < K) v[e] = __float_as_uint(row[k + e]);
    } else {
#pragma unroll
        for (int e = 0; e < V; ++e)
            if (k + e < K) v[e >> 1] |= (uint32_t)row[k + e] << (16 * (e & 1));
    }
    return v;
}

// acc[nb][mb] += rows of W (w[nb], 16 per block) times rows of X (x[mb]) over
// this wave's share of K: lane l holds row l & 15 of each block.
template <class T, int NB, int MB, bool AW, bool AX>
__device__ __forceinline__ void dot_tile(f32x4_t (&acc)[NB][MB], const T *const (&w)[NB], const T *const (&x)[MB],
                                         int64_t K, int wave, int lane)
{
    constexpr int V = Elem<T>::VEC, STEP = 8 * V, U = 2;
    const int64_t first = (int64_t)wave * STEP + (lane >> 4) * V;
    for (int64_t k = first; k - first + wave * STEP < K; k += (int64_t)WAVES * STEP) {
        u32x4_t fw[U][NB], fx[U][MB];
#pragma unroll
        for (int u = 0; u < U; ++u) {
#pragma unroll
            for (int nb = 0; nb < NB; ++nb) fw[u][nb] = load_k<T, AW>(w[nb], k + u * 4 * V, K);
#pragma unroll
            for (int mb = 0; mb < MB; ++mb) fx[u][mb] = load_k<T, AX>(x[mb], k + u * 4 * V, K);
        }
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                for (int mb = 0; mb < MB; ++mb) acc[nb][mb] = mfma16<T>(fw[u][nb], fx[u][mb], acc[nb][mb]);
    }
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

// ---------------------------------------------------------------- few rows

// GATE < 0: NB blocks of 16 rows of W; else NB / 2 blocks of gate rows, then
// the NB / 2 blocks of up rows of the same outputs.
template <class T, int NB, int MB, int GATE, bool AW, bool AX>
__global__ __launch_bounds__(64 * WAVES) void few_rows_kernel(FewRows a, Adapters ad)
{
    __shared__ __attribute__((aligned(16))) float lds[WAVES * NB * MB * 256];
    constexpr int OUT = (GATE < 0 ? NB : NB / 2) * 16;              // outputs per row of the workgroup
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t n0 = (int64_t)blockIdx.x * OUT, m0 = (int64_t)blockIdx.y * (16 * MB);
    const T *W = (const T *)a.W, *X = (const T *)a.X;
    const T *w[NB], *x[MB];
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
        const int b = GATE < 0 ? nb : nb % (NB / 2);
        int64_t row = lmin(n0 + b * 16 + (lane & 15), a.N - 1);
        if (GATE >= 0 && nb >= NB / 2) row += a.N;
        w[nb] = W + row * a.ldw;
    }
#pragma unroll
    for (int mb = 0; mb < MB; ++mb) x[mb] = X + lmin(m0 + mb * 16 + (lane & 15), a.M - 1) * a.ldx;
    f32x4_t acc[NB][MB];
#pragma unroll
    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
        for (int mb = 0; mb < MB; ++mb) acc[nb][mb] = f32x4_t{};
    dot_tile<T, NB, MB, AW, AX>(acc, w, x, a.K, wave, lane);
    put_sums<NB, MB>(lds, acc, wave, lane);
    __syncthreads();
    const T *bias = (const T *)a.bias;
    T *Y = (T *)a.Y;
    for (int o = threadIdx.x; o < OUT * 16 * MB; o += 64 * WAVES) {
        const int n = o % OUT, m = o / OUT;
        if (n0 + n >= a.N || m0 + m >= a.M) continue;
        float v = get_sum<NB, MB>(lds, n, m);
        if (bias != nullptr) v += Elem<T>::load(bias + n0 + n);
        if constexpr (GATE >= 0) {
            float u = get_sum<NB, MB>(lds, OUT + n, m);
            if (bias != nullptr) u += Elem<T>::load(bias + a.N + n0 + n);
            v = gate_act<GATE>(v) * u;
        } else if (a.S != nullptr) {
            const int32_t i = ad.ids[m0 + m];
            if (i >= 0 && i < ad.n) {
                const T *up = (const T *)ad.up + ((int64_t)i * a.N + n0 + n) * ad.r;
                const float *s = a.S + (m0 + m) * ((ad.r + 15) / 16 * 16);
                float d = 0.0f;
                for (int64_t j = 0; j < ad.r; ++j) d = __builtin_fmaf(s[j], Elem<T>::load(up + j), d);
                v += d;
            }
        }
        Y[(m0 + m) * a.ldy + n0 + n] = Elem<T>::store(v);
    }
}

template <class T, int NB, int MB, int GATE>
void launch_few_rows_al(const FewRows &a, hipStream_t stream)
{
    constexpr int OUT = (GATE < 0 ? NB : NB / 2) * 16, V = Elem<T>::VEC;
    const dim3 grid((unsigned)((a.N + OUT - 1) / OUT), (unsigned)((a.M + 16 * MB - 1) / (16 * MB)));
    const bool aw = a.K % V == 0 && a.ldw % V == 0 && aligned(a.W, 16);
    const bool ax = a.K % V == 0 && a.ldx % V == 0 && aligned(a.X, 16);
    const Adapters ad = a.ad != nullptr ? *a.ad : Adapters{};
    const dim3 block(64 * WAVES);
    if (aw && ax) hipLaunchKernelGGL((few_rows_kernel<T, NB, MB, GATE, true, true>), grid, block, 0, stream, a, ad);
    else if (aw) hipLaunchKernelGGL((few_rows_kernel<T, NB, MB, GATE, true, false>), grid, block, 0, stream, a, ad);
    else hipLaunchKernelGGL((few_rows_kernel<T, NB, MB, GATE, false, false>), grid, block, 0, stream, a, ad);
}

template <class T, int NB, int GATE>
void launch_few_rows_mb(const FewRows &a, hipStream_t stream)
{
    if (a.M <= 16) launch_few_rows_al<T, NB, 1, GATE>(a, stream);
    else if (a.M <= 32) launch_few_rows_al<T, NB, 2, GATE>(a, stream);
    else launch_few_rows_al<T, NB, 4, GATE>(a, stream);
}

template <class T, int GATE>
void launch_few_rows_nb(const FewRows &a, int num_cus, hipStream_t stream)
{
    if constexpr (GATE >= 0) {
        if (a.N >= (int64_t)32 * num_cus) launch_few_rows_mb<T, 4, GATE>(a, stream);
        else launch_few_rows_mb<T, 2, GATE>(a, stream);
    } else {
        if (a.N >= (int64_t)64 * num_cus) launch_few_rows_mb<T, 4, GATE>(a, stream);
        else if (a.N >= (int64_t)32 * num_cus) launch_few_rows_mb<T, 2, GATE>(a, stream);
        else launch_few_rows_mb<T, 1, GATE>(a, stream);
    }
}

template <class T>
hipError_t launch_few_rows_t(const FewRows &a, int num_cus, hipStream_t stream)
{
    switch (a.gate) {
    case kSilu: launch_few_rows_nb<T, kSilu>(a, num_cus, stream); break;
    case kGelu: launch_few_rows_nb<T, kGelu>(a, num_cus, stream); break;
    case kGeluTanh: launch_few_rows_nb<T, kGeluTanh>(a, num_cus, stream); break;
    case kSigmoid: launch_few_rows_nb<T, kSigmoid>(a, num_cus, stream); break;
    case kRelu: launch_few_rows_nb<T, kRelu>(a, num_cus, stream); break;
    default: launch_few_rows_nb<T, -1>(a, num_cus, stream);
    }
    return hipGetLastError();
}

// ---------------------------------------------------------------- shrink
// S[t] = scale[i] down[i] X[t].  A workgroup takes 16 MB rows and walks the
// adapters that occur in them (ascending ids): each pass multiplies all the
// tile's rows by that adapter's r rows and keeps the rows that belong to it.
// Rows of one request are neighbours, so a tile of a prompt holds one or two
// adapters; gridDim.y workgroups share a tile's adapters where every row may
// have its own (single tokens).
template <class T, int NB, int MB, bool AL>
__global__ __launch_bounds__(64 * WAVES) void shrink_kernel(int64_t M, int64_t K, const T *X, int64_t ldx, Adapters ad,
                                                            float *S, int64_t rp)
{
    __shared__ __attribute__((aligned(16))) float lds[WAVES * NB * MB * 256];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t m0 = (int64_t)blockIdx.x * (16 * MB);
    constexpr int ROWS = 16 * MB;
    int id = -1;
    if (lane < ROWS && m0 + lane < M) {
        const int v = ad.ids[m0 + lane];
        id = v >= 0 && v < ad.n ? v : -1;
    }
    const T *x[MB];
#pragma unroll
    for (int mb = 0; mb < MB; ++mb) x[mb] = X + lmin(m0 + mb * 16 + (lane & 15), M - 1) * ldx;

    if (blockIdx.y == 0) {
        // rows without an adapter
        for (int64_t o = threadIdx.x; o < ROWS * rp; o += 64 * WAVES) {
            const int64_t m = m0 + o / rp;
            if (m < M) {
                const int v = ad.ids[m];
                if (!(v >= 0 && v < ad.n)) S[m * rp + o % rp] = 0.0f;
            }
        }
    }
    int last = -1;
    for (unsigned slot = 0;; ++slot) {
        int next = id > last ? id : 0x7FFFFFFF;
#pragma unroll
        for (int s = 1; s < 64; s <<= 1) next = imin(next, __shfl_xor(next, s));
        next = __builtin_amdgcn_readfirstlane(next);
        if (next == 0x7FFFFFFF) break;
        last = next;
        if (slot % gridDim.y != blockIdx.y) continue;
        const T *down = (const T *)ad.down + (int64_t)next * ad.r * K;
        const float scale = ad.scale != nullptr ? ad.scale[next] : 1.0f;
        for (int64_t r0 = 0; r0 < rp; r0 += 16 * NB) {
            const T *w[NB];
#pragma unroll
            for (int nb = 0; nb < NB; ++nb) w[nb] = down + lmin(r0 + nb * 16 + (lane & 15), ad.r - 1) * K;
            f32x4_t acc[NB][MB];
#pragma unroll
            for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                for (int mb = 0; mb < MB; ++mb) acc[nb][mb] = f32x4_t{};
            dot_tile<T, NB, MB, AL, AL>(acc, w, x, K, wave, lane);
            put_sums<NB, MB>(lds, acc, wave, lane);
            __syncthreads();
            for (int o = threadIdx.x; o < 16 * NB * ROWS; o += 64 * WAVES) {
                const int n = o % (16 * NB), m = o / (16 * NB);
                if (m0 + m < M && r0 + n < rp && ad.ids[m0 + m] == next)
                    S[(m0 + m) * rp + r0 + n] = r0 + n < ad.r ? scale * get_sum<NB, MB>(lds, n, m) : 0.0f;
            }
            __syncthreads();
        }
    }
}

template <class T, int NB, int MB>
void launch_shrink_mb(int64_t M, int64_t K, const T *X, int64_t ldx, const Adapters &ad, float *S, bool few,
                      hipStream_t stream)
{
    constexpr int V = Elem<T>::VEC;
    const dim3 grid((unsigned)((M + 16 * MB - 1) / (16 * MB)), few ? 16 * MB : 1);
    const bool al = K % V == 0 && ldx % V == 0 && aligned(X, 16) && aligned(ad.down, 16);
    if (al)
        hipLaunchKernelGGL((shrink_kernel<T, NB, MB, true>), grid, dim3(64 * WAVES), 0, stream, M, K, X, ldx, ad, S,
                           rank_pad(ad.r));
    else
        hipLaunchKernelGGL((shrink_kernel<T, NB, MB, false>), grid, dim3(64 * WAVES), 0, stream, M, K, X, ldx, ad, S,
                           rank_pad(ad.r));
}

template <class T, int NB>
void launch_shrink_nb(int64_t M, int64_t K, const T *X, int64_t ldx, const Adapters &ad, float *S, hipStream_t stream)
{
    // every row of a small batch may have its own adapter: one workgroup each
    if (M <= 256) launch_shrink_mb<T, NB, 1>(M, K, X, ldx, ad, S, true, stream);
    else launch_shrink_mb<T, NB, 2>(M, K, X, ldx, ad, S, false, stream);
}

template <class T>
hipError_t launch_shrink_t(int64_t M, int64_t K, const T *X, int64_t ldx, const Adapters &ad, float *S,
                           hipStream_t stream)
{
    if (ad.r <= 16) launch_shrink_nb<T, 1>(M, K, X, ldx, ad, S, stream);
    else if (ad.r <= 32) launch_shrink_nb<T, 2>(M, K, X, ldx, ad, S, stream);
    else launch_shrink_nb<T, 4>(M, K, X, ldx, ad, S, stream);
    return hipGetLastError();
}

// ---------------------------------------------------------------- expand

template <class T>
__global__ __launch_bounds__(256) void expand_kernel(int64_t M, int64_t N, const float *S, int64_t rp, Adapters ad,
                                                     T *Y, int64_t ldy)
{
    for (int64_t m = blockIdx.y; m < M; m += gridDim.y) {
        const int32_t i = ad.ids[m];
        const int64_t n = (int64_t)blockIdx.x * 256 + threadIdx.x;
        if (!(i >= 0 && i < ad.n) || n >= N) continue;
        const T *up = (const T *)ad.up + ((int64_t)i * N + n) * ad.r;
        float d = 0.0f;
        for (int64_t j = 0; j < ad.r; ++j) d = __builtin_fmaf(S[m * rp + j], Elem<T>::load(up + j), d);
        Y[m * ldy + n] = Elem<T>::store(Elem<T>::load(Y + m * ldy + n) + d);
    }
}

// ---------------------------------------------------------------- grouping rows by adapter
// Workgroup i lists the rows of adapter i, ascending: it counts the ids below
// its own (where its rows start) and its own, then writes its rows in order
// (ballots and a prefix over the waves).  No atomics: the order, and with it
// the gradients' order of additions, is fixed.
constexpr int GROUP_NT = 1024;
__global__ __launch_bounds__(GROUP_NT) void group_kernel(int64_t M, const int32_t *ids, int64_t n, int32_t *offs,
                                                         int32_t *rows)
{
    __shared__ int32_t less_sum[GROUP_NT / 64], own_sum[GROUP_NT / 64], found[GROUP_NT / 64];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int32_t me = (int32_t)blockIdx.x;
    int32_t less = 0, own = 0;
    for (int64_t t = tid; t < M; t += GROUP_NT) {
        const int32_t v = ids[t];
        less += v >= 0 && v < me;
        own += v == me;
    }
#pragma unroll
    for (int s = 1; s < 64; s <<= 1) {
        less += __shfl_xor(less, s);
        own += __shfl_xor(own, s);
    }
    if (lane == 0) { less_sum[wave] = less; own_sum[wave] = own; }
    __syncthreads();
    int32_t at = 0, mine = 0;
    for (int w = 0; w < GROUP_NT / 64; ++w) { at += less_sum[w]; mine += own_sum[w]; }
    if (tid == 0) {
        offs[me] = at;
        if (me == n - 1) offs[n] = at + mine;
    }
    if (mine == 0) return;
    for (int64_t base = 0; base < M; base += GROUP_NT) {
        const int64_t t = base + tid;
        const bool hit = t < M && ids[t] == me;
        const uint64_t mask = __ballot(hit);
        if (lane == 0) found[wave] = __popcll(mask);
        __syncthreads();
        int32_t before = 0, all = 0;
        for (int w = 0; w < GROUP_NT / 64; ++w) {
            before += w < wave ? found[w] : 0;
            all += found[w];
        }
        if (hit) rows[at + before + __popcll(mask & ((1ull << lane) - 1))] = (int32_t)t;
        at += all;
        __syncthreads();
    }
}

// ---------------------------------------------------------------- gradients of the low-rank factors
// G[i] = sum over adapter i's rows t of L[t] (x) R[t] (r x C).  The rows,
// grouped by adapter (group_kernel), are cut into chunks of CH; workgroup
// (column block, chunk) sums the pieces of the adapters that its chunk meets,
// each into slot chunk + i of the partials (chunks and adapters both ascend
// along the list, so a piece's slot is its own), and a second kernel adds each
// adapter's slots in order.  t is the k of an FP32 MFMA, so both operands are
// read as they lie: rows of R 128 bits per lane, a lane's elements going to as
// many instructions.
constexpr int GRAD_WAVES = 4;

template <class T, int RB>
__global__ __launch_bounds__(64 * GRAD_WAVES) void lowrank_grad_kernel(int64_t C, int64_t n, int64_t r, int64_t rp,
                                                                       const float *L, const T *R, int64_t ldr,
                                                                       bool vec, const int32_t *offs,
                                                                       const int32_t *rows, int64_t CH,
                                                                       float *partials)
{
    constexpr int V = Elem<T>::VEC;
    __shared__ __attribute__((aligned(16))) f32x4_t lds[GRAD_WAVES][RB][64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t c = (int64_t)blockIdx.x * (16 * V) + (lane & 15) * V, r0 = (int64_t)blockIdx.z * (16 * RB);
    const int64_t total = offs[n], first = (int64_t)blockIdx.y * CH, end = lmin(first + CH, total);
    if (first >= end) return;
    // the adapter that holds position `first`: the last i with offs[i] <= first
    int64_t lo = 0, hi = n - 1;
    while (lo < hi) {
        const int64_t mid = (lo + hi + 1) >> 1;
        if (offs[mid] <= first) lo = mid;
        else hi = mid - 1;
    }
    for (int64_t i = lo; i < n && offs[i] < end; ++i) {
        const int64_t pb = offs[i] > first ? offs[i] : first, pe = lmin(offs[i + 1], end);
        if (pb >= pe) continue;
        f32x4_t acc[RB][V];
#pragma unroll
        for (int b = 0; b < RB; ++b)
#pragma unroll
            for (int e = 0; e < V; ++e) acc[b][e] = f32x4_t{};
        for (int64_t p = pb + wave * 4; p < pe; p += GRAD_WAVES * 4) {
            const int64_t q = p + (lane >> 4);
            float l[RB], x[V];
#pragma unroll
            for (int b = 0; b < RB; ++b) l[b] = 0.0f;
#pragma unroll
            for (int e = 0; e < V; ++e) x[e] = 0.0f;
            if (q < pe) {
                const int64_t t = rows[q];
#pragma unroll
                for (int b = 0; b < RB; ++b) {
                    const int64_t rr = r0 + b * 16 + (lane & 15);
                    if (rr < rp) l[b] = L[t * rp + rr];
                }
                const T *src = R + t * ldr + c;
                if (vec && c + V <= C) {
                    const u32x4_t v = *reinterpret_cast<const u32x4_t *>(src);
#pragma unroll
                    for (int e = 0; e < V; ++e) {
                        if constexpr (sizeof(T) == 4) x[e] = __uint_as_float(v[e]);
                        else x[e] = bf2f((uint16_t)(v[e >> 1] >> (16 * (e & 1))));
                    }
                } else {
#pragma unroll
                    for (int e = 0; e < V; ++e)
                        if (c + e < C) x[e] = Elem<T>::load(src + e);
                }
            }
#pragma unroll
            for (int b = 0; b < RB; ++b)
#pragma unroll
                for (int e = 0; e < V; ++e)
                    acc[b][e] = __builtin_amdgcn_mfma_f32_16x16x4f32(l[b], x[e], acc[b][e], 0, 0, 0);
        }
        // waves in order; result (rank row 4 (lane >> 4) + k, column c + e)
        float *const part = partials + ((int64_t)blockIdx.y + i) * r * C;
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
                    if (rr < r && c + e < C) part[rr * C + c + e] = v[k];
                }
            }
        }
    }
}

template <class T>
__global__ __launch_bounds__(256) void lowrank_grad_sum_kernel(int64_t C, int64_t r, const int32_t *offs, int64_t CH,
                                                               const float *partials, bool transposed, T *G)
{
    const int64_t i = blockIdx.y, o = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (o >= r * C) return;
    const int64_t pb = offs[i], pe = offs[i + 1];
    float v = 0.0f;
    if (pb < pe)
        for (int64_t ch = pb / CH; ch <= (pe - 1) / CH; ++ch) v += partials[(ch + i) * r * C + o];
    const int64_t rr = o / C, c = o % C;
    G[i * r * C + (transposed ? c * r + rr : o)] = Elem<T>::store(v);
}

int64_t grad_chunk(int64_t M, int64_t C, int64_t r, int vec, int num_cus)
{
    if (M == 0 || C == 0) return 16;
    const int64_t blocks = ((C + 16 * vec - 1) / (16 * vec)) * ((r + 63) / 64);
    int64_t chunks = (4 * (int64_t)num_cus + blocks - 1) / blocks;
    if (chunks > (M + 63) / 64) chunks = (M + 63) / 64;
    return round_up((M + chunks - 1) / chunks, 16);
}

template <class T>
hipError_t launch_lowrank_grad_t(int64_t M, int64_t C, int64_t n, int64_t r, const float *L, const T *R, int64_t ldr,
                                 const int32_t *offs, const int32_t *rows, bool transposed, T *G, float *partials,
                                 int num_cus, hipStream_t stream)
{
    constexpr int V = Elem<T>::VEC;
    const int64_t CH = grad_chunk(M, C, r, V, num_cus), chunks = (M + CH - 1) / CH, rp = rank_pad(r);
    const bool vec = ldr % V == 0 && aligned(R, 16);
    const unsigned cb = (unsigned)((C + 16 * V - 1) / (16 * V));
    const dim3 block(64 * GRAD_WAVES);
    if (M > 0) {
        if (r <= 16)
            hipLaunchKernelGGL((lowrank_grad_kernel<T, 1>), dim3(cb, (unsigned)chunks, 1), block, 0, stream, C, n, r,
                               rp, L, R, ldr, vec, offs, rows, CH, partials);
        else if (r <= 32)
            hipLaunchKernelGGL((lowrank_grad_kernel<T, 2>), dim3(cb, (unsigned)chunks, 1), block, 0, stream, C, n, r,
                               rp, L, R, ldr, vec, offs, rows, CH, partials);
        else
            hipLaunchKernelGGL((lowrank_grad_kernel<T, 4>), dim3(cb, (unsigned)chunks, (unsigned)((r + 63) / 64)),
                               block, 0, stream, C, n, r, rp, L, R, ldr, vec, offs, rows, CH, partials);
    }
    hipLaunchKernelGGL((lowrank_grad_sum_kernel<T>), dim3((unsigned)((r * C + 255) / 256), (unsigned)n), dim3(256), 0,
                       stream, C, r, offs, CH, partials, transposed, G);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_few_rows(int dtype, const FewRows &a, int num_cus, hipStream_t stream)
{
    return dtype == kF32 ? launch_few_rows_t<float>(a, num_cus, stream)
                         : launch_few_rows_t<uint16_t>(a, num_cus, stream);
}

hipError_t launch_shrink(int dtype, int64_t M, int64_t K, const void *X, int64_t ldx, const Adapters &ad, float *S,
                         int num_cus, hipStream_t stream)
{
    (void)num_cus;
    return dtype == kF32 ? launch_shrink_t<float>(M, K, (const float *)X, ldx, ad, S, stream)
                         : launch_shrink_t<uint16_t>(M, K, (const uint16_t *)X, ldx, ad, S, stream);
}

hipError_t launch_expand(int dtype, int64_t M, int64_t N, const float *S, const Adapters &ad, void *Y, int64_t ldy,
                         int num_cus, hipStream_t stream)
{
    (void)num_cus;
    const dim3 grid((unsigned)((N + 255) / 256), (unsigned)(M < 32768 ? M : 32768));
    if (dtype == kF32)
        hipLaunchKernelGGL((expand_kernel<float>), grid, dim3(256), 0, stream, M, N, S, rank_pad(ad.r), ad, (float *)Y,
                           ldy);
    else
        hipLaunchKernelGGL((expand_kernel<uint16_t>), grid, dim3(256), 0, stream, M, N, S, rank_pad(ad.r), ad,
                           (uint16_t *)Y, ldy);
    return hipGetLastError();
}

hipError_t launch_group(int64_t M, const int32_t *ids, int64_t n, int32_t *offs, int32_t *rows, hipStream_t stream)
{
    hipLaunchKernelGGL(group_kernel, dim3((unsigned)n), dim3(GROUP_NT), 0, stream, M, ids, n, offs, rows);
    return hipGetLastError();
}

int64_t lowrank_grad_floats(int64_t M, int64_t C, int64_t n, int64_t r, int num_cus)
{
    // the chunk of either type's column blocks, whichever makes more slots
    const int64_t a = grad_chunk(M, C, r, 4, num_cus), b = grad_chunk(M, C, r, 8, num_cus);
    const int64_t CH = a < b ? a : b;
    return ((M + CH - 1) / CH + n) * r * C;
}

hipError_t launch_lowrank_grad(int dtype, int64_t M, int64_t C, int64_t n, int64_t r, const float *L, const void *R,
                               int64_t ldr, const int32_t *offs, const int32_t *rows, bool transposed, void *G,
                               float *partials, int num_cus, hipStream_t stream)
{
    if (dtype == kF32)
        return launch_lowrank_grad_t<float>(M, C, n, r, L, (const float *)R, ldr, offs, rows, transposed, (float *)G,
                                            partials, num_cus, stream);
    return launch_lowrank_grad_t<uint16_t>(M, C, n, r, L, (const uint16_t *)R, ldr, offs, rows, transposed,
                                           (uint16_t *)G, partials, num_cus, stream);
}

}  // namespace sgemm_emu_dev
