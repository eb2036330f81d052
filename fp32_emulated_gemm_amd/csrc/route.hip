// route.hip -- tokens sorted by expert, and back.
//
// Sort: a counting sort that keeps the order inside an expert.  A wave takes its
// pairs 64 at a time in order; lanes of one expert find each other by a ballot per
// bit of the id, so a lane's rank among them is a population count, and the
// wave's running position of each expert lies in LDS.  Counts come first: with up
// to BLOCK pairs in the workgroup itself (one launch), with more by a launch of
// their own, behind which every workgroup adds the counts of those before it.
//
// The rest moves rows.  A unit is a piece of 2 KB of one token: it is read once
// and written to the rows of its pairs (gather), or the pairs' rows are read and
// added (combine).  Memory bounds both: 16384 tokens of 2048 bfloat16, four experts each,
// are gathered in 78 us and added up again in 75, 335 MB either way, 4.3 to 4.5 TB/s (a
// large copy on this card: 5.2); 8191 tokens of 2044, eight experts each, added with
// weights in 68, 4.4 TB/s, and its gradients (rows and weights) taken in 135 with the call,
// 4.2 TB/s.  The sort of 65536 pairs takes 5 + 7 us, of 32 pairs 4; with the call a million
// 22, 4194240 pairs 89 among 64 experts and 263 among 1024, whose counts every workgroup reads.
#include "ops_device.hpp"
#include "experts.hpp"

namespace sgemm_emu_dev {

namespace {

constexpr int SORT_THREADS = 1024, SORT_WAVES = SORT_THREADS / 64, SORT_STEPS = 4;
constexpr int SORT_BLOCK = SORT_THREADS * SORT_STEPS;      // pairs of a workgroup

struct Sort {
    int64_t P;
    int n, bits, blocks;
    const int32_t *ids;
    int32_t *offsets, *pairs, *places, *counts;            // counts: blocks x (n + 1)
};

// Pair of step s of this lane: a wave's steps are consecutive.
__device__ __forceinline__ int64_t sort_pair(int s)
{
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
    return (int64_t)blockIdx.x * SORT_BLOCK + (wave * SORT_STEPS + s) * 64 + lane;
}

// Keys of this lane's pairs: the expert, n where there is none, n + 1 past the last pair.
__device__ __forceinline__ void sort_keys(const Sort &a, int (&key)[SORT_STEPS])
{
#pragma unroll
    for (int s = 0; s < SORT_STEPS; ++s) {
        const int64_t p = sort_pair(s);
        key[s] = a.n + 1;
        if (p < a.P) {
            const int32_t id = a.ids[p];
            key[s] = id >= 0 && id < a.n ? id : a.n;
        }
    }
}

__global__ __launch_bounds__(SORT_THREADS) void sort_count_kernel(Sort a)
{
    __shared__ int32_t count[kMaxExperts + 1];
    for (int e = threadIdx.x; e <= a.n; e += SORT_THREADS) count[e] = 0;
    int key[SORT_STEPS];
    sort_keys(a, key);
    __syncthreads();
#pragma unroll
    for (int s = 0; s < SORT_STEPS; ++s)
        if (key[s] <= a.n) atomicAdd(&count[key[s]], 1);   // a count: the order of the additions does not show
    __syncthreads();
    for (int e = threadIdx.x; e <= a.n; e += SORT_THREADS) a.counts[(int64_t)blockIdx.x * (a.n + 1) + e] = count[e];
}

// ONE: the only workgroup, which counts for itself.
template <bool ONE>
__global__ __launch_bounds__(SORT_THREADS) void sort_place_kernel(Sort a)
{
    __shared__ int32_t at[SORT_WAVES][kMaxExperts + 1];    // counts of a wave, then its next position
    __shared__ int32_t sums[SORT_WAVES];
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63, n = a.n;
    for (int e = lane; e <= n; e += 64) at[wave][e] = 0;
    int key[SORT_STEPS];
    sort_keys(a, key);
    __syncthreads();
#pragma unroll
    for (int s = 0; s < SORT_STEPS; ++s)
        if (key[s] <= n) atomicAdd(&at[wave][key[s]], 1);
    __syncthreads();

    // thread e: expert e's pairs in the workgroups before this one, and in all
    const int e = threadIdx.x;
    int before = 0, all = 0;
    if (e < n) {
        if constexpr (ONE) {
#pragma unroll
            for (int w = 0; w < SORT_WAVES; ++w) all += at[w][e];
        } else {
            // loads of several workgroups' counts under way at a time
#pragma unroll 16
            for (int b = 0; b < a.blocks; ++b) {
                const int c = a.counts[(int64_t)b * (n + 1) + e];
                before += b < (int)blockIdx.x ? c : 0;
                all += c;
            }
        }
    }
    int start = all;                                       // inclusive sum over the experts
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const int v = __shfl_up(start, d);
        if (lane >= d) start += v;
    }
    if (lane == 63) sums[wave] = start;
    __syncthreads();
    int total = 0, lower = 0;
#pragma unroll
    for (int w = 0; w < SORT_WAVES; ++w) {
        lower += w < wave ? sums[w] : 0;
        total += sums[w];
    }
    start += lower - all;
    if (blockIdx.x == 0) {
        if (e < n) a.offsets[e] = start;
        if (e == 0) a.offsets[n] = total;
    }
    // each wave's first position of every expert; the pairs without one (key n) lie behind the last
    if (e < n) {
        int pos = start + before;
#pragma unroll
        for (int w = 0; w < SORT_WAVES; ++w) {
            const int c = at[w][e];
            at[w][e] = pos;
            pos += c;
        }
    }
    if (e == SORT_THREADS - 1) {
        int pos = total;
        if constexpr (!ONE)
#pragma unroll 16
            for (int b = 0; b < (int)blockIdx.x; ++b) pos += a.counts[(int64_t)b * (n + 1) + n];
#pragma unroll
        for (int w = 0; w < SORT_WAVES; ++w) {
            const int c = at[w][n];
            at[w][n] = pos;
            pos += c;
        }
    }
    __syncthreads();
    for (int s = 0; s < SORT_STEPS; ++s) {
        uint64_t same = ~0ull;
        for (int b = 0; b < a.bits; ++b) {
            const uint64_t set = __ballot((key[s] >> b) & 1);
            same &= (key[s] >> b) & 1 ? set : ~set;
        }
        const int rank = __popcll(same & ((1ull << lane) - 1));
        int pos = 0;
        if (key[s] <= n) pos = at[wave][key[s]];
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");   // every lane has read before the first one writes
        __builtin_amdgcn_wave_barrier();
        if (key[s] <= n && rank == 0) at[wave][key[s]] = pos + __popcll(same);
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
        if (key[s] <= n) {
            const int64_t p = sort_pair(s);
            pos += rank;
            a.places[p] = key[s] < n ? pos : -1;
            // ids that change while they are sorted must not lead outside
            if (pos < a.P) a.pairs[pos] = key[s] < n ? (int32_t)p : -1;
        }
    }
}

// ---------------------------------------------------------------- rows

constexpr int WAVES = 4, NT = 64 * WAVES;
constexpr int PIECES = 2;                                  // 16-byte vectors of a lane

template <class T>
struct Piece {
    static constexpr int V = Elem<T>::VEC, COLS = 64 * V * PIECES;
    u32x4_t v[PIECES];

    // Columns c0.. of a row; past K zeros.  ONCE: nobody reads them again.
    template <bool ONCE = false>
    __device__ __forceinline__ void load(const T *row, int64_t c0, int64_t K, int lane)
    {
#pragma unroll
        for (int i = 0; i < PIECES; ++i) {
            const int64_t c = c0 + (i * 64 + lane) * V;
            v[i] = u32x4_t{0, 0, 0, 0};
            if (c + V <= K) {
                const u32x4_any *const p = reinterpret_cast<const u32x4_any *>(row + c);
                v[i] = ONCE ? __builtin_nontemporal_load(p) : *p;
            } else {
                for (int e = 0; e < V; ++e)
                    if (c + e < K) {
                        if constexpr (sizeof(T) == 4) set(v[i], e, __float_as_uint(row[c + e]));
                        else set(v[i], e, row[c + e]);
                    }
            }
        }
    }
    // past: past the caches, for outputs that they would not hold until they are read.
    __device__ __forceinline__ void store(T *row, int64_t c0, int64_t K, int lane, bool past = false) const
    {
#pragma unroll
        for (int i = 0; i < PIECES; ++i) {
            const int64_t c = c0 + (i * 64 + lane) * V;
            if (c + V <= K) {
                if (past) __builtin_nontemporal_store(v[i], reinterpret_cast<u32x4_t *>(row + c));
                else *reinterpret_cast<u32x4_any *>(row + c) = v[i];
            } else {
                for (int e = 0; e < V; ++e)
                    if (c + e < K) {
                        if constexpr (sizeof(T) == 4) row[c + e] = __uint_as_float(get(v[i], e));
                        else row[c + e] = (uint16_t)get(v[i], e);
                    }
            }
        }
    }
    // Element e of a vector, without an index into registers.
    static __device__ __forceinline__ uint32_t get(const u32x4_t &q, int e)
    {
        uint32_t w = q[0];
        const int d = sizeof(T) == 4 ? e : e >> 1;
        w = d == 1 ? q[1] : w;
        w = d == 2 ? q[2] : w;
        w = d == 3 ? q[3] : w;
        return sizeof(T) == 4 ? w : (w >> (16 * (e & 1))) & 0xFFFFu;
    }
    static __device__ __forceinline__ void set(u32x4_t &q, int e, uint32_t x)
    {
        const int d = sizeof(T) == 4 ? e : e >> 1;
        const uint32_t w = sizeof(T) == 4 ? x : x << (16 * (e & 1));
#pragma unroll
        for (int i = 0; i < 4; ++i) q[i] |= d == i ? w : 0u;
    }
    __device__ __forceinline__ float f(int i, int e) const
    {
        if constexpr (sizeof(T) == 4) return __uint_as_float(v[i][e]);
        else return __uint_as_float(e & 1 ? v[i][e >> 1] & 0xFFFF0000u : v[i][e >> 1] << 16);
    }
    __device__ __forceinline__ void put(const float (&f)[PIECES][V])
    {
#pragma unroll
        for (int i = 0; i < PIECES; ++i) {
            if constexpr (sizeof(T) == 4) {
#pragma unroll
                for (int e = 0; e < 4; ++e) v[i][e] = __float_as_uint(f[i][e]);
            } else {
#pragma unroll
                for (int e = 0; e < 4; ++e) v[i][e] = pack2(f[i][2 * e], f[i][2 * e + 1]);
            }
        }
    }
};

// Rows from offsets[n] on belong to no expert: zeros, a row for each of the
// launch's units in turn.
template <class T>
__device__ __forceinline__ void clear_rest(const Route<T> &a, T *rows, int64_t ld, int64_t unit, int64_t units,
                                           int64_t c0, int64_t c1, int lane)
{
    const int64_t last = a.offsets[a.n];
    Piece<T> zero;
#pragma unroll
    for (int i = 0; i < PIECES; ++i) zero.v[i] = u32x4_t{0, 0, 0, 0};
    for (int64_t r = (last < 0 ? 0 : last) + unit; r < a.P; r += units)
        for (int64_t c = c0; c < c1; c += Piece<T>::COLS) zero.store(rows + r * ld, c, a.K, lane, a.past);
}

template <class T>
__global__ __launch_bounds__(NT) void gather_kernel(Route<T> a)
{
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t t = (int64_t)blockIdx.x * WAVES + wave, c0 = (int64_t)blockIdx.y * Piece<T>::COLS;
    if (t >= a.tokens) return;
    Piece<T> x;
    x.load(a.x + t * a.ldx, c0, a.K, lane);
    const int32_t *const place = a.places + t * a.k;
    for (int64_t j = 0; j < a.k; ++j) {
        const int64_t r = place[j];
        if (r >= 0 && r < a.P) x.store(a.rows_out + r * a.ldr_out, c0, a.K, lane, a.past);
    }
    clear_rest(a, a.rows_out, a.ldr_out, t, a.tokens, c0, c0 + 1, lane);
}

constexpr int AT_ONCE = 4;                                 // rows of a token in flight

template <class T, bool WEIGHTS>
__global__ __launch_bounds__(NT) void combine_kernel(Route<T> a)
{
    constexpr int V = Piece<T>::V;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t t = (int64_t)blockIdx.x * WAVES + wave, c0 = (int64_t)blockIdx.y * Piece<T>::COLS;
    if (t >= a.tokens) return;
    const int32_t *const place = a.places + t * a.k;
    float acc[PIECES][V];
#pragma unroll
    for (int i = 0; i < PIECES; ++i)
#pragma unroll
        for (int e = 0; e < V; ++e) acc[i][e] = 0.0f;
    for (int64_t j0 = 0; j0 < a.k; j0 += AT_ONCE) {
        Piece<T> y[AT_ONCE];
        float w[AT_ONCE];
        bool in[AT_ONCE];
#pragma unroll
        for (int q = 0; q < AT_ONCE; ++q) {
            const int64_t r = j0 + q < a.k ? place[j0 + q] : -1;
            in[q] = r >= 0 && r < a.P;
            if (in[q]) {
                y[q].template load<true>(a.rows + r * a.ldr, c0, a.K, lane);
                w[q] = WEIGHTS ? a.weights[t * a.k + j0 + q] : 1.0f;
            }
        }
#pragma unroll
        for (int q = 0; q < AT_ONCE; ++q)
            if (in[q]) {
#pragma unroll
                for (int i = 0; i < PIECES; ++i)
#pragma unroll
                    for (int e = 0; e < V; ++e)
                        acc[i][e] = WEIGHTS ? __builtin_fmaf(w[q], y[q].f(i, e), acc[i][e]) : acc[i][e] + y[q].f(i, e);
            }
    }
    Piece<T> out;
    out.put(acc);
    out.store(a.x_out + t * a.ldx_out, c0, a.K, lane, a.past);
}

// One wave per pair: the token's gradient is read once from memory and by its
// other pairs, mostly of the same workgroup, from the caches.
template <class T, bool WEIGHTS>
__global__ __launch_bounds__(NT) void combine_backward_kernel(Route<T> a)
{
    constexpr int V = Piece<T>::V;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t p = (int64_t)blockIdx.x * WAVES + wave;
    if (p >= a.P) return;
    const int64_t t = p / a.k, r = a.places[p];
    const bool in = r >= 0 && r < a.P;
    float dot = 0.0f;
    if (in) {
        const float w = WEIGHTS ? a.weights[p] : 1.0f;
        for (int64_t c0 = 0; c0 < a.K; c0 += Piece<T>::COLS) {
            Piece<T> dy, y;
            dy.load(a.x + t * a.ldx, c0, a.K, lane);
            if (a.dweights != nullptr) y.load(a.rows + r * a.ldr, c0, a.K, lane);
            float g[PIECES][V];
#pragma unroll
            for (int i = 0; i < PIECES; ++i)
#pragma unroll
                for (int e = 0; e < V; ++e) g[i][e] = dy.f(i, e);
            if (a.dweights != nullptr) {
#pragma unroll
                for (int i = 0; i < PIECES; ++i)
#pragma unroll
                    for (int e = 0; e < V; ++e) dot = __builtin_fmaf(g[i][e], y.f(i, e), dot);
            }
            if (a.rows_out != nullptr) {
#pragma unroll
                for (int i = 0; i < PIECES; ++i)
#pragma unroll
                    for (int e = 0; e < V; ++e) g[i][e] *= w;
                dy.put(g);
                dy.store(a.rows_out + r * a.ldr_out, c0, a.K, lane, a.past);
            }
        }
    }
    if (a.dweights != nullptr) {
#pragma unroll
        for (int d = 32; d > 0; d >>= 1) dot += __shfl_xor(dot, d);
        if (lane == 0) a.dweights[p] = dot;
    }
    if (a.rows_out != nullptr) clear_rest(a, a.rows_out, a.ldr_out, p, a.P, 0, a.K, lane);
}

template <class T>
dim3 token_grid(const Route<T> &a)
{
    return dim3((unsigned)((a.tokens + WAVES - 1) / WAVES), (unsigned)((a.K + Piece<T>::COLS - 1) / Piece<T>::COLS));
}

// With sorted rows of more than half of the last-level cache (256 MB) outputs go past
// it: what was written first would be gone before the next kernel reads it, and its
// way out competes with reads (65536 x 2048 bfloat16 gathered, then as many summed:
// 187 us in all, 161 past the caches).  Rows of whole 16-byte pieces only: others
// would be stored element by element.
template <class T>
hipError_t route(int what, const Route<T> &args, hipStream_t stream)
{
    Route<T> a = args;
    const void *const to = what == kCombine ? (const void *)a.x_out : a.rows_out;
    const int64_t ld = what == kCombine ? a.ldx_out : a.ldr_out;
    a.past = a.P * a.K * (int64_t)sizeof(T) > (int64_t)128 << 20 && ld * (int64_t)sizeof(T) % 16 == 0 && aligned(to, 16);
    if (a.tokens == 0 || a.K == 0) return hipSuccess;
    const bool w = a.weights != nullptr;
    const dim3 tokens = token_grid(a), pairs((unsigned)((a.P + WAVES - 1) / WAVES));
    switch (what) {
    case kGather: hipLaunchKernelGGL(gather_kernel<T>, tokens, dim3(NT), 0, stream, a); break;
    case kCombine:
        if (w) hipLaunchKernelGGL((combine_kernel<T, true>), tokens, dim3(NT), 0, stream, a);
        else hipLaunchKernelGGL((combine_kernel<T, false>), tokens, dim3(NT), 0, stream, a);
        break;
    default:
        if (a.P == 0) return hipSuccess;
        if (w) hipLaunchKernelGGL((combine_backward_kernel<T, true>), pairs, dim3(NT), 0, stream, a);
        else hipLaunchKernelGGL((combine_backward_kernel<T, false>), pairs, dim3(NT), 0, stream, a);
    }
    return hipGetLastError();
}

__global__ __launch_bounds__(256) void clear_floats_kernel(float *p, int64_t n)
{
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256) p[i] = 0.0f;
}

}  // namespace

int64_t sort_counts(int64_t P, int64_t n)
{
    return P <= SORT_BLOCK ? 0 : (P + SORT_BLOCK - 1) / SORT_BLOCK * (n + 1);
}

hipError_t launch_sort(int64_t P, int64_t n, const int32_t *ids, int32_t *offsets, int32_t *pairs, int32_t *places,
                       int32_t *counts, hipStream_t stream)
{
    Sort a{P, (int)n, 0, (int)(P <= SORT_BLOCK ? 1 : (P + SORT_BLOCK - 1) / SORT_BLOCK), ids, offsets, pairs, places,
           counts};
    while ((n + 1) >> a.bits) ++a.bits;
    if (a.blocks == 1) {
        hipLaunchKernelGGL(sort_place_kernel<true>, dim3(1), dim3(SORT_THREADS), 0, stream, a);
    } else {
        hipLaunchKernelGGL(sort_count_kernel, dim3((unsigned)a.blocks), dim3(SORT_THREADS), 0, stream, a);
        hipLaunchKernelGGL(sort_place_kernel<false>, dim3((unsigned)a.blocks), dim3(SORT_THREADS), 0, stream, a);
    }
    return hipGetLastError();
}

hipError_t launch_route(int what, const Route<float> &a, hipStream_t stream) { return route(what, a, stream); }
hipError_t launch_route(int what, const Route<uint16_t> &a, hipStream_t stream) { return route(what, a, stream); }

hipError_t launch_clear_floats(float *p, int64_t n, hipStream_t stream)
{
    if (n == 0) return hipSuccess;
    const int64_t blocks = (n + 255) / 256;
    hipLaunchKernelGGL(clear_floats_kernel, dim3((unsigned)(blocks < 4096 ? blocks : 4096)), dim3(256), 0, stream, p, n);
    return hipGetLastError();
}

}  // namespace sgemm_emu_dev
