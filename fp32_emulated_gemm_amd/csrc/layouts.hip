// layouts.hip -- laying out operands (K padded with zeros, transposes), the
// gate's elementwise passes and its backward.
//
// Everything here is one pass over its data, bound by memory; the transposes
// go through LDS tiles so that both sides are read and written in rows, four
// elements at a time: 14.5 us of 8192 x 2048 bfloat16 (4.6 TB/s; 27 us with single
// elements).
#include <type_traits>

#include "ops_device.hpp"
#include "split_device.hpp"
#include "ops.hpp"

namespace sgemm_emu_dev {

namespace {

unsigned blocks_for(int64_t items, int64_t per_block, int64_t most)
{
    const int64_t b = (items + per_block - 1) / per_block;
    return (unsigned)(b < 1 ? 1 : b < most ? b : most);
}

// One thread splits 8 consecutive elements of a padded row.
__global__ __launch_bounds__(256) void split_padded_kernel(int64_t rows, int64_t cols, int64_t kp, const float *X,
                                                           int64_t ldx, uint16_t *P, bool interleave)
{
    const int64_t groups = kp / 8, plane = rows * kp;
    for (int64_t q = (int64_t)blockIdx.x * 256 + threadIdx.x; q < rows * groups; q += (int64_t)gridDim.x * 256) {
        const int64_t row = q / groups, c = (q - row * groups) * 8;
        const float *src = X + (interleave ? (row & 1) * (rows >> 1) + (row >> 1) : row) * ldx + c;
        float x[8];
        if (c + 8 <= cols && ((uintptr_t)src % 16) == 0) {
            const f32x4_t a = reinterpret_cast<const f32x4_t *>(src)[0], b = reinterpret_cast<const f32x4_t *>(src)[1];
#pragma unroll
            for (int e = 0; e < 4; ++e) { x[e] = a[e]; x[4 + e] = b[e]; }
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) x[e] = c + e < cols ? src[e] : 0.0f;
        }
        uint32_t p0[4], p1[4], p2[4];
        split8_packed<false>(x, p0, p1, p2);
        uint16_t *dst = P + row * kp + c;
        *reinterpret_cast<u32x4_t *>(dst) = u32x4_t{p0[0], p0[1], p0[2], p0[3]};
        *reinterpret_cast<u32x4_t *>(dst + plane) = u32x4_t{p1[0], p1[1], p1[2], p1[3]};
        *reinterpret_cast<u32x4_t *>(dst + 2 * plane) = u32x4_t{p2[0], p2[1], p2[2], p2[3]};
    }
}

// 16 bytes of a row per thread.
template <class T>
__global__ __launch_bounds__(256) void copy_padded_kernel(int64_t rows, int64_t cols, int64_t kp, const T *X,
                                                          int64_t ldx, T *P)
{
    constexpr int V = 16 / sizeof(T);
    const int64_t groups = kp / V;
    for (int64_t q = (int64_t)blockIdx.x * 256 + threadIdx.x; q < rows * groups; q += (int64_t)gridDim.x * 256) {
        const int64_t row = q / groups, c = (q - row * groups) * V;
        const T *src = X + row * ldx + c;
        u32x4_t v = {0, 0, 0, 0};
        if (c + V <= cols) {
            v = *reinterpret_cast<const u32x4_any *>(src);
        } else {
#pragma unroll
            for (int e = 0; e < V; ++e)
                if (c + e < cols) {
                    if constexpr (sizeof(T) == 2) v[e >> 1] |= (uint32_t)src[e] << (16 * (e & 1));
                    else v[e] = src[e];
                }
        }
        *reinterpret_cast<u32x4_t *>(P + row * kp + c) = v;
    }
}

// Four elements and the access that takes them at any element's address.
template <class T>
struct Four {
    T v[4];
    typedef std::conditional_t<sizeof(T) == 4, u32x4_any, u32x2_any> access_t;
    static __device__ __forceinline__ Four load(const T *p)
    {
        return __builtin_bit_cast(Four, *reinterpret_cast<const access_t *>(p));
    }
    __device__ __forceinline__ void store(T *p) const
    {
        *reinterpret_cast<access_t *>(p) = __builtin_bit_cast(access_t, *this);
    }
};

// A 64 x 64 tile through LDS, by 256 threads: rows r0.., columns c0.. of src (rows x
// cols) -> dst (cols x out_rows with pitch ldo), zeros in rows rows..out_rows.
template <class T>
__device__ __forceinline__ void transpose_tile(int64_t rows, int64_t cols, int64_t out_rows, const T *src,
                                               int64_t lds_, T *dst, int64_t ldo, int64_t r0, int64_t c0)
{
    // four elements per access, rows in dwords an odd number apart
    __shared__ T tile[64][64 + 4 / sizeof(T)];
    const int q = (threadIdx.x & 15) * 4, hi = threadIdx.x >> 4;
    Four<T> v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int r = hi + 16 * i;
        const T *const p = src + (r0 + r) * lds_ + c0 + q;
        if (r0 + r < rows && c0 + q + 4 <= cols) {
            v[i] = Four<T>::load(p);
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e) v[i].v[e] = r0 + r < rows && c0 + q + e < cols ? p[e] : (T)0;
        }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) tile[hi + 16 * i][q + e] = v[i].v[e];
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int c = hi + 16 * i;
        if (c0 + c >= cols) continue;
        T *const p = dst + (c0 + c) * ldo + r0 + q;
        const Four<T> t = {{tile[q][c], tile[q + 1][c], tile[q + 2][c], tile[q + 3][c]}};
        if (r0 + q + 4 <= out_rows) {
            t.store(p);
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (r0 + q + e < out_rows) p[e] = t.v[e];
        }
    }
}

template <class T>
__global__ __launch_bounds__(256) void transpose_kernel(int64_t rows, int64_t cols, int64_t out_rows, const T *src,
                                                        int64_t lds_, T *dst, int64_t ldo)
{
    transpose_tile<T>(rows, cols, out_rows, src, lds_, dst, ldo, (int64_t)blockIdx.x * 64, (int64_t)blockIdx.y * 64);
}

// ---------------------------------------------------------------- before the adapters' backward

// Lists the rows of adapter `me`, ascending, by 256 threads: a thread takes a run of
// ids, counts those below its own (where its rows start) and its own, and, with
// the counts of the threads before it, writes its rows.  No atomics: the order,
// and with it the gradients' order of additions, is fixed.
__device__ __forceinline__ void group_rows_of(int32_t me, int64_t M, const int32_t *ids, int64_t n, int32_t *offs,
                                              int32_t *rows)
{
    __shared__ int32_t less_sum[4], own_sum[4];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t run = ((M + 255) / 256 + 3) / 4 * 4, begin = run * threadIdx.x, end = lmin(begin + run, M);
    auto each = [&](auto f) {
#pragma unroll 4
        for (int64_t t = begin; t < end; t += 4) {
            const u32x4_t v = t + 4 <= end ? (u32x4_t)*reinterpret_cast<const u32x4_any *>(ids + t)
                                           : u32x4_t{(uint32_t)ids[t], t + 1 < end ? (uint32_t)ids[t + 1] : ~0u,
                                                     t + 2 < end ? (uint32_t)ids[t + 2] : ~0u, ~0u};
#pragma unroll
            for (int e = 0; e < 4; ++e) f(t + e, (int32_t)v[e]);
        }
    };
    int32_t less = 0, own = 0;
    each([&](int64_t, int32_t v) {
        less += v >= 0 && v < me;
        own += v == me;
    });
    int32_t before = own;                        // of this wave's threads up to this one
#pragma unroll
    for (int s = 1; s < 64; s <<= 1) {
        less += __shfl_xor(less, s);
        const int32_t v = __shfl_up(before, s);
        before += lane >= s ? v : 0;
    }
    if (lane == 63) { less_sum[wave] = less; own_sum[wave] = before; }
    __syncthreads();
    const int32_t first = less_sum[0] + less_sum[1] + less_sum[2] + less_sum[3];
    if (threadIdx.x == 0) {
        offs[me] = first;
        if (me == n - 1) offs[n] = first + own_sum[0] + own_sum[1] + own_sum[2] + own_sum[3];
    }
    if (own == 0) return;
    int32_t at = first + before - own;
    for (int w = 0; w < wave; ++w) at += own_sum[w];
    each([&](int64_t t, int32_t v) {
        if (v == me) rows[at++] = (int32_t)t;
    });
}

// The adapters' factors transposed and their rows grouped, in one launch: each of
// the three alone is a few us of latency (8 adapters of rank 16, 8192 rows, 4096 x
// 4096 bfloat16: 8 us, in three launches 20).
template <class T>
__global__ __launch_bounds__(256) void prepare_kernel(AdapterPrepare q)
{
    int64_t b = blockIdx.x;
    if (b < q.groups) {
        group_rows_of((int32_t)b, q.M, q.ids, q.n, q.offs, q.rows);
        return;
    }
    b -= q.groups;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        const AdapterPrepare::Bank &m = q.bank[k];
        const int64_t tr = (m.rows + 63) / 64, tc = (m.cols + 63) / 64, tiles = m.dst != nullptr ? q.n * tr * tc : 0;
        if (b < tiles) {
            const int64_t i = b / (tr * tc), t = b - i * (tr * tc), step = i * m.rows * m.cols;
            transpose_tile<T>(m.rows, m.cols, m.rows, (const T *)m.src + step, m.cols, (T *)m.dst + step, m.rows,
                              t % tr * 64, t / tr * 64);
            return;
        }
        b -= tiles;
    }
}

// ---------------------------------------------------------------- gate

// The product with an empty K is its bias.
template <int GATE>
__global__ __launch_bounds__(256) void gate_bias_kernel(int64_t M, int64_t F, const float *bias, float *H, int64_t ldh,
                                                        float *Z, int64_t zup)
{
    const int64_t f = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (f >= F) return;
    const float g = bias != nullptr ? bias[f] : 0.0f, u = bias != nullptr ? bias[F + f] : 0.0f;
    const float h = gate_act<GATE>(g) * u;
    for (int64_t m = blockIdx.y; m < M; m += gridDim.y) {
        H[m * ldh + f] = h;
        if (Z != nullptr) {
            Z[m * 2 * zup + f] = g;
            Z[m * 2 * zup + zup + f] = u;
        }
    }
}

// 64 rows x 64 outputs per workgroup; a thread takes four consecutive outputs
// of four rows, loaded before any is used.  The tile of dZ waits in LDS for its
// transpose and the column sums, which take the unrounded values.  A bfloat16 dZ is
// rounded to its 8 bits here, once, as the operand of two bfloat16 products: two
// parts (16 bits) would make each of them two, 660 us more of 8192 x 2048 x 5461's
// 1300, where rounding moves the relative error of dX and dW, outputs of 8 bits
// themselves, from 0.0017 to 0.0023.  Bound by memory:
// float32 24576 x 1024 (704 MB) 141 us, 5.0 TB/s; bfloat16 8192 x 5461 (805 MB, Z in 32
// bits) 208 us, 3.9 TB/s.
template <class T, int GATE>
__global__ __launch_bounds__(256) void gate_backward_kernel(int64_t M, int64_t F, const float *Z, const T *dH,
                                                            int64_t lddh, T *dZ, T *dZt, float *sums)
{
    __shared__ float tile[2][64][65];
    typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
    const int64_t f0 = (int64_t)blockIdx.y * 64, m0 = (int64_t)blockIdx.x * 64;
    const int tc = (threadIdx.x & 15) * 4, tr = threadIdx.x >> 4;
    const int64_t f = f0 + tc, zup = (F + 7) / 8 * 8, dup = (F + 31) / 32 * 32, mp = (M + 63) / 64 * 64;
    f32x4_t zg[4], zu[4];
    float dh[4][4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int64_t m = m0 + tr + 16 * i;
        zg[i] = zu[i] = f32x4_t{0, 0, 0, 0};
#pragma unroll
        for (int e = 0; e < 4; ++e) dh[i][e] = 0.0f;
        if (m < M && f < F) {                    // Z's rows are padded: four always fit
            zg[i] = *reinterpret_cast<const f32x4_t *>(Z + m * 2 * zup + f);
            zu[i] = *reinterpret_cast<const f32x4_t *>(Z + m * 2 * zup + zup + f);
            const T *p = dH + m * lddh + f;
            if (f + 4 <= F) {
                if constexpr (sizeof(T) == 4) {
                    const u32x4_t x = *reinterpret_cast<const u32x4_any *>(p);
#pragma unroll
                    for (int e = 0; e < 4; ++e) dh[i][e] = __uint_as_float(x[e]);
                } else {
                    const u32x2 x = *reinterpret_cast<const u32x2_any *>(p);
#pragma unroll
                    for (int e = 0; e < 4; ++e) dh[i][e] = bf2f((uint16_t)(x[e >> 1] >> (16 * (e & 1))));
                }
            } else {
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (f + e < F) dh[i][e] = Elem<T>::load(p + e);
            }
        }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int row = tr + 16 * i;
        float dg[4], du[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            float a, d;
            gate_act_grad<GATE>(zg[i][e], a, d);
            const bool in = m0 + row < M && f + e < F;      // the padding of Z may hold anything
            dg[e] = in ? dh[i][e] * zu[i][e] * d : 0.0f;
            du[e] = in ? dh[i][e] * a : 0.0f;
            tile[0][row][tc + e] = dg[e];
            tile[1][row][tc + e] = du[e];
        }
        // a tile reaches past dup only where dup is not a multiple of 64
        if (dZ != nullptr && m0 + row < M && f < dup) {
            T *const p = dZ + (m0 + row) * 2 * dup + f;
            if constexpr (sizeof(T) == 4) {
                *reinterpret_cast<f32x4_t *>(p) = f32x4_t{dg[0], dg[1], dg[2], dg[3]};
                *reinterpret_cast<f32x4_t *>(p + dup) = f32x4_t{du[0], du[1], du[2], du[3]};
            } else {
                *reinterpret_cast<u32x2 *>(p) = u32x2{pack2(dg[0], dg[1]), pack2(dg[2], dg[3])};
                *reinterpret_cast<u32x2 *>(p + dup) = u32x2{pack2(du[0], du[1]), pack2(du[2], du[3])};
            }
        }
    }
    __syncthreads();
    if (dZt != nullptr) {
        // four rows of the tile are 16 (8) bytes of a transposed row
        const int q = (threadIdx.x & 15) * 4, hi = threadIdx.x >> 4;
#pragma unroll
        for (int s = 0; s < 2; ++s)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int c = hi + 16 * i;
                if (f0 + c < F) {
                    T *const p = dZt + (s * F + f0 + c) * mp + m0 + q;
                    const float v0 = tile[s][q][c], v1 = tile[s][q + 1][c], v2 = tile[s][q + 2][c],
                                v3 = tile[s][q + 3][c];
                    if constexpr (sizeof(T) == 4) *reinterpret_cast<f32x4_t *>(p) = f32x4_t{v0, v1, v2, v3};
                    else *reinterpret_cast<u32x2 *>(p) = u32x2{pack2(v0, v1), pack2(v2, v3)};
                }
            }
    }
    if (sums != nullptr && threadIdx.x < 128) {
        const int s = threadIdx.x >> 6, c = threadIdx.x & 63;
        float v = 0.0f;
#pragma unroll 8
        for (int row = 0; row < 64; ++row) v += tile[s][row][c];
        if (f0 + c < F) sums[(int64_t)blockIdx.x * 2 * F + s * F + f0 + c] = v;
    }
}

// out[c] = the tiles' sums: 16 threads per column, each over a run of tiles,
// added in order.
template <class T>
__global__ __launch_bounds__(1024) void sum_tiles_kernel(int64_t tiles, int64_t cols, const float *sums, T *out)
{
    __shared__ float part[16][64];
    const int l = threadIdx.x & 63, q = threadIdx.x >> 6;
    const int64_t c = (int64_t)blockIdx.x * 64 + l;
    float v = 0.0f;
    if (c < cols) {
        const int64_t end = tiles * (q + 1) / 16;
#pragma unroll 8
        for (int64_t t = tiles * q / 16; t < end; ++t) v += sums[t * cols + c];
    }
    part[q][l] = v;
    __syncthreads();
    if (q == 0 && c < cols) {
#pragma unroll
        for (int k = 1; k < 16; ++k) v += part[k][l];
        out[c] = Elem<T>::store(v);
    }
}

template <class T>
hipError_t gate_backward_t(int64_t M, int64_t F, const float *Z, const T *dH, int64_t lddh, int gate, T *dZ, T *dZt,
                           float *sums, hipStream_t stream)
{
    const dim3 grid((unsigned)gate_tiles(M), (unsigned)((F + 63) / 64));
#define LAUNCH(G)                                                                                                 \
    hipLaunchKernelGGL((gate_backward_kernel<T, G>), grid, dim3(256), 0, stream, M, F, Z, dH, lddh, dZ, dZt, sums)
    switch (gate) {
    case kSilu: LAUNCH(kSilu); break;
    case kGelu: LAUNCH(kGelu); break;
    case kGeluTanh: LAUNCH(kGeluTanh); break;
    case kSigmoid: LAUNCH(kSigmoid); break;
    case kRelu: LAUNCH(kRelu); break;
    default: return hipErrorInvalidValue;
    }
#undef LAUNCH
    return hipGetLastError();
}

}  // namespace

hipError_t launch_split_padded(int64_t rows, int64_t cols, const float *X, int64_t ldx, uint16_t *P, bool interleave,
                               hipStream_t stream)
{
    const int64_t kp = pad_k(cols);
    hipLaunchKernelGGL(split_padded_kernel, dim3(blocks_for(rows * (kp / 8), 256, 16384)), dim3(256), 0, stream, rows,
                       cols, kp, X, ldx, P, interleave);
    return hipGetLastError();
}

hipError_t launch_copy_padded(int dtype, int64_t rows, int64_t cols, const void *X, int64_t ldx, void *P, int64_t kp,
                              hipStream_t stream)
{
    if (dtype == kF32)
        hipLaunchKernelGGL((copy_padded_kernel<uint32_t>), dim3(blocks_for(rows * (kp / 4), 256, 16384)), dim3(256), 0,
                           stream, rows, cols, kp, (const uint32_t *)X, ldx, (uint32_t *)P);
    else
        hipLaunchKernelGGL((copy_padded_kernel<uint16_t>), dim3(blocks_for(rows * (kp / 8), 256, 16384)), dim3(256), 0,
                           stream, rows, cols, kp, (const uint16_t *)X, ldx, (uint16_t *)P);
    return hipGetLastError();
}

hipError_t launch_transpose_padded(int64_t rows, int64_t cols, const uint16_t *X, int64_t ldx, uint16_t *P,
                                   int64_t out_rows, int64_t ldp, hipStream_t stream)
{
    hipLaunchKernelGGL((transpose_kernel<uint16_t>), dim3((unsigned)((out_rows + 63) / 64), (unsigned)((cols + 63) / 64)),
                       dim3(256), 0, stream, rows, cols, out_rows, X, ldx, P, ldp);
    return hipGetLastError();
}

hipError_t launch_adapter_prepare(int dtype, AdapterPrepare q, hipStream_t stream)
{
    q.groups = q.offs != nullptr ? q.n : 0;
    int64_t blocks = q.groups;
    for (const AdapterPrepare::Bank &m : q.bank)
        if (m.dst != nullptr) blocks += q.n * ((m.rows + 63) / 64) * ((m.cols + 63) / 64);
    if (blocks == 0) return hipSuccess;
    if (blocks > INT32_MAX) return hipErrorInvalidValue;
    if (dtype == kF32)
        hipLaunchKernelGGL((prepare_kernel<float>), dim3((unsigned)blocks), dim3(256), 0, stream, q);
    else
        hipLaunchKernelGGL((prepare_kernel<uint16_t>), dim3((unsigned)blocks), dim3(256), 0, stream, q);
    return hipGetLastError();
}

hipError_t launch_gate_bias(int64_t M, int64_t F, const float *bias, int gate, float *H, int64_t ldh, float *Z,
                            hipStream_t stream)
{
    const dim3 grid((unsigned)((F + 255) / 256), (unsigned)(M < 16384 ? M : 16384));
#define LAUNCH(G) hipLaunchKernelGGL((gate_bias_kernel<G>), grid, dim3(256), 0, stream, M, F, bias, H, ldh, Z, z_pitch(F) / 2)
    switch (gate) {
    case kSilu: LAUNCH(kSilu); break;
    case kGelu: LAUNCH(kGelu); break;
    case kGeluTanh: LAUNCH(kGeluTanh); break;
    case kSigmoid: LAUNCH(kSigmoid); break;
    case kRelu: LAUNCH(kRelu); break;
    default: return hipErrorInvalidValue;
    }
#undef LAUNCH
    return hipGetLastError();
}

hipError_t launch_gate_backward(int dtype, int64_t M, int64_t F, const float *Z, const void *dH, int64_t lddh,
                                int gate, void *dZ, void *dZt, float *sums, hipStream_t stream)
{
    if (dtype == kF32)
        return gate_backward_t<float>(M, F, Z, (const float *)dH, lddh, gate, (float *)dZ, (float *)dZt, sums, stream);
    return gate_backward_t<uint16_t>(M, F, Z, (const uint16_t *)dH, lddh, gate, (uint16_t *)dZ, (uint16_t *)dZt, sums,
                                     stream);
}

hipError_t launch_sum_tiles(int dtype, int64_t tiles, int64_t cols, const float *sums, void *out, hipStream_t stream)
{
    const dim3 grid((unsigned)((cols + 63) / 64));
    if (dtype == kF32)
        hipLaunchKernelGGL((sum_tiles_kernel<float>), grid, dim3(1024), 0, stream, tiles, cols, sums, (float *)out);
    else
        hipLaunchKernelGGL((sum_tiles_kernel<uint16_t>), grid, dim3(1024), 0, stream, tiles, cols, sums,
                           (uint16_t *)out);
    return hipGetLastError();
}

}  // namespace sgemm_emu_dev
