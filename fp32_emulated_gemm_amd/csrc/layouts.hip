// layouts.hip -- laying out operands (K padded with zeros, transposes), the
// gate's elementwise passes and its backward.
//
// Everything here is one pass over its data, bound by memory; the transposes
// go through LDS tiles so that both sides are read and written in rows.
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
                                                           int64_t ldx, uint16_t *P)
{
    const int64_t groups = kp / 8, plane = rows * kp;
    for (int64_t q = (int64_t)blockIdx.x * 256 + threadIdx.x; q < rows * groups; q += (int64_t)gridDim.x * 256) {
        const int64_t row = q / groups, c = (q - row * groups) * 8;
        const float *src = X + row * ldx + c;
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

__global__ __launch_bounds__(256) void copy_padded_kernel(int64_t rows, int64_t cols, int64_t kp, const uint16_t *X,
                                                          int64_t ldx, uint16_t *P)
{
    const int64_t groups = kp / 8;
    for (int64_t q = (int64_t)blockIdx.x * 256 + threadIdx.x; q < rows * groups; q += (int64_t)gridDim.x * 256) {
        const int64_t row = q / groups, c = (q - row * groups) * 8;
        const uint16_t *src = X + row * ldx + c;
        u32x4_t v = {0, 0, 0, 0};
        if (c + 8 <= cols && ((uintptr_t)src % 16) == 0) {
            v = *reinterpret_cast<const u32x4_t *>(src);
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (c + e < cols) v[e >> 1] |= (uint32_t)src[e] << (16 * (e & 1));
        }
        *reinterpret_cast<u32x4_t *>(P + row * kp + c) = v;
    }
}

// 64 x 64 tiles through LDS: src rows x cols (batch b at b * src_step) -> dst
// cols x out_rows with pitch ldo, zeros in rows rows..out_rows.
template <class T>
__global__ __launch_bounds__(256) void transpose_kernel(int64_t rows, int64_t cols, int64_t out_rows, const T *src,
                                                        int64_t lds_, int64_t src_step, T *dst, int64_t ldo,
                                                        int64_t dst_step)
{
    __shared__ T tile[64][64 + 4 / sizeof(T)];
    const int64_t r0 = (int64_t)blockIdx.x * 64, c0 = (int64_t)blockIdx.y * 64;
    src += (int64_t)blockIdx.z * src_step;
    dst += (int64_t)blockIdx.z * dst_step;
    const int lo = threadIdx.x & 63, hi = threadIdx.x >> 6;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        const int r = hi + 4 * i;
        tile[r][lo] = r0 + r < rows && c0 + lo < cols ? src[(r0 + r) * lds_ + c0 + lo] : (T)0;
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        const int c = hi + 4 * i;
        if (c0 + c < cols && r0 + lo < out_rows) dst[(c0 + c) * ldo + r0 + lo] = tile[lo][c];
    }
}

// ---------------------------------------------------------------- gate

template <int GATE>
__global__ __launch_bounds__(256) void gate_kernel(int64_t M, int64_t F, const float *Z, int64_t ldz, float *H,
                                                   int64_t ldh)
{
    const int64_t f = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (f >= F) return;
    for (int64_t m = blockIdx.y; m < M; m += gridDim.y)
        H[m * ldh + f] = gate_act<GATE>(Z[m * ldz + f]) * Z[m * ldz + F + f];
}

// 64 rows x 64 outputs per workgroup; a thread takes four consecutive outputs
// of four rows.  The tile of dZ waits in LDS for its transpose and the column
// sums, which take the unrounded values.
template <class T, int GATE>
__global__ __launch_bounds__(256) void gate_backward_kernel(int64_t M, int64_t F, const T *Z, int64_t ldz, const T *dH,
                                                            int64_t lddh, bool vec, T *dZ, int64_t ldd, T *dZt,
                                                            int64_t mp, float *sums)
{
    __shared__ float tile[2][64][65];
    const int64_t f0 = (int64_t)blockIdx.y * 64, m0 = (int64_t)blockIdx.x * 64;
    const int tc = (threadIdx.x & 15) * 4, tr = threadIdx.x >> 4;
    typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
    auto load4 = [&](const T *p, int64_t f, float (&v)[4]) {
        if (vec && f + 4 <= F) {
            if constexpr (sizeof(T) == 4) {
                const f32x4_t x = *reinterpret_cast<const f32x4_t *>(p);
#pragma unroll
                for (int e = 0; e < 4; ++e) v[e] = x[e];
            } else {
                const u32x2 x = *reinterpret_cast<const u32x2 *>(p);
#pragma unroll
                for (int e = 0; e < 4; ++e) v[e] = bf2f((uint16_t)(x[e >> 1] >> (16 * (e & 1))));
            }
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e) v[e] = f + e < F ? Elem<T>::load(p + e) : 0.0f;
        }
    };
    auto store4 = [&](T *p, int64_t f, const float (&v)[4]) {
        if (vec && f + 4 <= F) {
            if constexpr (sizeof(T) == 4) *reinterpret_cast<f32x4_t *>(p) = f32x4_t{v[0], v[1], v[2], v[3]};
            else *reinterpret_cast<u32x2 *>(p) = u32x2{pack2(v[0], v[1]), pack2(v[2], v[3])};
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (f + e < F) p[e] = Elem<T>::store(v[e]);
        }
    };
    const int64_t f = f0 + tc;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int row = tr + 16 * i;
        const int64_t m = m0 + row;
        float zg[4] = {0, 0, 0, 0}, zu[4] = {0, 0, 0, 0}, dh[4] = {0, 0, 0, 0}, dg[4], du[4];
        if (m < M && f < F) {
            load4(Z + m * ldz + f, f, zg);
            load4(Z + m * ldz + F + f, f, zu);
            load4(dH + m * lddh + f, f, dh);
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            float a, d;
            gate_act_grad<GATE>(zg[e], a, d);
            dg[e] = dh[e] * zu[e] * d;
            du[e] = dh[e] * a;
            tile[0][row][tc + e] = dg[e];
            tile[1][row][tc + e] = du[e];
        }
        if (dZ != nullptr && m < M && f < F) {
            store4(dZ + m * ldd + f, f, dg);
            store4(dZ + m * ldd + F + f, f, du);
        }
    }
    if (dZ != nullptr && blockIdx.y == gridDim.y - 1) {
        // the pitch's padding
        const int64_t pad = ldd - 2 * F;
        for (int64_t o = threadIdx.x; o < 64 * pad; o += 256)
            if (m0 + o / pad < M) dZ[(m0 + o / pad) * ldd + 2 * F + o % pad] = Elem<T>::store(0.0f);
    }
    __syncthreads();
    if (dZt != nullptr) {
        const int lo = threadIdx.x & 63, hi = threadIdx.x >> 6;
#pragma unroll
        for (int s = 0; s < 2; ++s)
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const int c = hi + 4 * i;
                if (f0 + c < F) dZt[(s * F + f0 + c) * mp + m0 + lo] = Elem<T>::store(tile[s][lo][c]);
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

template <class T>
__global__ __launch_bounds__(256) void sum_tiles_kernel(int64_t tiles, int64_t cols, const float *sums, T *out)
{
    // 64 columns, four threads each over a quarter of the tiles, added in order
    __shared__ float part[4][64];
    const int64_t c = (int64_t)blockIdx.x * 64 + (threadIdx.x & 63);
    const int q = threadIdx.x >> 6;
    float v = 0.0f;
    if (c < cols)
        for (int64_t t = tiles * q / 4; t < tiles * (q + 1) / 4; ++t) v += sums[t * cols + c];
    part[q][threadIdx.x & 63] = v;
    __syncthreads();
    if (q == 0 && c < cols) {
        const int l = threadIdx.x & 63;
        out[c] = Elem<T>::store(((part[0][l] + part[1][l]) + part[2][l]) + part[3][l]);
    }
}

template <class T>
hipError_t gate_backward_t(int64_t M, int64_t F, const T *Z, int64_t ldz, const T *dH, int64_t lddh, int gate, T *dZ,
                           int64_t ldd, T *dZt, float *sums, hipStream_t stream)
{
    const dim3 grid((unsigned)gate_tiles(M), (unsigned)((F + 63) / 64));
    // four elements at once: every row of every operand, gate and up half, aligned to them
    const uintptr_t a = 4 * sizeof(T);
    const bool vec = F % 4 == 0 && ldz % 4 == 0 && lddh % 4 == 0 && ldd % 4 == 0 && aligned(Z, a) && aligned(dH, a) &&
                     aligned(dZ, a);
    const int64_t mp = pad_k(M);
#define LAUNCH(G)                                                                                                     \
    hipLaunchKernelGGL((gate_backward_kernel<T, G>), grid, dim3(256), 0, stream, M, F, Z, ldz, dH, lddh, vec, dZ, ldd, \
                       dZt, mp, sums)
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

hipError_t launch_split_padded(int64_t rows, int64_t cols, const float *X, int64_t ldx, uint16_t *P,
                               hipStream_t stream)
{
    const int64_t kp = pad_k(cols);
    hipLaunchKernelGGL(split_padded_kernel, dim3(blocks_for(rows * (kp / 8), 256, 16384)), dim3(256), 0, stream, rows,
                       cols, kp, X, ldx, P);
    return hipGetLastError();
}

hipError_t launch_copy_padded(int64_t rows, int64_t cols, const uint16_t *X, int64_t ldx, uint16_t *P,
                              hipStream_t stream)
{
    const int64_t kp = pad_k(cols);
    hipLaunchKernelGGL(copy_padded_kernel, dim3(blocks_for(rows * (kp / 8), 256, 16384)), dim3(256), 0, stream, rows,
                       cols, kp, X, ldx, P);
    return hipGetLastError();
}

hipError_t launch_transpose_padded(int64_t rows, int64_t cols, const uint16_t *X, int64_t ldx, uint16_t *P,
                                   hipStream_t stream)
{
    const int64_t rp = pad_k(rows);
    hipLaunchKernelGGL((transpose_kernel<uint16_t>), dim3((unsigned)(rp / 64), (unsigned)((cols + 63) / 64)), dim3(256),
                       0, stream, rows, cols, rp, X, ldx, (int64_t)0, P, rp, (int64_t)0);
    return hipGetLastError();
}

hipError_t launch_transpose_bank(int dtype, int64_t n, int64_t rows, int64_t cols, const void *src, void *dst,
                                 hipStream_t stream)
{
    const dim3 grid((unsigned)((rows + 63) / 64), (unsigned)((cols + 63) / 64), (unsigned)n);
    if (dtype == kF32)
        hipLaunchKernelGGL((transpose_kernel<float>), grid, dim3(256), 0, stream, rows, cols, rows, (const float *)src,
                           cols, rows * cols, (float *)dst, rows, rows * cols);
    else
        hipLaunchKernelGGL((transpose_kernel<uint16_t>), grid, dim3(256), 0, stream, rows, cols, rows,
                           (const uint16_t *)src, cols, rows * cols, (uint16_t *)dst, rows, rows * cols);
    return hipGetLastError();
}

hipError_t launch_gate(int64_t M, int64_t F, const float *Z, int64_t ldz, int gate, float *H, int64_t ldh,
                       hipStream_t stream)
{
    const dim3 grid((unsigned)((F + 255) / 256), (unsigned)(M < 16384 ? M : 16384));
    switch (gate) {
    case kSilu: hipLaunchKernelGGL((gate_kernel<kSilu>), grid, dim3(256), 0, stream, M, F, Z, ldz, H, ldh); break;
    case kGelu: hipLaunchKernelGGL((gate_kernel<kGelu>), grid, dim3(256), 0, stream, M, F, Z, ldz, H, ldh); break;
    case kGeluTanh:
        hipLaunchKernelGGL((gate_kernel<kGeluTanh>), grid, dim3(256), 0, stream, M, F, Z, ldz, H, ldh);
        break;
    case kSigmoid: hipLaunchKernelGGL((gate_kernel<kSigmoid>), grid, dim3(256), 0, stream, M, F, Z, ldz, H, ldh); break;
    case kRelu: hipLaunchKernelGGL((gate_kernel<kRelu>), grid, dim3(256), 0, stream, M, F, Z, ldz, H, ldh); break;
    default: return hipErrorInvalidValue;
    }
    return hipGetLastError();
}

hipError_t launch_gate_backward(int dtype, int64_t M, int64_t F, const void *Z, int64_t ldz, const void *dH,
                                int64_t lddh, int gate, void *dZ, int64_t ldd, void *dZt, float *sums,
                                hipStream_t stream)
{
    if (dtype == kF32)
        return gate_backward_t<float>(M, F, (const float *)Z, ldz, (const float *)dH, lddh, gate, (float *)dZ, ldd,
                                      (float *)dZt, sums, stream);
    return gate_backward_t<uint16_t>(M, F, (const uint16_t *)Z, ldz, (const uint16_t *)dH, lddh, gate, (uint16_t *)dZ,
                                     ldd, (uint16_t *)dZt, sums, stream);
}

hipError_t launch_sum_tiles(int dtype, int64_t tiles, int64_t cols, const float *sums, void *out, hipStream_t stream)
{
    const dim3 grid((unsigned)((cols + 63) / 64));
    if (dtype == kF32)
        hipLaunchKernelGGL((sum_tiles_kernel<float>), grid, dim3(256), 0, stream, tiles, cols, sums, (float *)out);
    else
        hipLaunchKernelGGL((sum_tiles_kernel<uint16_t>), grid, dim3(256), 0, stream, tiles, cols, sums,
                           (uint16_t *)out);
    return hipGetLastError();
}

}  // namespace sgemm_emu_dev
