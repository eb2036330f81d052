// expert_device.hpp -- device helpers of the experts' kernels: an expert's rows,
// and which of them a tile covers.
#pragma once
#include "experts.hpp"
#include "ops_device.hpp"
#include "split_device.hpp"

namespace sgemm_emu_dev {

// Where segment e starts and ends: expert e's rows, or for e = n the rows of no
// expert.  Held inside [0, P] whatever the array holds.
__device__ __forceinline__ int64_t expert_start(const int32_t *offsets, int64_t e, int64_t P)
{
    if (offsets == nullptr) return e == 0 ? 0 : P;
    const int64_t v = offsets[e];
    return v < 0 ? 0 : v < P ? v : P;
}
__device__ __forceinline__ int64_t expert_end(const int32_t *offsets, int64_t e, int64_t n, int64_t P)
{
    if (e >= n) return P;
    const int64_t s = expert_start(offsets, e, P), v = expert_start(offsets, e + 1, P);
    return v < s ? s : v;
}

// Row tiles of BM rows, counted through the segments 0 .. segments - 1.
struct RowTile {
    int segment;             // -1: there is no such tile
    int64_t row, end;        // first row; end of the segment
    int first;               // the segment's first tile
};

__device__ __forceinline__ int wave_sum(int v)
{
#pragma unroll
    for (int d = 32; d > 0; d >>= 1) v += __shfl_xor(v, d);
    return v;
}

template <int BM>
__device__ __forceinline__ int count_tiles(const int32_t *offsets, int64_t n, int64_t P, int e, int segments)
{
    return e < segments ? (int)((expert_end(offsets, e, n, P) - expert_start(offsets, e, P) + BM - 1) / BM) : 0;
}

// Tiles of all segments; uniform over the wave.
template <int BM>
__device__ __forceinline__ int all_tiles(const int32_t *offsets, int64_t n, int64_t P, int segments, int lane)
{
    int c = 0;
    for (int e = lane; e < segments; e += 64) c += count_tiles<BM>(offsets, n, P, e, segments);
    return __builtin_amdgcn_readfirstlane(wave_sum(c));
}

// Tile `index`; all lanes of the wave take part and get the same.
template <int BM>
__device__ __forceinline__ RowTile find_tile(const int32_t *offsets, int64_t n, int64_t P, int segments, int index,
                                             int lane)
{
    int base = 0;
    for (int e0 = 0; e0 < segments; e0 += 64) {
        const int c = count_tiles<BM>(offsets, n, P, e0 + lane, segments);
        int sum = c;                                       // inclusive over the lanes
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) {
            const int v = __shfl_up(sum, d);
            if (lane >= d) sum += v;
        }
        const uint64_t past = __ballot(base + sum > index);
        if (past != 0) {
            const int l = __builtin_ctzll(past);
            RowTile t;
            t.segment = e0 + l;
            t.first = base + __builtin_amdgcn_readlane(sum - c, l);
            t.row = expert_start(offsets, t.segment, P) + (int64_t)(index - t.first) * BM;
            t.end = expert_end(offsets, t.segment, n, P);
            return t;
        }
        base += __builtin_amdgcn_readlane(sum, 63);
    }
    return RowTile{-1, 0, 0, 0};
}

// Eight consecutive elements in registers, `left` of them there (others zero).
template <class T>
struct Eight {
    u32x4_t v[sizeof(T) / 2];

    __device__ __forceinline__ void load(const T *p, int64_t left)
    {
        constexpr int V = Elem<T>::VEC;
#pragma unroll
        for (int i = 0; i < (int)sizeof(T) / 2; ++i) v[i] = u32x4_t{0, 0, 0, 0};
        if (left >= 8) {
#pragma unroll
            for (int i = 0; i < (int)sizeof(T) / 2; ++i) v[i] = *reinterpret_cast<const u32x4_any *>(p + i * V);
        } else if (left > 0) {
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (e < left) {
                    if constexpr (sizeof(T) == 4) v[e >> 2][e & 3] = __float_as_uint(p[e]);
                    else v[0][e >> 1] |= (uint32_t)p[e] << (16 * (e & 1));
                }
        }
    }
};

// Rounded to BF16, two at a time; beyond the largest BF16 that, not Inf.
__device__ __forceinline__ uint32_t pack2_finite(float a, float b)
{
    constexpr float MOST = 3.38953139e38f;
    return pack2(__builtin_amdgcn_fmed3f(a, -MOST, MOST), __builtin_amdgcn_fmed3f(b, -MOST, MOST));
}

// The parts of eight FP32 values, x = x0 + 2^-8 x1 + 2^-16 x2, each stage rounded
// to nearest even by the hardware's conversion.  x0 and x1 stay finite: an Inf or
// NaN comes through in x2 (Inf - finite), so its products are those of IEEE.
__device__ __forceinline__ void split8_nearest(const Eight<float> &in, u32x4_t (&p)[3])
{
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float x = __uint_as_float(in.v[i >> 1][2 * (i & 1)]), y = __uint_as_float(in.v[i >> 1][2 * (i & 1) + 1]);
        const uint32_t w0 = pack2_finite(x, y);
        const float t = (x - u2f(w0 << 16)) * 256.0f, u = (y - u2f(w0 & 0xFFFF0000u)) * 256.0f;
        const uint32_t w1 = pack2_finite(t, u);
        const float a = (t - u2f(w1 << 16)) * 256.0f, b = (u - u2f(w1 & 0xFFFF0000u)) * 256.0f;
        p[0][i] = w0;
        p[1][i] = w1;
        p[2][i] = pack2(a, b);               // exact where finite: 8 significant bits
    }
}

}  // namespace sgemm_emu_dev
