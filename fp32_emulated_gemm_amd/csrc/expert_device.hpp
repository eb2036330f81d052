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

// This workgroup's number in a grid of grid_of(), whose last ones may lie past `blocks`.
__device__ __forceinline__ int workgroup() { return (int)(blockIdx.y * kGridX + blockIdx.x); }

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

// The row tiles of all segments and where each lies, found by whole waves.
template <int BM_>
struct RowTiles {
    const int32_t *offsets;
    int64_t n, P;
    int lane, segments, BM;
    int64_t start, end;      // of segment `lane`
    int count, sum;          // its tiles, and those up to it
    int total;               // of all segments; uniform

    // rows: of a tile, where BM_ is 0.
    __device__ __forceinline__ RowTiles(const int32_t *o, int64_t n_, int64_t P_, int segments_, int lane_, int rows = 0)
        : offsets(o), n(n_), P(P_), lane(lane_), segments(segments_), BM(BM_ != 0 ? BM_ : rows)
    {
        start = end = 0;                                                            // without a segment there is no tile
        count = sum = total = 0;
        for (int e0 = (segments - 1) & ~63; e0 >= 0; e0 -= 64) total += scan(e0);   // ends with the first 64
    }

    // Segments e0 + lane; returns their tiles.
    __device__ __forceinline__ int scan(int e0)
    {
        const int e = e0 + lane;
        start = end = 0;
        if (e < segments) {
            // both loads at once: a workgroup starts with them
            const int64_t s = offsets != nullptr ? offsets[lmin(e, n)] : e == 0 ? 0 : P;
            const int64_t t = offsets != nullptr && e < n ? offsets[lmin(e + 1, n)] : P;
            start = s < 0 ? 0 : lmin(s, P);
            end = t < start ? start : lmin(t, P);
        }
        count = sum = (int)(((uint32_t)(end - start) + (uint32_t)BM - 1u) / (uint32_t)BM);   // rows are below 2^22
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) {
            const int v = __shfl_up(sum, d);
            if (lane >= d) sum += v;
        }
        return __builtin_amdgcn_readlane(sum, 63);
    }

    // Tile `index`; every lane gets the same.
    __device__ __forceinline__ RowTile find(int index)
    {
        int base = 0;
        for (int e0 = 0;;) {
            const uint64_t past = __ballot(base + sum > index);
            if (past != 0) {
                const int l = __builtin_ctzll(past);
                RowTile t;
                t.segment = e0 + l;
                t.first = base + __builtin_amdgcn_readlane(sum - count, l);
                t.row = uniform(start, l) + (int64_t)(index - t.first) * BM;
                t.end = uniform(end, l);
                return t;
            }
            base += __builtin_amdgcn_readlane(sum, 63);
            e0 += 64;
            if (e0 >= segments) return RowTile{-1, 0, 0, 0};
            scan(e0);
        }
    }

    static __device__ __forceinline__ int64_t uniform(int64_t v, int l)
    {
        // rows are below 2^31
        return __builtin_amdgcn_readlane((int)v, l);
    }
};

// Rounded to BF16, two at a time; beyond the largest BF16 that, not Inf.
__device__ __forceinline__ uint32_t pack2_finite(float a, float b)
{
    constexpr float MOST = 3.38953139e38f;
    return pack2(__builtin_amdgcn_fmed3f(a, -MOST, MOST), __builtin_amdgcn_fmed3f(b, -MOST, MOST));
}

// The parts of two FP32 values, x = x0 + 2^-8 x1 + 2^-16 x2, each stage rounded to
// nearest even by the hardware's conversion.  x0 and x1 stay finite, so that a value
// beyond the largest BF16 keeps its own; an Inf or NaN comes through in x2, and what it
// reaches is Inf or NaN (NaN where the largest BF16 times the other operand's smaller
// part overflows to the other side).
__device__ __forceinline__ void split2_nearest(float x, float y, uint32_t &p0, uint32_t &p1, uint32_t &p2)
{
    p0 = pack2_finite(x, y);
    const float t = (x - u2f(p0 << 16)) * 256.0f, u = (y - u2f(p0 & 0xFFFF0000u)) * 256.0f;
    p1 = pack2_finite(t, u);
    const float a = (t - u2f(p1 << 16)) * 256.0f, b = (u - u2f(p1 & 0xFFFF0000u)) * 256.0f;
    p2 = pack2(a, b);                        // exact where finite: 8 significant bits
}

// 16 bytes of a row in registers, `left` of its elements there (others zero).
template <class T>
__device__ __forceinline__ u32x4_t load_piece(const T *p, int64_t left)
{
    constexpr int V = Elem<T>::VEC;
    u32x4_t v = {0, 0, 0, 0};
    if (left >= V) {
        v = *reinterpret_cast<const u32x4_any *>(p);
    } else if (left > 0) {
#pragma unroll
        for (int e = 0; e < V; ++e)
            if (e < left) {
                if constexpr (sizeof(T) == 4) v[e] = __float_as_uint(p[e]);
                else v[e >> 1] |= (uint32_t)p[e] << (16 * (e & 1));
            }
    }
    return v;
}

// Rows that a workgroup of a weight gradient takes: an expert's, or with partial sums
// one of the pieces of g.chunk rows that all experts' rows are cut into.
__device__ __forceinline__ RowTile weight_rows(const ExpertProduct &g, int chunk, int lane)
{
    RowTile t{chunk, 0, 0, 0};
    if (g.partials == nullptr) {
        t.row = expert_start(g.offsets, chunk, g.P);
        t.end = expert_end(g.offsets, chunk, g.n, g.P);
    } else {
        t = RowTiles<0>(g.offsets, g.n, g.P, (int)g.n, lane, (int)g.chunk).find(chunk);
        t.end = lmin(t.end, t.row + g.chunk);
    }
    return t;
}

// tile_of_index (device_common.hpp) in its two halves: the tile that workgroup v of
// T takes, so that each XCD has a run of them, and where tile t lies.
__device__ __forceinline__ int xcd_order(int v, int T)
{
    const int per = T >> 3, extra = T & 7, xcd = v & 7;
    return xcd * per + imin(xcd, extra) + (v >> 3);
}
__device__ __forceinline__ void tile_at(int t, int tiles_m, int tiles_n, int group_m, int &tm, int &tn)
{
    const int group = t / (group_m * tiles_n), first = group * group_m, gm = imin(tiles_m - first, group_m);
    const int in = t - group * group_m * tiles_n;
    tm = first + in % gm;
    tn = in / gm;
}

}  // namespace sgemm_emu_dev
