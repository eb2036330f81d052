// expert_rows.hpp -- blocks of 16 rows by 128 columns in a wave's registers, as the
// kernels of few rows take them (expert_few.hip, quant4.hip).
#pragma once
#include "expert_device.hpp"

namespace sgemm_emu_dev {

namespace {

// The columns 8 (lane >> 4) .. + 7 of four steps of 32 of a row, as they come:
// one row of a tile of 16 in each lane.
template <class T>
struct RowBlock {
    u32x4_t v[4][sizeof(T) / 2];

    // LIES: rows at whole dwords, loaded through a descriptor that ends with the dword of
    // the last element.  Rows past the last read zeros.
    template <bool LIES>
    __device__ __forceinline__ void load(const T *X, int64_t ld, int64_t row, int64_t rows, int64_t k0, int64_t K, int lane)
    {
        constexpr int PIECES = sizeof(T) / 2;
        if constexpr (LIES) {
            // a descriptor for the tile's 16 rows; the row of this lane lies `lane & 15` further
            const int64_t first = row - (lane & 15), left = rows - first;
            const int64_t bytes = ((lmin(left, 16) - 1) * ld + K) * (int64_t)sizeof(T);
            const rsrc_t r = make_rsrc(X + first * ld, left > 0 ? (bytes + 3) & ~3ll : 0);
            const uint32_t off = row < rows ? (uint32_t)(((lane & 15) * ld + (lane >> 4) * 8) * sizeof(T)) : 0xFFFFFFF0u;
#pragma unroll
            for (int d = 0; d < 4; ++d)
#pragma unroll
                for (int i = 0; i < PIECES; ++i)
                    v[d][i] = bload_u32x4(r, off == 0xFFFFFFF0u ? off : off + (uint32_t)((k0 + d * 32) * sizeof(T) + i * 16), 0);
            if (k0 + 128 <= K) return;
            // the last block: what the pieces hold behind K
#pragma unroll
            for (int d = 0; d < 4; ++d) {
                const int64_t end = K - (k0 + d * 32 + (lane >> 4) * 8);
#pragma unroll
                for (int i = 0; i < PIECES; ++i)
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        if constexpr (sizeof(T) == 4) v[d][i][q] = i * 4 + q < end ? v[d][i][q] : 0u;
                        else v[d][i][q] = 2 * q + 1 < end ? v[d][i][q] : 2 * q < end ? v[d][i][q] & 0xFFFFu : 0u;
                    }
            }
        } else {
#pragma unroll
            for (int d = 0; d < 4; ++d) {
                const int64_t k = k0 + d * 32 + (lane >> 4) * 8;
#pragma unroll
                for (int i = 0; i < PIECES; ++i)
                    v[d][i] = load_piece<T>(X + row * ld + k + i * Elem<T>::VEC, row < rows ? K - k - i * Elem<T>::VEC : 0);
            }
        }
    }
    __device__ __forceinline__ void parts(int d, u32x4_t (&p)[sizeof(T) == 4 ? 3 : 1]) const
    {
        if constexpr (sizeof(T) == 4) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                uint32_t p0, p1, p2;
                split2_nearest(__uint_as_float(v[d][i >> 1][2 * (i & 1)]), __uint_as_float(v[d][i >> 1][2 * (i & 1) + 1]), p0,
                               p1, p2);
                p[0][i] = p0;
                p[1][i] = p1;
                p[2][i] = p2;
            }
        } else {
            p[0] = v[d][0];
        }
    }
};

__device__ __forceinline__ float gate_value(int gate, float z)
{
    switch (gate) {
    case kSilu: return gate_act<kSilu>(z);
    case kGelu: return gate_act<kGelu>(z);
    case kGeluTanh: return gate_act<kGeluTanh>(z);
    case kSigmoid: return gate_act<kSigmoid>(z);
    default: return gate_act<kRelu>(z);
    }
}

}  // namespace

}  // namespace sgemm_emu_dev
