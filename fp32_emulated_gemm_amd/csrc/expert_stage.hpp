// expert_stage.hpp -- tiles staged through registers into LDS, one BF16 plane or
// three (expert_gemm.hip, expert_f32.hip).
#pragma once
#include "expert_device.hpp"

namespace sgemm_emu_dev {

namespace {

constexpr int BK = 32;                       // K step: one MFMA's
typedef short s16x4_t __attribute__((ext_vector_type(4)));

template <int WAVES_M_, int WAVES_N_, int TM_, int TN_>
struct Tile {
    static constexpr int WAVES_M = WAVES_M_, WAVES_N = WAVES_N_, NT = 64 * WAVES_M * WAVES_N;
    static constexpr int TM = TM_, TN = TN_, BM = WAVES_M * TM, BN = WAVES_N * TN;
    static constexpr int MI = TM / 16, NI = TN / 16;
};

// An operand's tile in LDS: R rows (outputs' rows or columns) by BK, one plane after
// another.  !KM: R rows of BK elements.  KM: BK rows of R elements.  16-byte slots
// are permuted so that the fragment reads spread over the banks.
template <class T, int R, bool KM, int PLANES, int NT>
struct Stage {
    static constexpr int PLANE = R * BK, ELEMS = PLANES * PLANE;
    static constexpr int V = Elem<T>::VEC, PIECES = R * BK / V, MINE = PIECES / NT;   // 16 bytes of the operand
    static constexpr int WIDE = KM ? R / 8 : BK / 8;                   // slots of an LDS row
    static constexpr int ROW = WIDE * 8 / V;                           // pieces of a row
    static_assert(PIECES % NT == 0, "pieces split evenly");

    static __device__ __forceinline__ int slot(int row, int c)
    {
        if constexpr (KM) return c ^ ((((row & 3) | ((row >> 1) & 4)) << 1) & (WIDE - 1));
        else return c ^ ((row >> 2) & 3);
    }
    // Offset of chunk c of LDS row `row` in a plane.
    static __device__ __forceinline__ int at(int row, int c) { return row * WIDE * 8 + slot(row, c) * 8; }

    // Offset in a plane of a thread's piece c.  The permutation repeats after 16 rows: one
    // address serves all pieces where they lie so far apart.
    static __device__ __forceinline__ int piece(int thread, int c)
    {
        constexpr int ROWS = NT / ROW;
        const int k = thread % ROW * V;
        if constexpr (ROWS % 16 == 0) return at(thread / ROW, k >> 3) + (k & 7) + c * NT * V;
        else return at(thread / ROW + c * ROWS, k >> 3) + (k & 7);
    }

    // Fragment: k 8 (lane >> 4) .. + 7 of index base + (lane & 15).
    static __device__ __forceinline__ bf16x8_t frag(const uint16_t *plane, int base, int lane)
    {
        if constexpr (KM) {
            typedef __attribute__((address_space(3))) s16x4_t lds_t;
            const int i = lane & 15, col = base + 4 * (i & 3);
            s16x4_t v[2];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int k = 8 * (lane >> 4) + 4 * h + (i >> 2);
                v[h] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_t *)(plane + at(k, col >> 3) + (col & 7)));
            }
            return __builtin_bit_cast(bf16x8_t, __builtin_shufflevector(v[0], v[1], 0, 1, 2, 3, 4, 5, 6, 7));
        } else {
            return ld_frag(plane + at(base + (lane & 15), lane >> 4));
        }
    }
};

// A piece to offset `at` of the planes.
template <class T, class S>
__device__ __forceinline__ void put_piece(uint16_t *buf, int at, const u32x4_t &v)
{
    if constexpr (sizeof(T) == 4) {
        typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
        u32x2 w[3];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            uint32_t p0, p1, p2;
            split2_nearest(__uint_as_float(v[2 * i]), __uint_as_float(v[2 * i + 1]), p0, p1, p2);
            w[0][i] = p0;
            w[1][i] = p1;
            w[2][i] = p2;
        }
#pragma unroll
        for (int q = 0; q < 3; ++q) *reinterpret_cast<u32x2 *>(buf + at + q * S::PLANE) = w[q];
    } else {
        *reinterpret_cast<u32x4_t *>(buf + at) = v;
    }
}

// Four results, columns n.. of a row, `left` of them there.
template <class T>
__device__ __forceinline__ void store4(T *p, const float (&f)[4], int64_t left)
{
    if (left >= 4) {
        if constexpr (sizeof(T) == 4) {
            *reinterpret_cast<u32x4_any *>(p) = u32x4_t{f2u(f[0]), f2u(f[1]), f2u(f[2]), f2u(f[3])};
        } else {
            typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
            *reinterpret_cast<u32x2_any *>(p) = u32x2{pack2(f[0], f[1]), pack2(f[2], f[3])};
        }
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (e < left) p[e] = Elem<T>::store(f[e]);
    }
}

}  // namespace

}  // namespace sgemm_emu_dev
