// bf16_tile.hpp -- tiles of the bfloat16 products (bf16_gemm.hip, expert_bf16.hip):
// shapes, fragments, the order of a step and the way of the results out.
#pragma once
#include "ops_device.hpp"

namespace sgemm_emu_dev {

namespace {

constexpr int KS = 64;                       // K step

template <int WAVES_M_, int WAVES_N_, int TM_, int TN_, int RING_, int PER_CU_>
struct Tile {
    static constexpr int RING = RING_, PER_CU = PER_CU_;           // ring buffers, workgroups per CU
    static constexpr int WAVES_M = WAVES_M_, WAVES_N = WAVES_N_, WAVES = WAVES_M * WAVES_N, NT = 64 * WAVES;
    static constexpr int TM = TM_, TN = TN_;                       // one wave's part
    static constexpr int BM = WAVES_M * TM, BN = WAVES_N * TN;
    static constexpr int MI = TM / 16, NI = TN / 16;
    static constexpr int A_COPIES = BM / 8 / WAVES, B_COPIES = BN / 8 / WAVES;   // 8-row copies per wave and step
    static constexpr int STAGE = (BM + BN) * KS;                   // BF16 elements of one ring buffer
    static constexpr int PITCH = TN + 8;                           // epilogue rows: an odd number of 16-byte slots
    static constexpr int EPI_WAVE = TM * PITCH;
    static constexpr int LDS = RING * STAGE > WAVES * EPI_WAVE ? RING * STAGE : WAVES * EPI_WAVE;
    static_assert(BM % (8 * WAVES) == 0 && BN % (8 * WAVES) == 0, "tile rows split into 8-row copies");
};

using Tile256 = Tile<2, 4, 128, 64, 2, 1>;        // 8 waves
using Tile128 = Tile<2, 2, 64, 64, 2, 2>;         // 4 waves
using Tile128Deep = Tile<2, 4, 64, 32, 4, 1>;     // 8 waves: a CU of its own, its loads further ahead
using Tile64 = Tile<2, 2, 32, 32, 4, 2>;          // 4 waves

constexpr uint32_t OUT_OF_RANGE = 0xFFFFFFF0u;   // past every descriptor: reads zeros

template <class T>
struct Frag {
    bf16x8_t a[T::MI], b[T::NI];
};

// 16-byte slot of k group kg (8 elements) of tile row `row`.
__device__ __forceinline__ int kslot(int row, int kg) { return kg ^ ((row >> 1) & 7); }

// Fragments of a slice of 32 k: lane l holds k 8 (l >> 4) .. + 7 of row l & 15 of each block.
template <class T>
__device__ __forceinline__ void read_frag(Frag<T> &f, const uint16_t *buf, int slice, int wm, int wn, int lane)
{
    const int kg = slice * 4 + (lane >> 4);
#pragma unroll
    for (int j = 0; j < T::NI; ++j) {
        const int row = wn * T::TN + j * 16 + (lane & 15);
        f.b[j] = ld_frag(buf + T::BM * KS + row * KS + kslot(row, kg) * 8);
    }
#pragma unroll
    for (int i = 0; i < T::MI; ++i) {
        const int row = wm * T::TM + i * 16 + (lane & 15);
        f.a[i] = ld_frag(buf + row * KS + kslot(row, kg) * 8);
    }
}

// Waits until at most N of this wave's copies are outstanding and its fragment
// reads are done, then for the other waves.  Builtins, so that the compiler knows
// the reads have arrived and adds no waits of its own.
template <int N>
__device__ __forceinline__ void step_barrier()
{
    static_assert(N >= 0 && N < 64, "vmcnt range");
    __builtin_amdgcn_sched_barrier(0);
    __builtin_amdgcn_s_waitcnt((N & 15) | ((N >> 4) << 14) | (0x7 << 4));
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
}

// Schedules N reads (and N2 copies) one behind each of the first of NM MFMAs:
// issued together they would hold the MFMAs back; left to the compiler, they sink
// to the end and the next barrier waits for them.
template <int NM, int N, int KIND, int N2 = 0, int KIND2 = 0>
__device__ __forceinline__ void spread()
{
    constexpr int PER = (N + N2 + NM - 1) / NM;
#pragma unroll
    for (int q = 0; q < (N + PER - 1) / PER; ++q) {
        __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
        __builtin_amdgcn_sched_group_barrier(KIND, PER, 0);
    }
    if constexpr (N2 > 0) {
#pragma unroll
        for (int q = 0; q < (N2 + PER - 1) / PER; ++q) {
            __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
            __builtin_amdgcn_sched_group_barrier(KIND2, PER, 0);
        }
    }
}

template <class T>
__device__ __forceinline__ void mfma_slice(f32x4_t (&acc)[T::NI][T::MI], const Frag<T> &f)
{
#pragma unroll
    for (int i = 0; i < T::MI; ++i)
#pragma unroll
        for (int j = 0; j < T::NI; ++j)
            acc[j][i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(f.b[j], f.a[i], acc[j][i], 0, 0, 0);
}

// One wave's TM x W block of BF16 results in LDS (rows of PITCH elements) ->
// rows m0w.., columns c0.. of a matrix of `cols` columns, in 128-bit stores
// whatever the rows' alignment (the hardware takes any), the last columns one by
// one.
template <class T, int W>
__device__ __forceinline__ void flush_block(const uint16_t *buf, uint16_t *out, int64_t ld, int64_t M, int64_t cols,
                                            int64_t m0w, int64_t c0, int lane)
{
    constexpr int PER_ROW = W / 8, ROWS = 64 / PER_ROW;            // lanes per row, rows per pass
    const int c = (lane % PER_ROW) * 8;
    const int64_t left = cols - (c0 + c);                          // columns from this lane's first on
    const uint16_t *src = buf + lane / PER_ROW * T::PITCH + c;
    uint16_t *dst = out + (m0w + lane / PER_ROW) * ld + c0 + c;
    const int rows = (int)lmin(M - m0w, T::TM) - lane / PER_ROW;
#pragma unroll 4
    for (int p = 0; p < T::TM; p += ROWS, src += ROWS * T::PITCH, dst += ROWS * ld) {
        const u32x4_t v = *reinterpret_cast<const u32x4_t *>(src);
        if (p < rows && left >= 8) *reinterpret_cast<u32x4_any *>(dst) = v;
    }
    if (left <= 0 || left >= 8) return;
    src -= T::TM * T::PITCH;
    dst -= T::TM * ld;
    for (int p = 0; p < rows; p += ROWS, src += ROWS * T::PITCH, dst += ROWS * ld)
        for (int e = 0; e < left; ++e) dst[e] = src[e];
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

}  // namespace

}  // namespace sgemm_emu_dev
