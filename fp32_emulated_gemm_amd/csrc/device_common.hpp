// device_common.hpp -- device helpers shared by the kernel files: vector types,
// the XCD-aware tile order, raw buffer loads, LDS hand-offs and waits.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

namespace sgemm_emu_dev {

typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef float f32x16_t __attribute__((ext_vector_type(16)));
typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));

__device__ __forceinline__ int imin(int a, int b) { return a < b ? a : b; }
__device__ __forceinline__ int64_t lmin(int64_t a, int64_t b) { return a < b ? a : b; }

// Tile index v in [0, T) -> (tile_m, tile_n).  Consecutive v are dealt
// round-robin to the 8 XCDs, so v is remapped to give each XCD a contiguous
// run of tiles, and tiles run in groups of group_m tile-rows (column-major
// inside a group) so the tiles an XCD runs at once share A and B panels in
// its L2.
__device__ __forceinline__ void tile_of_index(int v, int T, int tiles_m, int tiles_n, int group_m, int &tm,
                                              int &tn)
{
    const int per = T >> 3, extra = T & 7, xcd = v & 7, idx = v >> 3;
    const int t = xcd * per + imin(xcd, extra) + idx;
    const int group_size = group_m * tiles_n;
    const int group = t / group_size;
    const int first_m = group * group_m;
    const int gm = imin(tiles_m - first_m, group_m);
    const int in = t - group * group_size;
    tm = first_m + in % gm;
    tn = in / gm;
}

typedef __amdgpu_buffer_rsrc_t rsrc_t;
constexpr int RSRC_WORD3 = 0x00020000;   // raw, untyped buffer on gfx9-family GPUs

// Descriptor of `bytes` bytes at `base`.  Callers pass wave-uniform values;
// readfirstlane states that to the compiler, which otherwise may keep a
// value in vector registers and wrap every load in a loop over lanes.
__device__ __forceinline__ rsrc_t make_rsrc(const void *base, int64_t bytes)
{
    const uint32_t n = bytes <= 0 ? 0u : (bytes >= 0xFFFFFFFFll ? 0xFFFFFFFFu : (uint32_t)bytes);
    const uint64_t p = (uint64_t)(uintptr_t)base;
    const uint32_t lo = __builtin_amdgcn_readfirstlane((uint32_t)p);
    const uint32_t hi = __builtin_amdgcn_readfirstlane((uint32_t)(p >> 32));
    void *ub = (void *)(uintptr_t)(((uint64_t)hi << 32) | lo);
    return __builtin_amdgcn_make_buffer_rsrc(ub, (short)0, (int)__builtin_amdgcn_readfirstlane(n), RSRC_WORD3);
}

__device__ __forceinline__ float bload_f32(rsrc_t r, uint32_t off, uint32_t soff)
{
    return __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(r, (int)off, (int)soff, 0));
}

__device__ __forceinline__ uint32_t bload_u32(rsrc_t r, uint32_t off, uint32_t soff)
{
    return __builtin_amdgcn_raw_buffer_load_b32(r, (int)off, (int)soff, 0);
}

__device__ __forceinline__ uint32_t bload_u16(rsrc_t r, uint32_t off, uint32_t soff)
{
    return (uint32_t)__builtin_amdgcn_raw_buffer_load_b16(r, (int)off, (int)soff, 0);
}

__device__ __forceinline__ u32x4_t bload_u32x4(rsrc_t r, uint32_t off, uint32_t soff)
{
    return __builtin_amdgcn_raw_buffer_load_b128(r, (int)off, (int)soff, 0);
}

__device__ __forceinline__ bf16x8_t ld_frag(const uint16_t *p)
{
    return __builtin_bit_cast(bf16x8_t, *reinterpret_cast<const u32x4_t *>(p));
}

// Workgroup barrier for LDS hand-offs: waits for this wave's LDS operations,
// then for the other waves.  Unlike __syncthreads() it does not wait for the
// wave's outstanding LDS-DMA copies (the step that follows issued them for
// later use); callers wait for the copies they need with wait_vmem_at_most.
// The memory clobber keeps the compiler from moving LDS accesses across it.
__device__ __forceinline__ void lds_barrier()
{
    asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
}

__device__ __forceinline__ int bslot(int row, int kg) { return kg ^ ((row >> 2) & 3); }

// Wait until at most n vector-memory operations of this wave are outstanding
// (they complete in issue order), leaving the other counters unconstrained.
template <int N>
__device__ __forceinline__ void wait_vmem_at_most()
{
    static_assert(N >= 0 && N < 64, "vmcnt range");
    __builtin_amdgcn_s_waitcnt((N & 15) | ((N >> 4) << 14) | (0x7 << 4) | (0xF << 8));
}

// GELU in its exact form, 0.5 z (1 + erf(z / sqrt(2))), evaluated as
// 0.5 z erfc(-z / sqrt(2)): the same function, without the cancellation of
// 1 + erf(.) for negative z, so the relative error stays a few ulp.
__device__ __forceinline__ float gelu_erf(float z)
{
    return (0.5f * z) * erfcf(z * -0.70710678118654752f);
}

}  // namespace sgemm_emu_dev
