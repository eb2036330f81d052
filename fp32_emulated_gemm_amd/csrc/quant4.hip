// quant4.hip -- weights of 4 bits: quantised, packed, unpacked, and their products
// with few rows.
//
// A value q of 0..15 stands for (q - zero) scale.  Packed, a tile of 16 rows by 128
// columns is 1 KB: lane l's 16 bytes hold row l & 15, dword d the columns 32 d + 8
// (l >> 4) + e, e = 0..7, at bits 4 (e >> 1) + 16 (e & 1).  That is the first operand
// of four 16x16x32 MFMAs, so a wave loads a tile in one contiguous access.  Tiles of
// 16 rows follow each other along K.  Behind the values: scales [group][row] in
// FP32, then zeros [group][row], 16 added, in a byte.
//
// A nibble pair becomes two BF16 with a shift and an and-or: 0x4180 is 16, whose
// last four mantissa bits count ones, so 0x4180 | q << 3 is 16 + q, exactly.  With
// xs = the sum of x over the group (an MFMA with ones, shared by all rows of W),
//   sum (q - zero) x = sum (16 + q) x - (16 + zero) xs,
// formed in FP32 and scaled once a group.  The offset of 16 costs two or three of
// FP32's 24 bits (128 + q, one shift less, would cost five).  FP32 rows of X come in
// three BF16 parts; a weight is one, so three products in three bands.
//
// One bfloat16 row of 4096 x 4096 takes 6.4 us (9 MB), bounded by the loads' latency;
// 64 rows over 64 experts of 2816 x 2048, gated, 34.6 us, 123 MB at 3.6 TB/s: vector
// instructions (widening, scales, sums) issue in half of the SIMDs' cycles, MFMAs in a
// twelfth, and waves wait in 37 % of theirs; 16 float32 rows of 8192 x 1024 in groups of
// 32 9.0 us, each wave splitting its rows anew.  Unpacking 4096 x 4096 to bfloat16 takes
// 12.6 us, 42 MB at 3.3 TB/s, a bank of 64 of 2816 x 2048 174, 5.3 TB/s.  Quantising that
// bank takes 728 us, packing 659: once a weight, element by element.
#include <type_traits>

#include "expert_rows.hpp"

namespace sgemm_emu_dev {

namespace {

constexpr int KB = 128;                      // columns of a tile

// ---------------------------------------------------------------- quantise, pack, unpack

// One wave per group and row: 32 to 128 columns.
template <class T>
__global__ __launch_bounds__(256) void quantize_kernel(Quant4 w, const T *W, uint8_t *q, float *scale, uint8_t *zero)
{
    const int lane = threadIdx.x & 63;
    const int64_t groups = (w.K + w.group - 1) / w.group, total = w.n * w.N * groups;
    for (int64_t u = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6); u < total; u += (int64_t)gridDim.x * 4) {
        const int64_t row = u / groups, c = (u - row * groups) * w.group;
        const int64_t left = lmin(w.group, w.K - c);
        float v[2], lo = 0.0f, hi = 0.0f;
        bool finite = true;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int at = lane + 64 * i;
            v[i] = at < left ? Elem<T>::load(W + row * w.K + c + at) : 0.0f;
            lo = fminf(lo, v[i]);
            hi = fmaxf(hi, v[i]);
            finite = finite && __builtin_fabsf(v[i]) <= 3.40282347e38f;
        }
        finite = __all(finite);
#pragma unroll
        for (int d = 32; d > 0; d >>= 1) {
            lo = fminf(lo, __shfl_xor(lo, d));
            hi = fmaxf(hi, __shfl_xor(hi, d));
        }
        float s, z = 8.0f;
        if (zero != nullptr) {
            s = hi * (1.0f / 15.0f) - lo * (1.0f / 15.0f);       // apart: the difference may pass the largest float
            z = s > 0.0f ? fminf(fmaxf(__builtin_rintf(-lo / s), 0.0f), 15.0f) : 0.0f;
        } else {
            s = fmaxf(hi, -lo) * (1.0f / 7.0f);
        }
        // no level past the largest BF16, which the weights may be rounded to
        s = fminf(s, 3.38953139e38f / (zero != nullptr ? fmaxf(z, 15.0f - z) : 7.0f));
        if (!finite) s = __builtin_nanf("");
        const float most = zero != nullptr ? 15.0f - z : 7.0f, least = zero != nullptr ? -z : -7.0f;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int at = lane + 64 * i;
            const float t = s > 0.0f ? __builtin_rintf(v[i] / s) : 0.0f;
            if (at < left) q[row * w.K + c + at] = (uint8_t)(int)(fminf(fmaxf(t, least), most) + z);
        }
        if (lane == 0) {
            scale[u] = s;
            if (zero != nullptr) zero[u] = (uint8_t)(int)z;
        }
    }
}

struct Packed {
    const uint32_t *values;
    const float *scale;
    const uint8_t *zero;
};

__host__ __device__ __forceinline__ Packed packed_bank(const Quant4 &w, const void *packed, int64_t bank)
{
    const char *const p = (const char *)packed + bank * w.bank_bytes();
    return Packed{(const uint32_t *)p, (const float *)(p + w.value_bytes()),
                  (const uint8_t *)(p + w.value_bytes() + w.scale_bytes())};
}

// One thread per dword of values.
__global__ __launch_bounds__(256) void pack_values_kernel(Quant4 w, const uint8_t *q, char *packed)
{
    const int64_t per = w.value_bytes() / 4, total = w.n * per;
    for (int64_t u = (int64_t)blockIdx.x * 256 + threadIdx.x; u < total; u += (int64_t)gridDim.x * 256) {
        const int64_t bank = u / per, at = u - bank * per;
        const int64_t tile = at >> 8, blocks = w.blocks();
        const int l = (int)(at >> 2) & 63, d = (int)at & 3;
        const int64_t row = tile / blocks * 16 + (l & 15), c = tile % blocks * KB + d * 32 + (l >> 4) * 8;
        uint32_t v = 0;
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (row < w.N && c + e < w.K)
                v |= (uint32_t)(q[(bank * w.N + row) * w.K + c + e] & 15) << (4 * (e >> 1) + 16 * (e & 1));
        ((uint32_t *)(packed + bank * w.bank_bytes()))[at] = v;
    }
}

__global__ __launch_bounds__(256) void pack_scales_kernel(Quant4 w, const float *scale, const uint8_t *zero, char *packed)
{
    const int64_t rows = w.rows(), per = w.groups() * rows, total = w.n * per, groups = (w.K + w.group - 1) / w.group;
    for (int64_t u = (int64_t)blockIdx.x * 256 + threadIdx.x; u < total; u += (int64_t)gridDim.x * 256) {
        const int64_t bank = u / per, at = u - bank * per, g = at / rows, row = at - g * rows;
        const bool in = row < w.N && g < groups;
        const int64_t src = (bank * w.N + row) * groups + g;
        char *const p = packed + bank * w.bank_bytes() + w.value_bytes();
        ((float *)p)[at] = in ? scale[src] : 0.0f;
        if (w.zeros) ((uint8_t *)(p + w.scale_bytes()))[at] = in ? 16 + (zero[src] & 15) : 24;
        // spare bytes, read as scales of rows behind the last: nothing that is not finite
        if (at < 16) ((uint32_t *)(p + w.scale_bytes() + w.zero_bytes()))[at] = 0;
    }
}

// A wave takes 16 rows by 128 columns: a tile in one contiguous read, its rows out
// through LDS in whole pieces (a lane's own dwords belong to places 64 bytes apart:
// stored one by one, 4096 x 4096 took 83 us).
//
// In bfloat16 the weight (q - zero) scale is rounded to its 8 bits here, as the operand of
// a bfloat16 product, where the calls of few rows keep it exact: 2047 rows of 4096 x 4096
// have a relative error of 0.00235 against 0.00166 of the output's rounding alone.  Two
// parts (16 bits) reach 0.00166 too, but make the product two: 121 us for 66, and 100 for
// 56 of 512 rows of 11008 x 4096.  float32 calls round once, to 24 bits.
template <class T>
__global__ __launch_bounds__(256) void unpack_kernel(Quant4 w, const void *packed, T *W)
{
    constexpr int PITCH = KB + 16 / sizeof(T);             // rows of LDS, 16 bytes longer
    __shared__ __attribute__((aligned(16))) T buf[4][16 * PITCH];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t blocks = w.blocks(), rows = w.rows(), per = rows / 16 * blocks, total = w.n * per;
    T *const out = buf[wave];
    for (int64_t u = (int64_t)blockIdx.x * 4 + wave; u < total; u += (int64_t)gridDim.x * 4) {
        const int64_t bank = u / per, at = u - bank * per, row0 = at / blocks * 16, c0 = at % blocks * KB;
        const Packed p = packed_bank(w, packed, bank);
        const u32x4_t v = reinterpret_cast<const u32x4_t *>(p.values)[at * 64 + lane];
        const int64_t row = row0 + (lane & 15);
#pragma unroll
        for (int d = 0; d < 4; ++d) {
            const int64_t g = (c0 + d * 32) / w.group * rows + row;
            const float s = p.scale[g], z = w.zeros ? (float)(p.zero[g] - 16) : 8.0f;
            T e8[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) e8[e] = Elem<T>::store(((float)((v[d] >> (4 * (e >> 1) + 16 * (e & 1))) & 15) - z) * s);
            T *const to = out + (lane & 15) * PITCH + d * 32 + (lane >> 4) * 8;
#pragma unroll
            for (int i = 0; i < (int)sizeof(T) / 2; ++i)
                reinterpret_cast<u32x4_t *>(to)[i] = reinterpret_cast<const u32x4_t *>(e8)[i];
        }
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
        constexpr int V = Elem<T>::VEC, PER = KB / V;      // pieces of a row
#pragma unroll
        for (int i = 0; i < 16 * PER / 64; ++i) {
            const int q = i * 64 + lane, r = q / PER, c = q % PER * V;
            const int64_t left = w.K - c0 - c;
            const T *const from = out + r * PITCH + c;
            T *const to = W + (bank * w.N + row0 + r) * w.K + c0 + c;
            if (row0 + r < w.N && left > 0) {
                if (left >= V) {
                    *reinterpret_cast<u32x4_any *>(to) = *reinterpret_cast<const u32x4_t *>(from);
                } else {
                    for (int e = 0; e < left; ++e) to[e] = from[e];
                }
            }
        }
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
    }
}

// ---------------------------------------------------------------- few rows

// Eight values 16 + q of a dword as BF16; SIXTEEN: 16 times a power of two, twice.
template <uint32_t SIXTEEN>
__device__ __forceinline__ bf16x8_t widen(uint32_t w)
{
    u32x4_t v;
    v[0] = ((w << 3) & 0x00780078u) | SIXTEEN;
    v[1] = ((w >> 1) & 0x00780078u) | SIXTEEN;
    v[2] = ((w >> 5) & 0x00780078u) | SIXTEEN;
    v[3] = ((w >> 9) & 0x00780078u) | SIXTEEN;
    return __builtin_bit_cast(bf16x8_t, v);
}

typedef uint32_t u32_any __attribute__((aligned(1)));

__device__ __forceinline__ bool is_finite(float x) { return __builtin_fabsf(x) <= 3.40282347e38f; }

// GROUP columns share a scale.  A workgroup takes NB tiles of 16 rows of W (with a
// gate, NB / 2 of the gate's and those of the up projection's same outputs) and 16 MB
// rows of X at a time, its share of the expert's; its waves take the blocks of 128
// columns in turn, the next block's values loaded under the products of the one before.
template <class T, int WAVES, int NB, int MB, int GROUP, bool LIES>
__global__ __launch_bounds__(64 * WAVES) void quant4_few_kernel(Quant4 w, Quant4Product g)
{
    constexpr int NT = 64 * WAVES, PARTS = sizeof(T) == 4 ? 3 : 1, STEPS = GROUP / 32, GROUPS = KB / GROUP;
    __shared__ __attribute__((aligned(16))) f32x4_t sums[WAVES][NB][MB][64];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const bool gated = g.gate >= 0;
    const int OUT = gated ? NB / 2 * 16 : NB * 16;
    const int64_t e = blockIdx.y, F = gated ? w.N / 2 : w.N, n0 = (int64_t)blockIdx.x * OUT;
    const int64_t r0 = expert_start(g.offsets, e, g.P), r1 = expert_end(g.offsets, e, w.n, g.P);
    const int64_t first = r0 + (int64_t)blockIdx.z * 16 * MB;
    if (first >= r1 || (e >= w.n && blockIdx.z > 0)) return;
    T *const H = (T *)g.H;
    if (e >= w.n) {                                        // rows of no expert
        for (int64_t o = threadIdx.x; o < (r1 - r0) * OUT; o += NT) {
            const int64_t n = n0 + o % OUT;
            if (n < F) H[(r0 + o / OUT) * g.ldh + n] = Elem<T>::store(0.0f);
        }
        return;
    }
    const Packed p = packed_bank(w, g.packed, e);
    const int64_t blocks = w.blocks(), rows = w.rows();
    // First row of W of each tile.  Up rows begin at F, inside a packed tile where F is no
    // multiple of 16.  Rows past the last are other rows' or the bank's spare bytes; their
    // results are dropped.
    const uint32_t *values[NB];
    int64_t srow[NB];
#pragma unroll
    for (int b = 0; b < NB; ++b) {
        const int64_t base = gated ? (b < NB / 2 ? b * 16 : F + (b - NB / 2) * 16) + n0 : n0 + b * 16;
        const int64_t row = lmin(base + (lane & 15), rows - 1);
        values[b] = p.values + (((row >> 4) * blocks) << 8) + (((lane & 48) | (row & 15)) << 2);
        srow[b] = lmin(base, rows - 1) + 4 * (lane >> 4);
    }
    for (int64_t m0 = first; m0 < r1; m0 += 16 * MB * (int64_t)gridDim.z) {
        // The sums over this wave's blocks, of weights times 2^-DOWN.
        auto sum_blocks = [&](f32x4_t (&acc)[NB][MB], auto down) {
            constexpr uint32_t DOWN = decltype(down)::value * 0x00800080u, ONE = 0x3F803F80u - DOWN, SIXTEEN = 0x41804180u - DOWN;
            const bf16x8_t ones = __builtin_bit_cast(bf16x8_t, u32x4_t{ONE, ONE, ONE, ONE});
#pragma unroll
            for (int b = 0; b < NB; ++b)
#pragma unroll
                for (int m = 0; m < MB; ++m) acc[b][m] = f32x4_t{};
            u32x4_t next[NB];
            auto load_values = [&](int64_t kb) {
#pragma unroll
                for (int b = 0; b < NB; ++b) next[b] = *reinterpret_cast<const u32x4_t *>(values[b] + (kb << 8));
            };
            if (wave < blocks) load_values(wave);
            for (int64_t kb = wave; kb < blocks; kb += WAVES) {
                u32x4_t v[NB];
#pragma unroll
                for (int b = 0; b < NB; ++b) v[b] = next[b];
                RowBlock<T> x[MB];
#pragma unroll
                for (int m = 0; m < MB; ++m)
                    x[m].template load<LIES>((const T *)g.X, g.ldx, m0 + m * 16 + (lane & 15), r1, kb * KB, w.K, lane);
                f32x4_t scale[GROUPS][NB];
                uint32_t zero[GROUPS][NB];
#pragma unroll
                for (int gr = 0; gr < GROUPS; ++gr)
#pragma unroll
                    for (int b = 0; b < NB; ++b) {
                        const int64_t at = (kb * GROUPS + gr) * rows + srow[b];
                        scale[gr][b] = __builtin_bit_cast(f32x4_t, (u32x4_t)*reinterpret_cast<const u32x4_any *>(p.scale + at));
                        zero[gr][b] = w.zeros ? *reinterpret_cast<const u32_any *>(p.zero + at) : 0x18181818u;
                    }
                if (kb + WAVES < blocks) load_values(kb + WAVES);
#pragma unroll
                for (int gr = 0; gr < GROUPS; ++gr) {
                    f32x4_t part[PARTS][NB][MB], xs[PARTS][MB];
#pragma unroll
                    for (int q = 0; q < PARTS; ++q)
#pragma unroll
                        for (int m = 0; m < MB; ++m) {
                            xs[q][m] = f32x4_t{};
#pragma unroll
                            for (int b = 0; b < NB; ++b) part[q][b][m] = f32x4_t{};
                        }
#pragma unroll
                    for (int st = 0; st < STEPS; ++st) {
                        const int d = gr * STEPS + st;
                        bf16x8_t wf[NB];
#pragma unroll
                        for (int b = 0; b < NB; ++b) wf[b] = widen<SIXTEEN>(v[b][d]);
#pragma unroll
                        for (int m = 0; m < MB; ++m) {
                            u32x4_t xp[PARTS];
                            x[m].parts(d, xp);
#pragma unroll
                            for (int q = 0; q < PARTS; ++q) {
                                const bf16x8_t xf = __builtin_bit_cast(bf16x8_t, xp[q]);
                                xs[q][m] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(ones, xf, xs[q][m], 0, 0, 0);
#pragma unroll
                                for (int b = 0; b < NB; ++b)
                                    part[q][b][m] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wf[b], xf, part[q][b][m], 0, 0, 0);
                            }
                        }
                        if constexpr (DOWN != 0) __builtin_amdgcn_sched_barrier(0);   // rare: in few registers
                    }
#pragma unroll
                    for (int b = 0; b < NB; ++b)
#pragma unroll
                        for (int q = 0; q < 4; ++q) {
                            const float z = -(float)((zero[gr][b] >> (8 * q)) & 255u);
#pragma unroll
                            for (int m = 0; m < MB; ++m) {
                                float t = __builtin_fmaf(z, xs[0][m][q], part[0][b][m][q]);
                                if constexpr (PARTS == 3) {
                                    const float t1 = __builtin_fmaf(z, xs[1][m][q], part[1][b][m][q]);
                                    const float t2 = __builtin_fmaf(z, xs[2][m][q], part[2][b][m][q]);
                                    t += __builtin_fmaf(t2, 0x1p-16f, t1 * 0x1p-8f);
                                }
                                acc[b][m][q] = __builtin_fmaf(scale[gr][b][q], t, acc[b][m][q]);
                            }
                        }
                    // one group's products at a time: all of a block's together would not fit the registers
                    if constexpr (GROUPS > 1) __builtin_amdgcn_sched_barrier(0);
                }
            }
        };
        f32x4_t acc[NB][MB];
        sum_blocks(acc, std::integral_constant<int, 0>());
        float lost = 0.0f;                                 // NaN where a sum is not finite
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
            for (int m = 0; m < MB; ++m) {
#pragma unroll
                for (int q = 0; q < 4; ++q) lost = __builtin_fmaf(acc[b][m][q], 0.0f, lost);
                sums[wave][b][m][lane] = acc[b][m];
            }
        // The sums of (16 + q) x and (16 + zero) x reach 31 * 128 < 2^12 times the largest |x|.
        // Where that passes the largest float they leave Inf or NaN, though the product may be
        // neither: such a wave takes its blocks again, the weights times 2^-12, for the sums that
        // were lost.
        if (__builtin_expect(__any(lost != lost), 0)) {
            sum_blocks(acc, std::integral_constant<int, 12>());
#pragma unroll
            for (int b = 0; b < NB; ++b)
#pragma unroll
                for (int m = 0; m < MB; ++m) {
                    f32x4_t v = sums[wave][b][m][lane];
#pragma unroll
                    for (int q = 0; q < 4; ++q) v[q] = is_finite(v[q]) ? v[q] : acc[b][m][q] * 0x1p12f;
                    sums[wave][b][m][lane] = v;
                }
        }
        __syncthreads();
        const T *const bias = g.bias != nullptr ? (const T *)g.bias + e * w.N : nullptr;
        auto total = [&](int b, int n, int m) {            // row n of tile b, row m of X
            float v = 0.0f;
#pragma unroll
            for (int i = 0; i < WAVES; ++i) v += sums[i][b][m >> 4][(n >> 2) * 16 + (m & 15)][n & 3];
            return v;
        };
        const int here = (int)lmin(r1 - m0, 16 * MB);
        for (int o = threadIdx.x; o < OUT * here; o += NT) {
            const int n = o % OUT, m = o / OUT;
            if (n0 + n >= F) continue;
            float v = total(n >> 4, n & 15, m);
            if (bias != nullptr) v += Elem<T>::load(bias + n0 + n);
            if (gated) {
                float u = total(NB / 2 + (n >> 4), n & 15, m);
                if (bias != nullptr) u += Elem<T>::load(bias + F + n0 + n);
                v = gate_value(g.gate, v) * u;
            }
            H[(m0 + m) * g.ldh + n0 + n] = Elem<T>::store(v);
        }
        __syncthreads();
    }
}

unsigned blocks_for(int64_t items, int64_t per)
{
    const int64_t b = (items + per - 1) / per;
    return (unsigned)(b < 1 ? 1 : b < 16384 ? b : 16384);
}

template <class T, int WAVES, int NB, int MB, int GROUP, bool LIES>
hipError_t launch_few(const Quant4 &w, const Quant4Product &g, hipStream_t stream)
{
    const int64_t out = g.gate >= 0 ? w.N / 2 : w.N, per = g.gate >= 0 ? NB * 8 : NB * 16;
    // an expert's rows over as many workgroups as the CUs have room for: one after the other
    // they would wait for the same loads again
    const int64_t across = (out + per - 1) / per, with = w.n < g.P ? w.n : g.P;
    int64_t parts = 1;
    if (with > 0) {
        const int64_t each = (g.P + with - 1) / with, most = g.num_cus / (across * with);
        parts = (each + 16 * MB - 1) / (16 * MB);
        parts = parts < most ? parts : most < 1 ? 1 : most;
    }
    const dim3 grid((unsigned)across, (unsigned)(w.n + (g.offsets != nullptr ? 1 : 0)), (unsigned)parts);
    hipLaunchKernelGGL((quant4_few_kernel<T, WAVES, NB, MB, GROUP, LIES>), grid, dim3(64 * WAVES), 0, stream, w, g);
    return hipGetLastError();
}

// Rows of W and X of a workgroup: 16 rows of X where an expert has about as many or
// fewer, else as many as the registers hold beside the groups' scales, so that W
// passes once or twice; of W the more the more rows of X are read beside it, as long
// as there are workgroups for the CUs.
template <class T, int GROUP>
hipError_t few_rows(const Quant4 &w, const Quant4Product &g, hipStream_t stream)
{
    constexpr int MB = sizeof(T) == 2 && GROUP >= 64 ? 4 : 2, NB = GROUP == 128 || (sizeof(T) == 2 && GROUP == 64) ? 4 : 2;
    const bool lies = sizeof(T) == 4 || (g.ldx % 2 == 0 && aligned(g.X, 4));
    const int64_t each = w.n > 0 ? (g.P + w.n - 1) / w.n : 0, tiles = (w.N + 15) / 16 * (w.n < g.P ? w.n : g.P);
    if (!lies) return each <= 16 ? launch_few<T, 8, 2, 1, GROUP, false>(w, g, stream) : launch_few<T, 8, 2, MB, GROUP, false>(w, g, stream);
    if (each > 16) return launch_few<T, 8, 2, MB, GROUP, true>(w, g, stream);
    if (NB > 2 && each > 4 && tiles >= 4 * g.num_cus) return launch_few<T, 8, NB, 1, GROUP, true>(w, g, stream);
    if (g.gate >= 0 || tiles >= 2 * g.num_cus) return launch_few<T, 8, 2, 1, GROUP, true>(w, g, stream);
    return launch_few<T, 16, 1, 1, GROUP, true>(w, g, stream);
}

template <class T>
hipError_t few_group(const Quant4 &w, const Quant4Product &g, hipStream_t stream)
{
    switch (w.group) {
    case 32: return few_rows<T, 32>(w, g, stream);
    case 64: return few_rows<T, 64>(w, g, stream);
    default: return few_rows<T, 128>(w, g, stream);
    }
}

}  // namespace

hipError_t launch_quant4_quantize(int dtype, const Quant4 &w, const void *W, uint8_t *q, float *scale, uint8_t *zero,
                                  hipStream_t stream)
{
    const int64_t groups = w.n * w.N * ((w.K + w.group - 1) / w.group);
    if (groups == 0) return hipSuccess;
    const dim3 grid(blocks_for(groups, 4));
    if (dtype == kF32) hipLaunchKernelGGL(quantize_kernel<float>, grid, dim3(256), 0, stream, w, (const float *)W, q, scale, zero);
    else hipLaunchKernelGGL(quantize_kernel<uint16_t>, grid, dim3(256), 0, stream, w, (const uint16_t *)W, q, scale, zero);
    return hipGetLastError();
}

hipError_t launch_quant4_pack(const Quant4 &w, const uint8_t *q, const float *scale, const uint8_t *zero, void *packed,
                              hipStream_t stream)
{
    const int64_t dwords = w.n * w.value_bytes() / 4;
    if (dwords == 0) return hipSuccess;
    hipLaunchKernelGGL(pack_values_kernel, dim3(blocks_for(dwords, 256)), dim3(256), 0, stream, w, q, (char *)packed);
    hipLaunchKernelGGL(pack_scales_kernel, dim3(blocks_for(w.n * w.groups() * w.rows(), 256)), dim3(256), 0, stream, w,
                       scale, zero, (char *)packed);
    return hipGetLastError();
}

hipError_t launch_quant4_unpack(int dtype, const Quant4 &w, const void *packed, void *W, hipStream_t stream)
{
    const int64_t tiles = w.n * (w.rows() / 16) * w.blocks();
    if (tiles == 0) return hipSuccess;
    const dim3 grid(blocks_for(tiles, 4));
    if (dtype == kF32) hipLaunchKernelGGL(unpack_kernel<float>, grid, dim3(256), 0, stream, w, packed, (float *)W);
    else hipLaunchKernelGGL(unpack_kernel<uint16_t>, grid, dim3(256), 0, stream, w, packed, (uint16_t *)W);
    return hipGetLastError();
}

// A layer's calls of up to 64 rows read the packed weight, and so do a bank's with up to
// 16 rows an expert.  64 rows of 4096 x 4096 take 23 us in bfloat16 (groups of 128),
// unpacked 38 whatever the rows up to 256.  float32 rows stay up to 128 with the larger
// groups: 128 rows of 4096 x 4096 take 50 to 57 us, unpacked 130; of 11008 x 4096 184 to
// 207, unpacked 232.  With groups of 32, 64 rows of those take 41 and 135, unpacked 105
// and 193, and twice the rows twice as long.
//
// A bank's with its rows spread evenly, packed and unpacked (groups of 128): 1024 rows over
// 64 experts of 2816 x 2048, gated, 85 and 359 us in bfloat16, 138 and 978 in float32; 128
// over eight of those 16 and 42, 25 and 87; 4096 over 256 of 1024 x 512 76 and 154, 95 and
// 432.  With nine rows in ten on one expert, whose workgroups then take their rows one pass
// of W after the other, packing gains up to about 8 n rows (512 over the 64: 151 and 281) and
// loses beyond: 302 and 343, but 208 and 57 over 64 of 1024 x 1024, 679 and 160 over the 256.
// The host does not know which it is.
bool quant4_few(int dtype, const Quant4 &w, int64_t P)
{
    const int64_t most = dtype == kF32 && w.group >= 64 ? 2 * kFewRows : kFewRows;
    return P <= most || P <= 16 * w.n;
}

hipError_t launch_quant4_few(int dtype, const Quant4 &w, const Quant4Product &g, hipStream_t stream)
{
    if (g.P == 0 || w.N == 0) return hipSuccess;
    return dtype == kF32 ? few_group<float>(w, g, stream) : few_group<uint16_t>(w, g, stream);
}

}  // namespace sgemm_emu_dev
