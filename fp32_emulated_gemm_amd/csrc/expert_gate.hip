// expert_gate.hip -- the gate's backward on sorted rows and the bias gradients.
//
// One pass over Z and dH: a workgroup takes a tile of 64 rows of one expert and 64
// outputs, writes dZ and adds its columns; a second launch adds an expert's tiles
// in order, so the sums are deterministic.  The sums take the unrounded values.  A bfloat16
// dZ is rounded to its 8 bits here, once, as the operand of two bfloat16 products: two parts
// would make each of them two, 460 us more of 8191 x 2048 -> 2 x 1365's step of 770, where
// rounding moves the step's relative error from 0.0017 to 0.0023.  Memory bounds it: 16382 rows of 2 x 1365 in
// bfloat16, 316 MB, take 68 us, 4.6 TB/s (a large copy on this card: 5.2).
#include "expert_device.hpp"

namespace sgemm_emu_dev {

namespace {

constexpr int ROWS = 64, COLS = 64, NT = 256;

// Four elements of a row, `left` of them there (others zero).
__device__ __forceinline__ void load4(float (&f)[4], const float *p, int64_t left)
{
    if (left >= 4) {
        const u32x4_t v = *reinterpret_cast<const u32x4_any *>(p);
#pragma unroll
        for (int e = 0; e < 4; ++e) f[e] = __uint_as_float(v[e]);
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) f[e] = e < left ? p[e] : 0.0f;
    }
}
__device__ __forceinline__ void load4(float (&f)[4], const uint16_t *p, int64_t left)
{
    if (left >= 4) {
        const u32x2_any v = *reinterpret_cast<const u32x2_any *>(p);
#pragma unroll
        for (int e = 0; e < 4; ++e) f[e] = __uint_as_float(e & 1 ? v[e >> 1] & 0xFFFF0000u : v[e >> 1] << 16);
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) f[e] = e < left ? bf2f(p[e]) : 0.0f;
    }
}

// Four elements, columns c.. of a row of dZ (whose pitch is a multiple of 32).
__device__ __forceinline__ void store4(float *p, const float (&f)[4])
{
    *reinterpret_cast<f32x4_t *>(p) = f32x4_t{f[0], f[1], f[2], f[3]};
}
__device__ __forceinline__ void store4(uint16_t *p, const float (&f)[4])
{
    *reinterpret_cast<uint64_t *>(p) = (uint64_t)pack2(f[0], f[1]) | (uint64_t)pack2(f[2], f[3]) << 32;
}

template <class T, int GATE>
__global__ __launch_bounds__(NT) void expert_gate_kernel(ExpertGate g)
{
    constexpr int PARTS = GATE >= 0 ? 2 : 1;
    __shared__ float sums[PARTS][16][COLS];
    const int lane = threadIdx.x & 63, q = (threadIdx.x & 15) * 4, hi = threadIdx.x >> 4;
    const RowTile t = RowTiles<ROWS>(g.offsets, g.n, g.P, (int)g.n, lane).find((int)blockIdx.x);
    if (t.segment < 0) return;
    const int64_t c = (int64_t)blockIdx.y * COLS + q, left = g.F - c, h = expert_dz_pitch(g.F) / 2, zp = z_pitch(g.F);
    float sg[4] = {0, 0, 0, 0}, su[4] = {0, 0, 0, 0};
    // all loads first; rows past the tile re-read its last one
    float d[ROWS / 16][4], zg[ROWS / 16][4], zu[ROWS / 16][4];
#pragma unroll
    for (int i = 0; i < ROWS / 16; ++i) {
        const int64_t r = lmin(t.row + hi + 16 * i, t.end - 1);
        load4(d[i], (const T *)g.dH + r * g.lddh + c, left);
        if constexpr (GATE >= 0) {
            load4(zg[i], g.Z + r * zp + c, left);
            load4(zu[i], g.Z + r * zp + zp / 2 + c, left);
        }
    }
#pragma unroll
    for (int i = 0; i < ROWS / 16; ++i) {
        const int64_t r = t.row + hi + 16 * i;
        if (r >= t.end) break;
        if constexpr (GATE < 0) {
#pragma unroll
            for (int e = 0; e < 4; ++e) sg[e] += d[i][e];
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                float a, slope;
                gate_act_grad<GATE>(zg[i][e], a, slope);
                zg[i][e] = e < left ? d[i][e] * zu[i][e] * slope : 0.0f;
                zu[i][e] = e < left ? d[i][e] * a : 0.0f;
                sg[e] += zg[i][e];
                su[e] += zu[i][e];
            }
            if (g.dZ != nullptr && c < h) {
                T *const out = (T *)g.dZ + r * 2 * h + c;
                store4(out, zg[i]);
                store4(out + h, zu[i]);
            }
        }
    }
    if (g.sums == nullptr) return;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        sums[0][hi][q + e] = sg[e];
        if constexpr (PARTS == 2) sums[1][hi][q + e] = su[e];
    }
    __syncthreads();
    for (int o = threadIdx.x; o < PARTS * COLS; o += NT) {
        const int part = o / COLS, col = o % COLS;
        const int64_t f = (int64_t)blockIdx.y * COLS + col;
        if (f >= g.F) continue;
        float v = 0.0f;
#pragma unroll
        for (int i = 0; i < 16; ++i) v += sums[part][i][col];
        g.sums[(int64_t)blockIdx.x * PARTS * g.F + part * g.F + f] = v;
    }
}

template <class T>
__global__ __launch_bounds__(NT) void expert_sum_kernel(ExpertGate g, int64_t cols)
{
    const int lane = threadIdx.x & 63, e = (int)blockIdx.y;
    int before = 0;
    for (int i = lane; i < e; i += 64) before += count_tiles<ROWS>(g.offsets, g.n, g.P, i, (int)g.n);
    before = __builtin_amdgcn_readfirstlane(wave_sum(before));
    // offsets that do not ascend may count more tiles than there are
    const int most = (int)expert_gate_tiles(g.P, g.n), mine = count_tiles<ROWS>(g.offsets, g.n, g.P, e, (int)g.n);
    const int tiles = imin(mine, most - imin(before, most));
    const int64_t c = (int64_t)blockIdx.x * NT + threadIdx.x;
    if (c >= cols) return;
    float v = 0.0f;
#pragma unroll 8
    for (int t = 0; t < tiles; ++t) v += g.sums[(int64_t)(before + t) * cols + c];
    ((T *)g.dbias)[(int64_t)e * cols + c] = Elem<T>::store(v);
}

template <class T, int GATE>
hipError_t launch(const ExpertGate &g, hipStream_t stream)
{
    const int64_t width = GATE >= 0 ? expert_dz_pitch(g.F) / 2 : g.F, tiles = expert_gate_tiles(g.P, g.n);
    if (tiles > 0 && width > 0)
        hipLaunchKernelGGL((expert_gate_kernel<T, GATE>), dim3((unsigned)tiles, (unsigned)((width + COLS - 1) / COLS)),
                           dim3(NT), 0, stream, g);
    if (g.dbias != nullptr) {
        const int64_t cols = GATE >= 0 ? 2 * g.F : g.F;
        if (cols > 0 && g.n > 0)
            hipLaunchKernelGGL(expert_sum_kernel<T>, dim3((unsigned)((cols + NT - 1) / NT), (unsigned)g.n), dim3(NT), 0,
                               stream, g, cols);
    }
    return hipGetLastError();
}

template <class T>
hipError_t launch_gate(const ExpertGate &g, hipStream_t stream)
{
    switch (g.gate) {
    case kSilu: return launch<T, kSilu>(g, stream);
    case kGelu: return launch<T, kGelu>(g, stream);
    case kGeluTanh: return launch<T, kGeluTanh>(g, stream);
    case kSigmoid: return launch<T, kSigmoid>(g, stream);
    case kRelu: return launch<T, kRelu>(g, stream);
    default: return launch<T, -1>(g, stream);
    }
}

}  // namespace

hipError_t launch_expert_gate(int dtype, const ExpertGate &g, hipStream_t stream)
{
    return dtype == kF32 ? launch_gate<float>(g, stream) : launch_gate<uint16_t>(g, stream);
}

}  // namespace sgemm_emu_dev
