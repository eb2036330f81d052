// ops_device.hpp -- device helpers of the operators: element types, the gates
// and their derivatives.
#pragma once
#include "device_common.hpp"

namespace sgemm_emu_dev {

// 16 and 8 bytes at any address of an element: the hardware takes unaligned
// vector accesses, at the cost of a line more where one is crossed.
typedef u32x4_t u32x4_any __attribute__((aligned(2)));
typedef uint32_t u32x2_any __attribute__((ext_vector_type(2), aligned(2)));

enum { kF32 = 0, kBF16 = 1 };                                      // sgemm_emu_dtype
enum { kSilu = 0, kGelu = 1, kGeluTanh = 2, kSigmoid = 3, kRelu = 4, kGates = 5 };   // sgemm_emu_gate

typedef float f32x4_t __attribute__((ext_vector_type(4)));

__device__ __forceinline__ float bf2f(uint16_t b) { return __uint_as_float((uint32_t)b << 16); }

// Round to nearest even; NaN stays NaN (the compiler's conversion).
__device__ __forceinline__ uint16_t f2bf(float f) { return __builtin_bit_cast(uint16_t, (__bf16)f); }

__device__ __forceinline__ uint32_t pack2(float lo, float hi)
{
    return (uint32_t)f2bf(lo) | ((uint32_t)f2bf(hi) << 16);
}

template <class T>
struct Elem;
template <>
struct Elem<float> {
    static constexpr int VEC = 4;                                  // elements of a 128-bit load
    static __device__ __forceinline__ float load(const float *p) { return *p; }
    static __device__ __forceinline__ float store(float v) { return v; }
};
template <>
struct Elem<uint16_t> {
    static constexpr int VEC = 8;
    static __device__ __forceinline__ float load(const uint16_t *p) { return bf2f(*p); }
    static __device__ __forceinline__ uint16_t store(float v) { return f2bf(v); }
};

// Row of a gated weight (F gate rows, then F up rows) behind row n0 + c of a product's
// tile: alternating blocks of 16 gate and 16 up rows, so that both of an output meet in
// one lane.  Rows past the last are the last.
__device__ __forceinline__ int64_t gated_row(int64_t F, int64_t n0, int c)
{
    const int64_t f = lmin((n0 >> 1) + ((c >> 5) << 4) + (c & 15), F - 1);
    return (c & 16) ? F + f : f;
}

// 1 / (1 + exp(-z)) on the hardware's exp2 and reciprocal (1 ulp each): the
// rounding of z log2(e) leaves |z| 2^-24 or so of relative error.
__device__ __forceinline__ float sigmoidf(float z)
{
    return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(z * -1.44269504f));
}

// The normal distribution's upper tail 0.5 erfc(|z| / sqrt(2)) and exp(-z^2 / 2).
// erfc(x) = exp(-x^2) t Q(t) with t = 1 / (1 + x / 2) and Q a polynomial fitted
// to erfcx(x) / t (relative error 5e-8 over x <= 14).  exp(-z^2 / 2) = 2^n 2^f
// with f formed by FMAs from the exact square and a two-part log2(e), so the
// relative error does not grow with z.  No branches: the compiler's erfcf costs
// twice the time in the backward pass and in the GEMMs' epilogues.
__device__ __forceinline__ float normal_tail(float z, float &e)
{
    const float a = fminf(__builtin_fabsf(z), 20.0f);             // 2^-288: zero from there on
    const float h = a * a, l = __builtin_fmaf(a, a, -h);
    const float n = __builtin_rintf(h * -0.72134752f);
    float f = __builtin_fmaf(h, -0.72134752f, -n);
    f = __builtin_fmaf(h, -9.62981517e-09f, f);
    f = __builtin_fmaf(l, -0.72134752f, f);
    e = __builtin_amdgcn_ldexpf(__builtin_amdgcn_exp2f(f), (int)n);
    const float t = __builtin_amdgcn_rcpf(__builtin_fmaf(a, 0.35355339f, 1.0f));
    float q = -0.0593863646f;
    q = __builtin_fmaf(q, t, 0.286123563f);
    q = __builtin_fmaf(q, t, -0.490405697f);
    q = __builtin_fmaf(q, t, 0.281732714f);
    q = __builtin_fmaf(q, t, -0.0291482948f);
    q = __builtin_fmaf(q, t, 0.203752499f);
    q = __builtin_fmaf(q, t, 0.242835103f);
    q = __builtin_fmaf(q, t, 0.282412103f);
    q = __builtin_fmaf(q, t, 0.282084331f);
    return 0.5f * e * (t * q);
}

// act(z) and act'(z) of a gate.
template <int GATE>
__device__ __forceinline__ void gate_act_grad(float z, float &a, float &d)
{
    if constexpr (GATE == kSilu) {
        const float s = sigmoidf(z);
        a = z * s;
        d = s * (1.0f + z * (1.0f - s));
    } else if constexpr (GATE == kGelu) {
        float e;
        const float tail = normal_tail(z, e), cdf = z < 0.0f ? tail : 1.0f - tail;
        a = z * cdf;
        d = cdf + z * (0.3989422804014327f * e);
    } else if constexpr (GATE == kGeluTanh) {
        // 0.5 (1 + tanh(v)) = sigmoid(2 v)
        const float s = sigmoidf(1.5957691216057308f * z * (1.0f + 0.044715f * z * z));
        a = z * s;
        // s is 0 or 1 from |z| = 12 on; the square stops there, before it is Inf and its
        // product with s (1 - s) = 0 NaN
        d = s + z * s * (1.0f - s) * (1.5957691216057308f * (1.0f + fminf(0.134145f * z * z, 1e6f)));
    } else if constexpr (GATE == kSigmoid) {
        const float s = sigmoidf(z);
        a = s;
        d = s * (1.0f - s);
    } else {
        a = z > 0.0f ? z : (z == z ? 0.0f : z);
        d = z > 0.0f ? 1.0f : (z == z ? 0.0f : z);
    }
}

// act(z) alone.
template <int GATE>
__device__ __forceinline__ float gate_act(float z)
{
    float a, d;
    gate_act_grad<GATE>(z, a, d);
    return a;
}

// A float as two BF16: hi + lo is v to 16 bits or more.  Infinities and NaN stay in
// hi.  A finite v beyond the largest BF16 (3.3895e38, where hi would round to
// Inf and hi + lo to NaN) takes that as hi, and a lo cut off rather than rounded,
// so that the sum stays below 2^128.
__device__ __forceinline__ void split_hi_lo(float v, uint16_t &hi, uint16_t &lo)
{
    constexpr uint32_t INF = 0x7F80, MOST = 0x7F7F;
    const uint32_t bits = __float_as_uint(v), sign = (bits >> 16) & 0x8000u;
    const bool finite = (bits & 0x7FFFFFFFu) < 0x7F800000u;
    hi = f2bf(v);
    const bool over = finite && (hi & 0x7FFFu) == INF;
    if (over) hi = (uint16_t)(sign | MOST);
    const float rest = v - bf2f(hi);             // exact
    const uint16_t cut = (uint16_t)(__float_as_uint(rest) >> 16), near = f2bf(rest);
    lo = !finite ? (uint16_t)0 : over ? cut : near;
}

}  // namespace sgemm_emu_dev
