// ops_device.hpp -- device helpers of the operators: element types, the gates
// and their derivatives.
#pragma once
#include "device_common.hpp"

namespace sgemm_emu_dev {

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

__device__ __forceinline__ float sigmoidf(float z) { return 1.0f / (1.0f + __expf(-z)); }

// act(z) of a gate.
template <int GATE>
__device__ __forceinline__ float gate_act(float z)
{
    if constexpr (GATE == kSilu) return z * sigmoidf(z);
    else if constexpr (GATE == kGelu) return gelu_erf(z);
    else if constexpr (GATE == kGeluTanh) return z * sigmoidf(1.5957691216057308f * z * (1.0f + 0.044715f * z * z));
    else if constexpr (GATE == kSigmoid) return sigmoidf(z);
    else return z > 0.0f ? z : (z == z ? 0.0f : z);
}

// act(z) and act'(z).
template <int GATE>
__device__ __forceinline__ void gate_act_grad(float z, float &a, float &d)
{
    if constexpr (GATE == kSilu) {
        const float s = sigmoidf(z);
        a = z * s;
        d = s * (1.0f + z * (1.0f - s));
    } else if constexpr (GATE == kGelu) {
        const float cdf = 0.5f * erfcf(z * -0.70710678118654752f);
        a = z * cdf;
        d = cdf + z * (0.3989422804014327f * __expf(-0.5f * z * z));
    } else if constexpr (GATE == kGeluTanh) {
        // 0.5 (1 + tanh(v)) = sigmoid(2 v)
        const float s = sigmoidf(1.5957691216057308f * z * (1.0f + 0.044715f * z * z));
        a = z * s;
        d = s + z * s * (1.0f - s) * (1.5957691216057308f * (1.0f + 0.134145f * z * z));
    } else if constexpr (GATE == kSigmoid) {
        const float s = sigmoidf(z);
        a = s;
        d = s * (1.0f - s);
    } else {
        a = gate_act<kRelu>(z);
        d = z > 0.0f ? 1.0f : (z == z ? 0.0f : z);
    }
}

// The tail of a float's significand after rounding to BF16, as BF16: v is
// hi + lo to 16 bits or more.
__device__ __forceinline__ void split_hi_lo(float v, uint16_t &hi, uint16_t &lo)
{
    hi = f2bf(v);
    const float rest = v - bf2f(hi);
    // Inf - Inf (an infinite or overflowing v) would turn the sum into NaN
    lo = rest == rest ? f2bf(rest) : (uint16_t)0;
}

}  // namespace sgemm_emu_dev
