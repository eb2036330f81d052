// abi_checks.hpp -- argument checks and workspace layouts shared by the operators'
// C ABI files (ops_api.hip, experts_api.hip).  Not part of the public headers.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/sgemm_emu_ops.h"
#include "ops.hpp"

namespace {

using namespace sgemm_emu_dev;

constexpr int64_t kMaxBytes = INT64_MAX / 8;
constexpr int64_t kMaxLd = ((int64_t)1 << 32) / (128 * 4) - 64;   // as the GEMM's: 128-row tiles in 32-bit offsets
constexpr int64_t kMaxExtent = 65535 * 64;                        // grid extents of 64-wide tiles
constexpr int64_t kMaxAdapters = 65535;
constexpr int64_t kMaxBankElems = (int64_t)1 << 55;               // n r (K + N)

int64_t size_of(int dtype) { return dtype == SGEMM_EMU_F32 ? 4 : 2; }
bool dtype_ok(int dtype) { return dtype == SGEMM_EMU_F32 || dtype == SGEMM_EMU_BF16; }
bool extent_ok(int64_t v) { return v >= 0 && v <= kMaxExtent; }

// A rows x cols operand: its leading dimension, extent, pointer and alignment.
int check_operand(int dtype, int64_t rows, int64_t cols, const void *p, int64_t ld, bool optional = false)
{
    if (optional && p == nullptr) return SGEMM_EMU_OK;
    if (ld < (cols > 1 ? cols : 1) || ld > kMaxLd) return SGEMM_EMU_EINVAL;
    if (rows > 1 && cols > 0 && rows - 1 > (kMaxBytes - cols) / ld) return SGEMM_EMU_EINVAL;
    if (rows > 0 && cols > 0 && p == nullptr) return SGEMM_EMU_ENULL;
    if ((uintptr_t)p % (uintptr_t)size_of(dtype) != 0) return SGEMM_EMU_EINVAL;
    return SGEMM_EMU_OK;
}

int check_vector(int64_t n, const void *p, int64_t elem, bool optional)
{
    if (p == nullptr) return optional || n == 0 ? SGEMM_EMU_OK : SGEMM_EMU_ENULL;
    return (uintptr_t)p % (uintptr_t)elem != 0 ? SGEMM_EMU_EINVAL : SGEMM_EMU_OK;
}

#define CHECK(call)                                 \
    do {                                            \
        const int rc_ = (call);                     \
        if (rc_ != SGEMM_EMU_OK) return rc_;        \
    } while (0)

#define LAUNCH(call)                                          \
    do {                                                      \
        if ((call) != hipSuccess) return SGEMM_EMU_ELAUNCH;   \
    } while (0)

// Lays buffers out one after another, 256-byte aligned; without a base it only
// adds up their sizes.
struct Carve {
    char *base;
    int64_t bytes = 0;
    explicit Carve(void *ws) : base((char *)ws) {}
    template <class T>
    T *take(int64_t n)
    {
        T *const p = base != nullptr && n > 0 ? (T *)(base + bytes) : nullptr;
        bytes += round_up(n * (int64_t)sizeof(T), 256);
        return p;
    }
};

int check_ws(const void *ws, int64_t ws_bytes, int64_t need)
{
    if (need == 0) return SGEMM_EMU_OK;
    if (ws == nullptr) return SGEMM_EMU_ENULL;
    if ((uintptr_t)ws % 256 != 0 || ws_bytes < need) return SGEMM_EMU_EINVAL;
    return SGEMM_EMU_OK;
}

}  // namespace
