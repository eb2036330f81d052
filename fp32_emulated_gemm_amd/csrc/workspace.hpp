// workspace.hpp -- the per-stream workspace (api.hip) as one call holds it, and the
// FP32 products of the operators that share it.  Not part of the public headers.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <mutex>

#include "launch.hpp"

namespace sgemm_emu_dev {

// A stream's block in the device's table.
struct StreamWs {
    bool used = false;
    uintptr_t key = 0;           // the stream handle
    void *ptr = nullptr;
    size_t bytes = 0;
    hipEvent_t done = nullptr;   // recorded on the stream after the last call that used ptr
    bool recorded = false;
    uint64_t tick = 0;           // last use, for eviction
    uint32_t epoch = 0;          // stream-K flag value of the block's last launch (flags start at 0)
};

// Lease on a workspace for one call; release() after the call's last launch.
struct WsLease {
    std::unique_lock<std::mutex> lock;
    StreamWs *entry = nullptr;
    hipStream_t stream = nullptr;
    char *ptr = nullptr;         // the caller's bytes (behind the flags)
    size_t bytes = 0;            // and how many
    uint32_t *flags = nullptr;   // the block's stream-K flags (its first kFlagBytes)
    uint32_t epoch = 0;          // this call's flag value
    bool attached = false;       // the last kernel that used the block carries its event

    // The event of the held block, for the launch helpers to tie to the call's
    // last kernel (a separate event record costs the stream a few microseconds).
    void *event() const { return entry != nullptr ? (void *)entry->done : nullptr; }

    // Moves on to the flag value of a further launch.
    void next_epoch()
    {
        entry->epoch = entry->epoch == UINT32_MAX ? 1 : entry->epoch + 1;
        epoch = entry->epoch;
    }

    // tied: the call's last kernel already carries the event.
    void release(bool tied)
    {
        if (entry != nullptr) entry->recorded = tied || hipEventRecord(entry->done, stream) == hipSuccess;
        entry = nullptr;
        if (lock.owns_lock()) lock.unlock();
    }
    ~WsLease() { release(attached); }
};

// C = A B^T of these sizes, as gemm_padded_planes runs it.
struct PlaneProduct {
    int64_t M, N, K;
};

// What a call's products need of its stream's workspace, held until the lease
// ends.  Taken before the call's first launch, so that a call that is refused
// for want of it (SGEMM_EMU_ECAPTURE, SGEMM_EMU_ENOMEM) has enqueued nothing.
int lease_plane_workspace(const PlaneProduct *products, int count, hipStream_t stream, WsLease &lease);

// C = A B^T with FP32 A (M x K, lda) and B as zero-padded planes
// (launch_split_padded of an N x K matrix), nine products, by `launch`'s kernels;
// `lease` from lease_plane_workspace with this product among the call's.
int gemm_padded_planes(const GemmArgs &args, const PlaneLaunchers &launch, WsLease &lease, hipStream_t stream);

}  // namespace sgemm_emu_dev
