// item_ring.cuh -- how a persistent kernel's producer hands its work items to the CTA's
// other warps.
#pragma once

#include "ptx.cuh"

namespace diffattn {

// Work items are published by the producer thread into a small ring in shared
// memory; every consumer warp reads the same sequence.  With a scheduler
// counter each CTA claims its next item from a global counter when it needs
// one, so SMs that run slower simply take fewer items; without one, CTA c takes
// a static sequence.  -1 ends the sequence.
template <int SLOTS>
struct ItemRing {
    uint64_t* full;         // [SLOTS] producer -> consumers
    uint64_t* empty;        // [SLOTS] an arrival of each consumer
    volatile int* slots;
    const AbortState* ab;
    // producer
    __device__ __forceinline__ bool put(int k, int idx) const {
        const int s = k % SLOTS;
        if (k >= SLOTS && !mbar_wait(&empty[s], (uint32_t)(k / SLOTS - 1) & 1u, *ab)) return false;
        slots[s] = idx;
        mbar_arrive(&full[s]);
        return true;
    }
    // consumer side, single thread (the MMA-issuing thread of its warp)
    __device__ __forceinline__ bool get_one(int k, int& idx) const {
        const int s = k % SLOTS;
        if (!mbar_wait(&full[s], (uint32_t)(k / SLOTS) & 1u, *ab)) return false;
        idx = slots[s];
        mbar_arrive(&empty[s]);
        return true;
    }
    // consumer side, whole warp (all lanes call; lane 0 arrives for the warp)
    __device__ __forceinline__ bool get(int k, int& idx) const {
        const int s = k % SLOTS;
        if (!mbar_wait_warp(&full[s], (uint32_t)(k / SLOTS) & 1u, *ab)) return false;
        idx = slots[s];
        __syncwarp();
        if ((threadIdx.x & 31) == 0) mbar_arrive(&empty[s]);
        return true;
    }
};

}  // namespace diffattn
