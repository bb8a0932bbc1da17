// join.h -- workgroups that leave partial results in a workspace, of which the
// last one to arrive joins them.
//
// The order in which results are joined is fixed by their places, so it does
// not matter which workgroup comes last.  Counters are zero before a launch
// and zero again after it: a workspace is zeroed once, by its owner.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace ar {

constexpr int kJoin = 32;  // results that one workgroup joins

// Counters at the start of a workspace whose results are joined in two
// levels: one for the groups, then one for each group.
constexpr int kJoinCounters = 64;
static_assert(kJoinCounters >= 1 + kJoin, "a counter for each group and one for all");

// Every thread of the workgroup calls this after its stores.  True in all
// threads of the workgroup that is the last of `count` to arrive at `counter`:
// that one sees what the others have stored.  `order` is a word of LDS.
__device__ __forceinline__ bool arrive_last(uint32_t *counter, int count, uint32_t *order) {
    // each thread's own stores reach the point where other XCDs read them
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "agent");
    __syncthreads();
    if (threadIdx.x == 0) {
        const uint32_t n = __hip_atomic_fetch_add(counter, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        if (n + 1 == (uint32_t)count)
            __hip_atomic_store(counter, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        *order = n;
    }
    __syncthreads();
    const bool last = *order + 1 == (uint32_t)count;
    __syncthreads();  // `order` may be used again
    if (last) __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "agent");
    return last;
}

}  // namespace ar
