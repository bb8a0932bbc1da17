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

// Results pass between XCDs, each of which has an L2 of its own: they are
// stored through to the device's coherence point and loaded from it (agent
// scope), like the packets of the low-latency calls.  That needs no write-back
// of the whole L2, which a release fence of that scope does: with fences, 1024
// workgroups of the head norms' gradient took 187 us against 45 for their data.
typedef float f32x4_t __attribute__((ext_vector_type(4)));

__device__ __forceinline__ void store_shared(float *p, float v) {
    __hip_atomic_store(p, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ float load_shared(const float *p) {
    return __hip_atomic_load(const_cast<float *>(p), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
// Four at once, as two words of 8 bytes: each float is whole, which is all
// that is asked (the counter orders them).
__device__ __forceinline__ void store_shared(float *p, f32x4_t v) {
    const float w[4] = {v[0], v[1], v[2], v[3]};
    uint64_t *q = reinterpret_cast<uint64_t *>(p);
    __hip_atomic_store(q, __float_as_uint(w[0]) | (uint64_t)__float_as_uint(w[1]) << 32, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    __hip_atomic_store(q + 1, __float_as_uint(w[2]) | (uint64_t)__float_as_uint(w[3]) << 32, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ f32x4_t load_shared4(const float *p) {
    uint64_t *q = reinterpret_cast<uint64_t *>(const_cast<float *>(p));
    const uint64_t a = __hip_atomic_load(q, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    const uint64_t b = __hip_atomic_load(q + 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    return f32x4_t{__uint_as_float((uint32_t)a), __uint_as_float((uint32_t)(a >> 32)), __uint_as_float((uint32_t)b),
                   __uint_as_float((uint32_t)(b >> 32))};
}

// Every thread of the workgroup calls this after its store_shared.  True in
// all threads of the workgroup that is the last of `count` to arrive at
// `counter`: its load_shared sees what the others have stored.  `order` is a
// word of LDS.
__device__ __forceinline__ bool arrive_last(uint32_t *counter, int count, uint32_t *order) {
    // this wave's stores have reached the coherence point; the barrier makes
    // that so for the workgroup's, before its arrival is counted
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
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
    return last;
}

}  // namespace ar
