// rows.h -- rows of bf16 channels of the attention operators: an array
// (tokens, heads, dim) with the strides of the caller, whose channels are
// contiguous.  Eight channels are one lane's share of a row.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "device.h"
#include "host.h"

namespace ar {

struct Rows {
    const uint16_t *p;
    int64_t ts, hs;  // elements from token to token, from head to head
};

inline Rows rows(const RowsArg &r) {
    return Rows{static_cast<const uint16_t *>(r.r.p), r.r.token_stride, r.r.head_stride};
}

// VEC: 16-byte accesses; without it, element by element, for rows that do not
// all start on 16 bytes.
template <bool VEC>
__device__ __forceinline__ u32x4 load8(const uint16_t *p) {
    if (VEC) return *reinterpret_cast<const u32x4 *>(p);
    u32x4 r;
#pragma unroll
    for (int i = 0; i < 4; ++i) r[i] = (uint32_t)p[2 * i] | ((uint32_t)p[2 * i + 1] << 16);
    return r;
}

template <bool VEC>
__device__ __forceinline__ void store8(uint16_t *p, u32x4 v) {
    if (VEC) {
        *reinterpret_cast<u32x4 *>(p) = v;
        return;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        p[2 * i] = (uint16_t)v[i];
        p[2 * i + 1] = (uint16_t)(v[i] >> 16);
    }
}

// A cache of `pages` pages of `page_size` tokens: the sizes that the kernels
// take, and its bytes.  The page size is a power of two of whole tiles, so that
// a token's page is a shift, and slots fit 31 bits (bytes do not).
inline bool kv4_shape(int kv_heads, int dim, int64_t pages, int page_size, int *shift) {
    if (kv_heads < 1 || kv_heads > 1 << 16 || !(dim == 64 || dim == 128 || dim == 256) ||
        page_size < 32 || page_size > 1 << 16 || (page_size & (page_size - 1)) || pages < 0 ||
        pages > 0x7FFFFFFF / page_size)
        return false;
    *shift = __builtin_ctz((unsigned)page_size);
    return true;
}

inline int64_t kv4_bytes(int kv_heads, int dim, int64_t pages, int page_size) {
    return pages * kv_heads * (page_size / 32) * 34 * dim;
}

}  // namespace ar
