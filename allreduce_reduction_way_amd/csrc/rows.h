// rows.h -- rows of bf16 channels of the attention operators: an array
// (tokens, heads, dim) with the strides of the caller, whose channels are
// contiguous.  Eight channels are one lane's share of a row.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <numeric>

#include "device.h"
#include "host.h"

namespace ar {

// An ar_rows argument with its sizes: `heads` rows of `dim` bf16 for each of
// `tokens` tokens.
struct RowsArg {
    ar_rows r;
    int64_t tokens;
    int heads, dim;

    bool empty() const { return tokens == 0 || heads == 0; }
    // Strides that some array could have: none below zero, none so long that
    // an offset in bytes leaves 62 bits.
    bool valid() const {
        const int64_t most = (int64_t)1 << 40;
        if (empty()) return true;
        return r.p && aligned_to(r.p, 2) && r.token_stride >= 0 && r.token_stride <= most / tokens &&
               r.head_stride >= 0 && r.head_stride <= most / heads;
    }
    int64_t row_elems() const { return (int64_t)(heads - 1) * r.head_stride + dim; }  // of one token
    Span span() const {
        return empty() ? Span{0, 0} : span_of(r.p, 0, (tokens - 1) * r.token_stride + row_elems(), 2);
    }
    // Two rows share an element: a token's heads lie within each other, or
    // tokens do.
    bool self_overlap() const {
        if (empty()) return false;
        const bool heads_apart = heads == 1 || r.head_stride >= dim;
        const bool tokens_apart = tokens == 1 || r.token_stride >= row_elems();
        if (heads_apart && tokens_apart) return false;
        // heads outside of tokens (head after head, each of all tokens)
        return !((tokens == 1 || r.token_stride >= dim) &&
                 (heads == 1 || r.head_stride >= (tokens - 1) * r.token_stride + dim));
    }
    // 16-byte vectors can be used: every row starts on one.
    bool vec() const {
        return empty() || (aligned_to(r.p, 16) && r.token_stride % 8 == 0 && r.head_stride % 8 == 0);
    }
    bool same(const RowsArg &o) const {
        return r.p == o.r.p && tokens == o.tokens && heads == o.heads && dim == o.dim &&
               (tokens <= 1 || r.token_stride == o.r.token_stride) &&
               (heads <= 1 || r.head_stride == o.r.head_stride);
    }
    int64_t head_elems() const { return (tokens - 1) * r.token_stride + dim; }  // of one head
    // The distance that every row's start is a multiple of from the first (0:
    // there is one row).
    int64_t step() const {
        return std::gcd(tokens > 1 ? r.token_stride : 0, heads > 1 ? r.head_stride : 0);
    }
    // Whether pieces of `mine` elements of this array and of `theirs` of the
    // other, each array's at multiples of `period` from its start, lie apart.
    bool beside(const RowsArg &o, int64_t period, int64_t mine, int64_t theirs) const {
        if (period < mine + theirs) return false;
        const int64_t bytes = (int64_t)(addr(o.r.p) - addr(r.p)) % (2 * period);
        const int64_t at = bytes < 0 ? bytes + 2 * period : bytes;
        return at >= 2 * mine && at + 2 * theirs <= 2 * period;
    }
    // Whether the two share an element.  Arrays that lie beside each other in
    // every token (the queries and the keys of one projection's output), in
    // every head, or in a period of all their strides (each head's query, key
    // and value side by side) do not; any other crossing of their spans is taken
    // as sharing.
    bool overlaps(const RowsArg &o) const {
        if (!overlap(span(), o.span())) return false;
        if (r.token_stride == o.r.token_stride && beside(o, r.token_stride, row_elems(), o.row_elems()))
            return false;
        if (r.head_stride == o.r.head_stride && beside(o, r.head_stride, head_elems(), o.head_elems()))
            return false;
        return !beside(o, std::gcd(step(), o.step()), dim, o.dim);
    }
};

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
