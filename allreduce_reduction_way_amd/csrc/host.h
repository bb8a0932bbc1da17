// host.h -- host-side helpers of libar.so: argument checks, buffer-overlap
// checks, per-device properties and a launch wrapper that reports errors as
// return codes.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include <numeric>

#include "ar.h"

namespace ar {

constexpr int kThreads = 256;  // four 64-lane wavefronts per workgroup
constexpr int kMaxDevices = 64;  // per-device host caches hold this many GPUs

inline bool valid_P(int P) { return P >= 2 && P <= AR_MAX_P; }

inline uintptr_t addr(const void *p) { return reinterpret_cast<uintptr_t>(p); }

inline bool aligned_to(const void *p, uintptr_t a) { return (addr(p) & (a - 1)) == 0; }

inline int64_t round_up(int64_t v, int64_t m) { return (v + m - 1) / m * m; }

// A byte range [lo, lo + bytes) of one buffer argument.
struct Span {
    uintptr_t lo;
    uintptr_t bytes;
};

inline Span span_of(const void *p, int64_t elem_begin, int64_t elems, int64_t elem_bytes) {
    return Span{addr(p) + (uintptr_t)(elem_begin * elem_bytes), (uintptr_t)(elems * elem_bytes)};
}

// True when two non-empty spans share a byte.
inline bool overlap(Span a, Span b) {
    return a.bytes != 0 && b.bytes != 0 && a.lo < b.lo + b.bytes && b.lo < a.lo + a.bytes;
}

// True when two spans overlap without being the very same range.
inline bool partial_overlap(Span a, Span b) {
    return overlap(a, b) && !(a.lo == b.lo && a.bytes == b.bytes);
}

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

// Properties of the current device, queried once per device.
struct DeviceInfo {
    int device;
    int cus;  // compute units (256 on MI355X)
};

// Fills `out` for the current device; AR_OK or AR_ELAUNCH.
int current_device(DeviceInfo *out);

// Workgroups of `fn` (kThreads threads, no dynamic LDS) that fit on one CU at
// once, cached per device and kernel.  0 on error.
int blocks_per_cu(const DeviceInfo &dev, const void *fn);

// hipLaunchKernel of a kernel taking one by-value struct argument.
template <typename Args>
int launch(const void *fn, unsigned grid, unsigned block, const Args &a, void *stream) {
    void *args[] = {const_cast<Args *>(&a)};
    hipError_t e = hipLaunchKernel(fn, dim3(grid), dim3(block), args, 0,
                                   static_cast<hipStream_t>(stream));
    return e == hipSuccess ? AR_OK : AR_ELAUNCH;
}

// Two-shot slice rule (see ar_slice_range).
inline int64_t slice_len_unit(int P, int64_t n) { return (n / (128 * (int64_t)P)) * 128; }

}  // namespace ar
