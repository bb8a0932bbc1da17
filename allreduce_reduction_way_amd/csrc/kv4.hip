// kv4.hip -- keys and values quantised into a paged cache of 4 bits as they
// are written, and read back.
//
// A group of 32 channels of a token shares the scale 2**(byte - 127), the
// least power of two (from 2**-125 on) that leaves the group's largest
// magnitude below 7: 7 is where rounding would leave the largest code, 6, by
// more than the step there.  Each channel is then rounded to the nearest of
// 0, 0.5, 1, 1.5, 2, 3, 4, 6 and a sign, ties to the even code, which is what
// the conversion instruction does.
//
// Both kernels are bound by memory: 2 bytes of bf16 against 17/32 of codes and
// scales for each channel, and a few operations.  A row lies in D/8 lanes, 16
// bytes each; a group's largest is an exchange between four lanes.  16384 tokens
// of eight heads of 128, 170 MB, are written and read back in 32.7 us, 5.2 TB/s;
// 440 of one head in 7.0, which is what two launches cost their caller.
#include "host.h"
#include "kv4.h"
#include "rows.h"

namespace ar {
namespace {

// Above this many bytes of rows, they are read and written past the caches:
// 67 MB of them took 19.3 and 16.3 us to write and read back, and take 17.4 and 15.0.
constexpr int64_t kStreamBytes = (int64_t)32 << 20;

struct Kv4Args {
    Rows k, v;
    const int64_t *slots;
    uint8_t *cache;
    int64_t tokens;
    uint32_t capacity;  // slots of the cache
    int heads, page_shift;
};

template <bool VEC, bool NT>
__device__ __forceinline__ u32x4 load_row(const uint16_t *p) {
    return NT ? __builtin_nontemporal_load(reinterpret_cast<const u32x4 *>(p)) : load8<VEC>(p);
}

template <bool VEC, bool NT>
__device__ __forceinline__ void store_row(const uint16_t *to, u32x4 v) {
    uint16_t *p = const_cast<uint16_t *>(to);
    if (NT) __builtin_nontemporal_store(v, reinterpret_cast<u32x4 *>(p));
    else store8<VEC>(p, v);
}

// The head and the first of the T tokens that a wave works on: neighbours work
// on one head's tokens, whose bytes lie side by side in the cache.
template <int T>
__device__ __forceinline__ bool locate(const Kv4Args &a, int &head, int64_t &first) {
    const int item = __builtin_amdgcn_readfirstlane(blockIdx.x * (kThreads / 64) + threadIdx.x / 64);
    const int groups = (int)((a.tokens + T - 1) / T);
    head = item / groups;
    first = (int64_t)(item - head * groups) * T;
    return head < a.heads;
}

// The tile and the token within it of a slot.
template <int D>
__device__ __forceinline__ uint8_t *tile_of(const Kv4Args &a, uint32_t slot, int head) {
    const uint32_t page = slot >> a.page_shift, in = slot & ((1u << a.page_shift) - 1);
    const int64_t tile = (((int64_t)page * a.heads + head) << (a.page_shift - 5)) + in / kTile;
    return a.cache + tile * Kv4<D>::kBytes;
}

// Stores the codes of eight channels from c on into a V block, or two.
template <int D>
__device__ __forceinline__ void store_v(uint8_t *tile, int t, int c, uint32_t codes) {
    if (Kv4<D>::W >= 8) {
        *reinterpret_cast<uint32_t *>(tile + Kv4<D>::v_code(t, c)) = codes;
    } else {
        *reinterpret_cast<uint16_t *>(tile + Kv4<D>::v_code(t, c)) = (uint16_t)codes;
        *reinterpret_cast<uint16_t *>(tile + Kv4<D>::v_code(t, c + 4)) = (uint16_t)(codes >> 16);
    }
}

template <int D>
__device__ __forceinline__ uint32_t load_v(const uint8_t *tile, int t, int c) {
    if (Kv4<D>::W >= 8) return *reinterpret_cast<const uint32_t *>(tile + Kv4<D>::v_code(t, c));
    return (uint32_t)*reinterpret_cast<const uint16_t *>(tile + Kv4<D>::v_code(t, c)) |
           ((uint32_t)*reinterpret_cast<const uint16_t *>(tile + Kv4<D>::v_code(t, c + 4)) << 16);
}

template <int D, bool VEC, int T, bool NT>
__global__ __launch_bounds__(kThreads) void k_kv4_write(Kv4Args a) {
    constexpr int kLanes = D / 8, kRows = 64 / kLanes, kSteps = (T + kRows - 1) / kRows;
    const int lane = threadIdx.x % 64, c = lane % kLanes * 8;
    int head;
    int64_t first;
    if (!locate<T>(a, head, first)) return;
    u32x4 k[kSteps], v[kSteps];
    int64_t slot[kSteps];
#pragma unroll
    for (int u = 0; u < kSteps; ++u) {
        const int64_t t = first + u * kRows + lane / kLanes;
        k[u] = v[u] = u32x4{0, 0, 0, 0};
        slot[u] = -1;
        if (t < a.tokens && u * kRows + lane / kLanes < T) {
            slot[u] = a.slots[t];
            k[u] = load_row<VEC, NT>(a.k.p + t * a.k.ts + head * a.k.hs + c);
            v[u] = load_row<VEC, NT>(a.v.p + t * a.v.ts + head * a.v.hs + c);
        }
    }
#pragma unroll
    for (int u = 0; u < kSteps; ++u) {
        uint32_t kb, vb;
        const uint32_t kc = kv4_quantise(k[u], kb), vc = kv4_quantise(v[u], vb);
        if (slot[u] < 0 || slot[u] >= (int64_t)a.capacity) continue;
        uint8_t *tile = tile_of<D>(a, (uint32_t)slot[u], head);
        const int t = (int)(slot[u] % kTile);
        *reinterpret_cast<uint32_t *>(tile + Kv4<D>::k_code(t, c)) = kc;
        store_v<D>(tile, t, c, vc);
        if (c % kGroup == 0) {
            tile[Kv4<D>::k_scale(t, c / kGroup)] = (uint8_t)kb;
            tile[Kv4<D>::v_scale(t, c / kGroup)] = (uint8_t)vb;
        }
    }
}

template <int D, bool VEC, int T, bool NT>
__global__ __launch_bounds__(kThreads) void k_kv4_read(Kv4Args a) {
    constexpr int kLanes = D / 8, kRows = 64 / kLanes, kSteps = (T + kRows - 1) / kRows;
    const int lane = threadIdx.x % 64, c = lane % kLanes * 8;
    int head;
    int64_t first;
    if (!locate<T>(a, head, first)) return;
    uint32_t kc[kSteps], vc[kSteps], kb[kSteps], vb[kSteps];
#pragma unroll
    for (int u = 0; u < kSteps; ++u) {
        const int64_t t = first + u * kRows + lane / kLanes;
        kc[u] = vc[u] = kb[u] = vb[u] = 0;
        if (t < a.tokens && u * kRows + lane / kLanes < T) {
            const int64_t slot = a.slots[t];
            if (slot >= 0 && slot < (int64_t)a.capacity) {
                const uint8_t *tile = tile_of<D>(a, (uint32_t)slot, head);
                const int i = (int)(slot % kTile);
                kc[u] = *reinterpret_cast<const uint32_t *>(tile + Kv4<D>::k_code(i, c));
                vc[u] = load_v<D>(tile, i, c);
                kb[u] = tile[Kv4<D>::k_scale(i, c / kGroup)];
                vb[u] = tile[Kv4<D>::v_scale(i, c / kGroup)];
            }
        }
    }
#pragma unroll
    for (int u = 0; u < kSteps; ++u) {
        const int64_t t = first + u * kRows + lane / kLanes;
        if (t < a.tokens && u * kRows + lane / kLanes < T) {
            store_row<VEC, NT>(a.k.p + t * a.k.ts + head * a.k.hs + c, kv4_dequantise(kc[u], kb[u]));
            store_row<VEC, NT>(a.v.p + t * a.v.ts + head * a.v.hs + c, kv4_dequantise(vc[u], vb[u]));
        }
    }
}

template <bool READ, int D, bool VEC, int T, bool NT>
const void *kernel() {
    return READ ? reinterpret_cast<const void *>(&k_kv4_read<D, VEC, T, NT>)
                : reinterpret_cast<const void *>(&k_kv4_write<D, VEC, T, NT>);
}

template <bool READ, int D>
const void *pick_dim(bool vec, bool few, bool stream) {
    if (few) return vec ? kernel<READ, D, true, 4, false>() : kernel<READ, D, false, 4, false>();
    if (!vec) return kernel<READ, D, false, 8, false>();
    return stream ? kernel<READ, D, true, 8, true>() : kernel<READ, D, true, 8, false>();
}

template <bool READ>
const void *pick(int dim, bool vec, bool few, bool stream) {
    return dim == 64    ? pick_dim<READ, 64>(vec, few, stream)
           : dim == 128 ? pick_dim<READ, 128>(vec, few, stream)
                        : pick_dim<READ, 256>(vec, few, stream);
}

template <bool READ>
int kv4_call(ar_rows k, ar_rows v, const void *slots, void *cache, int64_t tokens, int kv_heads,
             int dim, int64_t pages, int page_size, void *stream) {
    int shift = 0;
    if (!kv4_shape(kv_heads, dim, pages, page_size, &shift) || tokens < 0 ||
        tokens > (int64_t)1 << 28)
        return AR_EINVAL;
    if (tokens == 0) return AR_OK;
    const RowsArg rk{k, tokens, kv_heads, dim}, rv{v, tokens, kv_heads, dim};
    if (!rk.valid() || !rv.valid() || !slots || !aligned_to(slots, 8) ||
        (pages > 0 && (!cache || !aligned_to(cache, 16))))
        return AR_EINVAL;
    if (READ && (rk.self_overlap() || rv.self_overlap())) return AR_EINVAL;
    const Span sc{addr(cache), (uintptr_t)kv4_bytes(kv_heads, dim, pages, page_size)};
    const Span ss{addr(slots), (uintptr_t)(8 * tokens)};
    if (overlap(rk.span(), sc) || overlap(rv.span(), sc) || overlap(ss, sc)) return AR_EALIAS;
    if (READ && (rk.overlaps(rv) || overlap(rk.span(), ss) || overlap(rv.span(), ss))) return AR_EALIAS;
    Kv4Args a = {};
    a.k = rows(rk), a.v = rows(rv);
    a.slots = static_cast<const int64_t *>(slots);
    a.cache = static_cast<uint8_t *>(cache);
    a.tokens = tokens, a.capacity = (uint32_t)(pages * page_size), a.heads = kv_heads, a.page_shift = shift;
    // eight tokens to a wave, four where that leaves waves out: 440 tokens take
    // 3.0 us to read back, and 3.6
    const bool few = (tokens + 7) / 8 * kv_heads < 2048;
    const int64_t items = (tokens + (few ? 3 : 7)) / (few ? 4 : 8) * kv_heads;
    const int64_t blocks = (items + kThreads / 64 - 1) / (kThreads / 64);
    if (blocks > 0x7FFFFFFF / kThreads) return AR_EINVAL;
    const bool stream_rows = 4 * tokens * kv_heads * dim > kStreamBytes;
    return launch(pick<READ>(dim, rk.vec() && rv.vec(), few, stream_rows), (unsigned)blocks, kThreads, a, stream);
}

}  // namespace
}  // namespace ar

using namespace ar;

extern "C" {

int64_t ar_kv4_cache_bytes(int64_t pages, int kv_heads, int dim, int page_size) {
    int shift = 0;
    if (!kv4_shape(kv_heads, dim, pages, page_size, &shift)) return AR_EINVAL;
    return kv4_bytes(kv_heads, dim, pages, page_size);
}

int ar_kv4_write(ar_rows k, ar_rows v, const void *slots, void *cache, int64_t tokens, int kv_heads,
                 int dim, int64_t pages, int page_size, void *stream) {
    return kv4_call<false>(k, v, slots, cache, tokens, kv_heads, dim, pages, page_size, stream);
}

int ar_kv4_read(const void *cache, const void *slots, ar_rows k_out, ar_rows v_out, int64_t tokens,
                int kv_heads, int dim, int64_t pages, int page_size, void *stream) {
    return kv4_call<true>(k_out, v_out, slots, const_cast<void *>(cache), tokens, kv_heads, dim, pages,
                          page_size, stream);
}

}  // extern "C"
