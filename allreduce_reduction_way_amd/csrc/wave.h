// wave.h -- for the operators around a block: sums over the lanes of a wave, bf16
// pairs, and eight elements from any even address.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "device.h"

namespace ar {

// v of the lane that the data-parallel primitive `CTRL` names; lanes without
// one add 0.
template <int CTRL, int ROWS>
__device__ __forceinline__ float dpp_add(float v) {
    const int moved = __builtin_amdgcn_update_dpp(0, __float_as_int(v), CTRL, ROWS, 0xf, false);
    return v + __int_as_float(moved);
}

// Sum of sixteen lanes side by side; every lane of them gets it.  Each step adds
// the lane that turning the sixteen by 8, 4, 2 and 1 brings: the same pairs in
// every lane, so that all have the same bits.
__device__ __forceinline__ float row16_sum(float v) {
    v = dpp_add<0x128, 0xf>(v);
    v = dpp_add<0x124, 0xf>(v);
    v = dpp_add<0x122, 0xf>(v);
    return dpp_add<0x121, 0xf>(v);
}

// Sum over the wave; every lane gets it, by the same pairs.
__device__ __forceinline__ float wave_sum(float v) {
    v = row16_sum(v);
    const auto a = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = __uint_as_float(a[0]) + __uint_as_float(a[1]);
    const auto b = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    return __uint_as_float(b[0]) + __uint_as_float(b[1]);
}

__device__ __forceinline__ uint32_t bf16_pair(float lo, float hi) {
    typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
    bf16x2_t r;
    r[0] = (__bf16)lo;
    r[1] = (__bf16)hi;
    return __builtin_bit_cast(uint32_t, r);
}

// Eight elements of a row.  Rows start on any even address, and memory takes
// 16-byte accesses there.
typedef u32x4 u32x4_any __attribute__((aligned(2)));

template <bool NT>
__device__ __forceinline__ u32x4 load_vec8(const uint16_t *p) {
    const u32x4_any *v = reinterpret_cast<const u32x4_any *>(p);
    return NT ? __builtin_nontemporal_load(v) : *v;
}

// The first n < 8 of them, zeros for the rest.
__device__ __forceinline__ u32x4 load_few(const uint16_t *p, int n) {
    u32x4 r = {0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < 7; ++i)
        if (i < n) r[i / 2] |= (uint32_t)p[i] << (i % 2 * 16);
    return r;
}

__device__ __forceinline__ void widen(u32x4 v, float (&f)[8]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) f[2 * i] = lo_f32(v[i]), f[2 * i + 1] = hi_f32(v[i]);
}

// `bytes` on from an address that is the same in all lanes: scalar registers hold
// that, and a lane its offset.
template <typename T>
__device__ __forceinline__ T *further(T *p, uint32_t bytes) {
    typedef typename std::conditional<std::is_const<T>::value, const char, char>::type Byte;
    return reinterpret_cast<T *>(reinterpret_cast<Byte *>(p) + bytes);
}

// The same value, which the compiler takes for another one: what was made of it
// before is made again where it is used, and takes no registers until then.
__device__ __forceinline__ u32x4 again(u32x4 v) {
    asm volatile("" : "+v"(v));
    return v;
}

// Element c of eight.
__device__ __forceinline__ float at8(u32x4 v, int c) { return c % 2 ? hi_f32(v[c / 2]) : lo_f32(v[c / 2]); }

}  // namespace ar
