// kv4.h -- the tiles of a key-value cache of 4 bits (the layout is described
// in include/ar.h) and the conversions to and from its codes.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "device.h"

namespace ar {

constexpr int kTile = 32;    // tokens of a tile
constexpr int kGroup = 32;   // channels that share a scale
constexpr int kNanScale = 255;
// From this scale on, 2^126, a group's values may be infinities or NaN: codes of
// 4 and more go beyond bf16.  Those that are written end at 252.
constexpr uint32_t kWildScale = 253;

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

template <int D>
struct Kv4 {
    static constexpr int W = D / 16;  // channels of a V block
    static constexpr int G = D / kGroup;
    static constexpr int kV = 16 * D, kKScale = 32 * D, kVScale = 33 * D, kBytes = 34 * D;

    // Bytes within a tile: of the codes that begin at even channel c of token
    // t, and of the scale of its group g.
    static __host__ __device__ __forceinline__ int k_code(int t, int c) { return t * (D / 2) + c / 2; }
    static __host__ __device__ __forceinline__ int v_code(int t, int c) {
        return kV + ((t / 8 * 16 + c / W) * 8 + t % 8) * (W / 2) + c % W / 2;
    }
    static __host__ __device__ __forceinline__ int k_scale(int t, int g) {
        return kKScale + (g * 16 + t / 8 * 4 + t % 4) * 2 + t % 8 / 4;
    }
    static __host__ __device__ __forceinline__ int v_scale(int t, int g) {
        return kVScale + (t / 8 * G + g) * 8 + t % 8;
    }
};

// 2**(byte - 127); infinity for kNanScale, which the conversions below turn
// into NaN.
__device__ __forceinline__ float kv4_scale(uint32_t byte) { return __uint_as_float(byte << 23); }

// The two channels of byte `sel` of eight codes, times the scale (exact).
__device__ __forceinline__ uint32_t kv4_pair(uint32_t codes, float scale, int sel) {
    bf16x2 r;
    switch (sel) {  // constant once loops are unrolled
        case 0: r = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 0); break;
        case 1: r = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 1); break;
        case 2: r = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 2); break;
        default: r = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 3); break;
    }
    return __builtin_bit_cast(uint32_t, r);
}

// Eight channels (four words) as codes, and the scale byte of their group;
// four lanes side by side hold a group.
__device__ __forceinline__ uint32_t kv4_quantise(u32x4 x, uint32_t &byte) {
    uint32_t most = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) most = max(most, max((x[i] << 16) & 0x7FFFFFFFu, x[i] & 0x7FFF0000u));
    most = max(most, (uint32_t)__shfl_xor((int)most, 1));
    most = max(most, (uint32_t)__shfl_xor((int)most, 2));
    most >>= 16;
    // the exponent, one more from 1.75 on (adding 0.25 carries), less two
    const uint32_t e = (most + 0x20u) >> 7;
    byte = min(max(e, 4u) - 2u, 252u);
    const float scale = kv4_scale(byte);
    const uint32_t w[4] = {x[0], x[1], x[2], x[3]};
    uint32_t codes = 0;
    codes = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(codes, __builtin_bit_cast(bf16x2, w[0]), scale, 0);
    codes = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(codes, __builtin_bit_cast(bf16x2, w[1]), scale, 1);
    codes = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(codes, __builtin_bit_cast(bf16x2, w[2]), scale, 2);
    codes = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(codes, __builtin_bit_cast(bf16x2, w[3]), scale, 3);
    if (most >= 0x7F80u) byte = kNanScale, codes = 0;
    return codes;
}

// Eight codes as values.
__device__ __forceinline__ u32x4 kv4_dequantise(uint32_t codes, uint32_t byte) {
    const float scale = kv4_scale(byte);
    u32x4 r;
#pragma unroll
    for (int i = 0; i < 4; ++i) r[i] = byte == kNanScale ? 0x7FC07FC0u : kv4_pair(codes, scale, i);
    return r;
}

}  // namespace ar
