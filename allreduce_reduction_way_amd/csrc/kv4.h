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

}  // namespace ar
