// w4.h -- weights of 4 bits (the layout is described in include/ar.h): sizes,
// and the operands of the matrix instructions made of them.
//
// The layout is the order in which v_mfma_f32_16x16x32_bf16 takes its operands.
// A chunk is 16 outputs x 128 inputs: with r = lane % 16 and a = lane / 16, lane
// (r, a) holds output r's inputs 32 a .. 32 a + 31, which share a scale, in one
// 16-byte load; step s of four takes the eight of them from 8 s on, so a product's
// 32 inputs are 32 a + 8 s + 0..7 for a = 0..3, and the other operand's lane takes
// the same of its row.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "kv4.h"
#include "wave.h"

namespace ar {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

constexpr int kW4Chunk = 128;       // inputs of a chunk
constexpr int kW4Codes = 1024;      // its bytes of codes
constexpr int kW4Scales = 256;      // bytes of the scales of four chunks
constexpr int64_t kW4MaxIn = 1 << 20, kW4MaxOut = 1 << 24;

// 16 outputs of a matrix are a tile: the codes of its chunks, then the scales.
struct W4Shape {
    int n_out, n_in, chunks, tiles;
    int64_t tile_bytes;

    __host__ __device__ int64_t bytes() const { return tiles * tile_bytes; }
};

inline bool w4_shape(int64_t n_out, int64_t n_in, W4Shape *s) {
    if (n_out < 1 || n_out > kW4MaxOut || n_in < 32 || n_in > kW4MaxIn || n_in % 32) return false;
    s->n_out = (int)n_out, s->n_in = (int)n_in;
    s->chunks = (int)((n_in + kW4Chunk - 1) / kW4Chunk), s->tiles = (int)((n_out + 15) / 16);
    s->tile_bytes = (int64_t)s->chunks * kW4Codes + (s->chunks + 3) / 4 * kW4Scales;
    return true;
}

// Where a lane's codes and scale of chunk c lie in a tile.
__device__ __forceinline__ int w4_code_at(int c, int lane) { return c * kW4Codes + lane * 16; }
__device__ __forceinline__ int w4_scale_at(int chunks, int c, int lane) {
    return chunks * kW4Codes + c / 4 * kW4Scales + lane * 4 + c % 4;
}

// The weights' operand of step s: eight codes of a lane as bf16, exactly.
__device__ __forceinline__ bf16x8 w4_operand(u32x4 codes, float scale, int s) {
    u32x4 v;
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = kv4_pair(codes[s], scale, e);
    return __builtin_bit_cast(bf16x8, v);
}

// The 32 elements from k on of a row of n, the other operand of four steps; zeros
// past the row, where codes are zeros too, but what memory holds need not be a
// number.
__device__ __forceinline__ void load_inputs(u32x4 (&x)[4], const uint16_t *row, int k, int n) {
#pragma unroll
    for (int s = 0; s < 4; ++s) x[s] = u32x4{0, 0, 0, 0};
    if (k < n) {
#pragma unroll
        for (int s = 0; s < 4; ++s) x[s] = load_vec8<false>(row + k + 8 * s);
    }
}

__device__ __forceinline__ f32x4 w4_product(bf16x8 w, u32x4 x, f32x4 acc) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(w, __builtin_bit_cast(bf16x8, x), acc, 0, 0, 0);
}

}  // namespace ar
