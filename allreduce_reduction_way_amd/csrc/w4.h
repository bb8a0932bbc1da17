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
#include "rows.h"
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

__host__ __device__ inline W4Shape w4_shape_of(int n_out, int n_in) {
    const int chunks = (n_in + kW4Chunk - 1) / kW4Chunk;
    return W4Shape{n_out, n_in, chunks, (n_out + 15) / 16, (int64_t)chunks * kW4Codes + (chunks + 3) / 4 * kW4Scales};
}

inline bool w4_shape(int64_t n_out, int64_t n_in, W4Shape *s) {
    if (n_out < 1 || n_out > kW4MaxOut || n_in < 32 || n_in > kW4MaxIn || n_in % 32) return false;
    *s = w4_shape_of((int)n_out, (int)n_in);
    return true;
}

// A lane's codes and scale byte of chunk c of a tile.  (The tile and the chunk are
// the same in all lanes: scalar registers hold the address, and a lane its offset.)
__device__ __forceinline__ u32x4 w4_codes(const uint8_t *tile, int c, int lane) {
    return *reinterpret_cast<const u32x4 *>(tile + c * kW4Codes + (uint32_t)lane * 16u);
}
__device__ __forceinline__ uint32_t w4_scale(const uint8_t *tile, int chunks, int c, int lane) {
    return (tile + chunks * kW4Codes + c / 4 * kW4Scales + c % 4)[(uint32_t)lane * 4u];
}

// Those of chunks c and c + 1, c even, in two bytes.
__device__ __forceinline__ uint32_t w4_two_scales(const uint8_t *tile, int chunks, int c, int lane) {
    return *reinterpret_cast<const uint16_t *>(tile + chunks * kW4Codes + c / 4 * kW4Scales + c % 4 + (uint32_t)lane * 4u);
}

// The weights' operand of step s: eight codes of a lane as bf16, exactly.
__device__ __forceinline__ bf16x8 w4_operand(u32x4 codes, float scale, int s) {
    u32x4 v;
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = kv4_pair(codes[s], scale, e);
    return __builtin_bit_cast(bf16x8, v);
}

// The other operand of a chunk's four steps comes from rows of n elements, sixteen
// of them as columns.  A compute unit takes 64 bytes in a cycle where lanes side by
// side ask for them, and 16 where each asks for another row, as the steps need
// them.  So eight lanes ask for 128 bytes of a row, a line of the cache, and a wave
// turns what it gets through a piece of LDS of its own: x[i] is elements
// 64 (i / 2) + 8 (l % 8) .. + 7 of row 8 (i % 2) + l / 8 until a Stage has made it
// 32 a + 8 i .. + 7 of row r.  (Asking as the steps need them, 16 tokens times
// 8192 x 28672 took 59 us, and 29.5 with this; with four lanes to a row 64 tokens took
// 51.3, and 50.1 with this.)  Past the row the stage leaves zeros: codes are
// zeros there too, but infinity times zero is none.
//
// The loads stand behind no branch, where the compiler would wait for each: past a
// row's end they take its last elements again.
struct Inputs {
    const uint16_t *row[2];

    Inputs() = default;
    // Of tokens [first, first + 16) of x; past `last` they are that one's.
    __device__ __forceinline__ Inputs(const Rows &x, int64_t first, int64_t last, int lane)
        : row{x.p + min(first + lane / 8, last) * x.ts, x.p + min(first + 8 + lane / 8, last) * x.ts} {}
    __device__ __forceinline__ void load(u32x4 (&x)[4], int chunk, int lane, int n) const {
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = load_vec8<false>(row[i % 2] + min(chunk * kW4Chunk + i / 2 * 64 + lane % 8 * 8, n - 8));
    }
};

// The same for few columns, of which lane (r, q) has `row`, from element 32 q on:
// loaded as the steps need them by the lanes that have a column, so that nothing is
// turned.  Four columns take a quarter of the time of sixteen.  What the other lanes
// have is left open: it stays in their columns.
__device__ __forceinline__ void load_few_inputs(u32x4 (&x)[4], const uint16_t *row, int step, bool mine) {
#pragma unroll
    for (int s = 0; s < 4; ++s) asm("" : "=v"(x[s]));
    if (mine) {
#pragma unroll
        for (int s = 0; s < 4; ++s) x[s] = load_vec8<false>(row + s * step);
    }
}

// A wave's piece of LDS: 16 rows of 256 bytes, 320 apart, with the 16-byte blocks of
// every 64 bytes in another order from four rows to the next.  Eight lanes at a time
// write 128 bytes of a row, and read a block of eight rows: neither meets in a bank.
constexpr int kStageRow = 320 / 16, kStage = 16 * kStageRow;  // in 16 bytes

struct Stage {
    u32x4 *to[2];
    const u32x4 *from[4];
    int lane;

    __device__ __forceinline__ Stage(u32x4 *p, int lane) : lane(lane) {
        const int r = lane % 16;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int row = i * 8 + lane / 8;
            to[i] = p + row * kStageRow + lane % 8 / 4 * 4 + (lane % 4 ^ row / 4);
        }
#pragma unroll
        for (int s = 0; s < 4; ++s) from[s] = p + r * kStageRow + lane / 16 * 4 + (s ^ r / 4);
    }
    // Inputs of chunk `chunk`, of rows of n, into the steps' order.
    __device__ __forceinline__ void turn(u32x4 (&x)[4], int chunk, int n) const {
        if ((chunk + 1) * kW4Chunk > n) {  // the same in all lanes
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (chunk * kW4Chunk + i / 2 * 64 + lane % 8 * 8 >= n) x[i] = u32x4{0, 0, 0, 0};
        }
        // one wave's accesses to LDS stay in order; the fences keep the compiler's
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
#pragma unroll
        for (int i = 0; i < 4; ++i) to[i % 2][i / 2 * 8] = x[i];
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
#pragma unroll
        for (int s = 0; s < 4; ++s) x[s] = *from[s];
    }
};

__device__ __forceinline__ f32x4 w4_product(bf16x8 w, u32x4 x, f32x4 acc) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(w, __builtin_bit_cast(bf16x8, x), acc, 0, 0, 0);
}

}  // namespace ar
