// w4.hip -- weights of 4 bits: packed from bf16 and unpacked, and a few tokens'
// products with them.
//
// out = x W^T with W's codes turned into bf16, which is exact, and products added
// up in binary32 by the matrix unit.  For up to some 64 tokens it is bound by the
// weights' bytes, 17/32 of one each, or by latency where there are few of those.
// Eight tokens x 8192 x 28672 take 25.7 us (4.9 TB/s); with more tokens the inputs' way
// into each compute unit weighs more: 55 x 5152 x 10001 take 14.6 us (2.0 TB/s).
#include "host.h"
#include "rows.h"
#include "w4.h"

namespace ar {
namespace {

struct PackArgs {
    W4Shape s;
    const uint16_t *w;
    int64_t row_stride;
    uint8_t *packed;
};

// A lane takes eight inputs of an output, four lanes side by side a group.  Every
// byte is written: what lies past the matrix becomes zeros.  28672 x 8192 take 135 us (4.4
// TB/s; its floor is 117), 8192 x 28672 160, 5120 x 10240 35, 5120 x 1024 4.9: a wave's
// stores are pieces of 16 bytes, 256 apart.
__global__ __launch_bounds__(kThreads) void k_w4_pack(PackArgs a) {
    const int octets = (a.s.chunks + 3) / 4 * 4 * kW4Chunk / 8;  // of an output, those of the last scales' chunks with them
    const int64_t item = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    const int64_t n = item / octets;
    const int k = (int)(item % octets) * 8;
    if (n >= (int64_t)a.s.tiles * 16) return;
    u32x4 x = {0, 0, 0, 0};
    if (n < a.s.n_out && k < a.s.n_in) x = load_vec8<false>(a.w + n * a.row_stride + k);
    uint32_t byte;
    const uint32_t codes = kv4_quantise(x, byte);
    uint8_t *tile = a.packed + n / 16 * a.s.tile_bytes;
    const int c = k / kW4Chunk, lane = k % kW4Chunk / 32 * 16 + (int)(n % 16);
    if (c < a.s.chunks) *reinterpret_cast<uint32_t *>(tile + c * kW4Codes + lane * 16 + k % 32 / 2) = codes;
    if (k % 32 == 0) tile[a.s.chunks * kW4Codes + c / 4 * kW4Scales + lane * 4 + c % 4] = (uint8_t)byte;
}

struct UnpackArgs {
    W4Shape s;
    const uint8_t *packed;
    uint16_t *w;
    int64_t row_stride;
};

// (28672 x 8192 take 143 us, 4.2 TB/s, 5120 x 10240 45.)
__global__ __launch_bounds__(kThreads) void k_w4_unpack(UnpackArgs a) {
    const int octets = a.s.n_in / 8;
    const int64_t item = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    const int64_t n = item / octets;
    const int k = (int)(item % octets) * 8;
    if (n >= a.s.n_out) return;
    const uint8_t *tile = a.packed + n / 16 * a.s.tile_bytes;
    const int c = k / kW4Chunk, lane = k % kW4Chunk / 32 * 16 + (int)(n % 16);
    const uint32_t codes = *reinterpret_cast<const uint32_t *>(tile + c * kW4Codes + lane * 16 + k % 32 / 2);
    *reinterpret_cast<u32x4_any *>(a.w + n * a.row_stride + k) = kv4_dequantise(codes, w4_scale(tile, a.s.chunks, c, lane));
}

constexpr int kCus = 256;

// A call's arguments in 56 bytes: with more than 64 a launch costs its caller 3.3 us and
// more, no less than small calls take (one token x 1024 x 5120 3.3 us so, 3.8 with 88
// bytes).
struct LinearArgs {
    const uint8_t *packed;
    const uint16_t *x;
    uint16_t *out;
    int64_t x_stride, out_stride;
    int n_out, n_in, tokens;
};

// The same as the kernels take them.
struct Linear {
    W4Shape s;
    const uint8_t *packed;
    Rows x, out;
    int64_t tokens;

    __device__ __forceinline__ explicit Linear(const LinearArgs &a)
        : s(w4_shape_of(a.n_out, a.n_in)), packed(a.packed), x{a.x, a.x_stride, 0}, out{a.out, a.out_stride, 0}, tokens(a.tokens) {}
};

constexpr int kJoin = 8;  // tiles of sums in LDS at once

// The waves' sums of RT tiles of outputs for C times 16 tokens, joined through LDS
// some tiles at a time, and stored.
template <int RT, int C>
__device__ __forceinline__ void join_waves(const Linear &a, const f32x4 (&acc)[RT][C], f32x4 *part, int tile0, int64_t token0) {
    const int lane = threadIdx.x % 64, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64), waves = blockDim.x / 64;
    constexpr int kTogether = RT * C < kJoin ? RT * C : kJoin;
#pragma unroll
    for (int first = 0; first < RT * C; first += kTogether) {
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kTogether; ++i)
            if (first + i < RT * C) part[(wave * kTogether + i) * 64 + lane] = acc[(first + i) / C][(first + i) % C];
        __syncthreads();
        for (int item = threadIdx.x; item < kTogether * 64; item += blockDim.x) {
            f32x4 v = part[item];
            for (int w = 1; w < waves; ++w) v += part[w * kTogether * 64 + item];
            const int i = first + item / 64, at = item % 64;
            if (i >= RT * C) break;
            const int64_t n = (int64_t)(tile0 + i / C) * 16 + at / 16 * 4, token = token0 + i % C * 16 + at % 16;
            if (token >= a.tokens) continue;
            uint16_t *to = const_cast<uint16_t *>(a.out.p) + token * a.out.ts + n;
            const uint32_t lo = bf16_pair(v[0], v[1]), hi = bf16_pair(v[2], v[3]);
            if (n + 4 <= a.s.n_out) {
                typedef uint32_t u32x2_any __attribute__((ext_vector_type(2), aligned(2)));
                *reinterpret_cast<u32x2_any *>(to) = u32x2_any{lo, hi};
            } else {
                if (n < a.s.n_out) to[0] = (uint16_t)lo;
                if (n + 1 < a.s.n_out) to[1] = (uint16_t)(lo >> 16);
                if (n + 2 < a.s.n_out) to[2] = (uint16_t)hi;
            }
        }
    }
}

// One or two tokens, and up to four with one tile to a workgroup: all inputs are held in
// LDS, so that what a wave loads for a chunk is its codes and a byte of scales to a
// lane, of two chunks side by side at once.  Sixteen tokens' worth of loads for one token
// are what bounds k_w4_linear there: one token x 14336 x 4096 takes 8.5 us, 11.7 by that,
// x 7168 x 7168 7.7 and 8.5, x 5120 x 20480 12.6 and 14.2, two tokens 9.3 and 11.6, 8.1
// and 8.4, 13.0 and 14.2, four 11.0 and 11.6, but 8.9 and 8.4, 14.7 and 14.3.  With four
// tiles and one workgroup to a compute unit k_w4_linear_few takes less: one token x 4096 x
// 14336 8.6 us, and 9.1 this.
constexpr int kHeldPad = 8;            // elements between tokens
constexpr int kHeldBytes = 150 << 10;  // of LDS, at most

int held_row(const W4Shape &s) { return s.chunks * kW4Chunk + kHeldPad; }

template <int RT>
__global__ __launch_bounds__(RT == 1 ? 1024 : 512) void k_w4_linear_held(LinearArgs args) {
    const Linear a(args);
    extern __shared__ f32x4 part[];  // the inputs of each token, and after that [waves][RT][64]
    uint16_t *held = reinterpret_cast<uint16_t *>(part);
    const int lane = threadIdx.x % 64, r = lane % 16, q = lane / 16;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64), waves = blockDim.x / 64;
    const int tile0 = blockIdx.x * RT;
    const uint8_t *tile[RT];
#pragma unroll
    for (int t = 0; t < RT; ++t) tile[t] = a.packed + min(tile0 + t, a.s.tiles - 1) * a.s.tile_bytes;
    const int last = a.s.chunks - 1, vecs = a.s.chunks * kW4Chunk / 8, row = a.s.chunks * kW4Chunk + kHeldPad;
    u32x4 codes[2][RT];
    uint32_t bytes[RT];
    const auto load = [&](int chunk) {
        const int c = min(chunk, last & ~1);  // past the end: again what is there
#pragma unroll
        for (int t = 0; t < RT; ++t) {
            codes[0][t] = w4_codes(tile[t], c, lane);
            codes[1][t] = w4_codes(tile[t], min(c + 1, last), lane);
            bytes[t] = w4_two_scales(tile[t], a.s.chunks, c, lane);
        }
    };
    load(2 * wave);
    for (int i = threadIdx.x; i < (int)a.tokens * vecs; i += blockDim.x) {
        const int t = i / vecs, k = (i - t * vecs) * 8;
        u32x4 v = {0, 0, 0, 0};
        if (k < a.s.n_in) v = load_vec8<false>(a.x.p + t * a.x.ts + k);
        *reinterpret_cast<u32x4 *>(held + t * row + k) = v;
    }
    __syncthreads();
    // a column past the tokens is not stored; it takes the last token's row
    const u32x4 *x = reinterpret_cast<const u32x4 *>(held + min(r, (int)a.tokens - 1) * row + q * 32);
    f32x4 acc[RT][1];
#pragma unroll
    for (int t = 0; t < RT; ++t) acc[t][0] = f32x4{0, 0, 0, 0};
    for (int c = 2 * wave; c <= last; c += 2 * waves) {
        bf16x8 w[2][RT][4];
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
            for (int t = 0; t < RT; ++t)
#pragma unroll
                for (int s = 0; s < 4; ++s) w[u][t][s] = w4_operand(codes[u][t], kv4_scale(bytes[t] >> 8 * u & 255), s);
        load(c + 2 * waves);
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            if (c + u > last) break;
#pragma unroll
            for (int s = 0; s < 4; ++s) {
                const u32x4 v = x[(c + u) * (kW4Chunk / 8) + s];
#pragma unroll
                for (int t = 0; t < RT; ++t) acc[t][0] = w4_product(w[u][t][s], v, acc[t][0]);
            }
        }
    }
    join_waves<RT, 1>(a, acc, part, tile0, 0);
}

// Up to eight tokens, and four tiles to a workgroup: the lanes that have a token load
// its inputs as the steps take them, with no turn through LDS, and with fewer
// registers.  (One token x 4096 x 14336 takes 8.6 us, 9.3 by k_w4_linear; eight x
// 8192 x 14336 15.1 and 15.4.  With fewer tiles the loads, which take 16 bytes of each
// row, weigh more: eight x 8192 x 5120 would take 9.2, and 8.1 there.)
__global__ __launch_bounds__(512) void k_w4_linear_few(LinearArgs args) {
    const Linear a(args);
    constexpr int RT = 4;
    extern __shared__ f32x4 part[];  // [waves][RT][64]
    const int lane = threadIdx.x % 64, r = lane % 16, q = lane / 16;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64), waves = blockDim.x / 64;
    const int tile0 = blockIdx.x * RT;
    const uint8_t *tile[RT];
#pragma unroll
    for (int t = 0; t < RT; ++t) tile[t] = a.packed + min(tile0 + t, a.s.tiles - 1) * a.s.tile_bytes;
    const bool mine = r < a.tokens;
    const uint16_t *row = a.x.p + (mine ? r : 0) * a.x.ts + q * 32;
    f32x4 acc[RT][1];
#pragma unroll
    for (int t = 0; t < RT; ++t) acc[t][0] = f32x4{0, 0, 0, 0};
    for (int c = wave; c < a.s.chunks; c += waves) {
        u32x4 codes[RT], x[4];
        uint32_t byte[RT];
#pragma unroll
        for (int t = 0; t < RT; ++t) {
            codes[t] = w4_codes(tile[t], c, lane);
            byte[t] = w4_scale(tile[t], a.s.chunks, c, lane);
        }
        load_few_inputs(x, row + min(c * kW4Chunk, a.s.n_in - 32 - q * 32), 8, mine);  // past the row: inside it
        if ((c + 1) * kW4Chunk > a.s.n_in && c * kW4Chunk + q * 32 >= a.s.n_in) {
#pragma unroll
            for (int s = 0; s < 4; ++s) x[s] = u32x4{0, 0, 0, 0};
        }
#pragma unroll
        for (int s = 0; s < 4; ++s)
#pragma unroll
            for (int t = 0; t < RT; ++t) acc[t][0] = w4_product(w4_operand(codes[t], kv4_scale(byte[t]), s), x[s], acc[t][0]);
    }
    join_waves<RT, 1>(a, acc, part, tile0, 0);
}

// A workgroup computes RT tiles of outputs for C times 16 tokens.  Its waves take
// the chunks in turn, each with sums of its own, and join them through LDS.  A
// chunk's weights are turned into bf16 once, for all columns.  While it works on 16
// columns a wave has the next 16's inputs on their way, and from a chunk's first
// columns on the next chunk's codes.  What bounds it is the inputs' way from L2 into each
// compute unit: for 64 tokens x 6144 that alone takes 209 workgroups 9.6 us, with the turn
// through LDS 10.8, and 10.9 with loads straight into LDS.  Other waves or depths gain
// nothing: 64 tokens x 7168 x 7168 take 28.7, 29.8 and 30.7 us with eight, twelve and
// sixteen waves and RT = 1, and 20.5 with a whole chunk's inputs ahead, 18.9 so, RT = 2.
template <int RT, int C>
__global__ __launch_bounds__(512) void k_w4_linear(LinearArgs args) {
    const Linear a(args);
    extern __shared__ f32x4 part[];  // [waves][min(RT C, kJoin)][64], and before that a stage of each wave
    const int lane = threadIdx.x % 64;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64), waves = blockDim.x / 64;
    const int tile0 = blockIdx.x * RT;
    const int64_t token0 = (int64_t)blockIdx.y * (16 * C);
    const uint8_t *tile[RT];
    Inputs in[C];
#pragma unroll
    for (int t = 0; t < RT; ++t) tile[t] = a.packed + min(tile0 + t, a.s.tiles - 1) * a.s.tile_bytes;
    // a column past the tokens is not stored; it takes the last token's row
#pragma unroll
    for (int c = 0; c < C; ++c) in[c] = Inputs(a.x, token0 + c * 16, a.tokens - 1, lane);
    const Stage stage(reinterpret_cast<u32x4 *>(part) + wave * kStage, lane);
    f32x4 acc[RT][C];
#pragma unroll
    for (int t = 0; t < RT; ++t)
#pragma unroll
        for (int c = 0; c < C; ++c) acc[t][c] = f32x4{0, 0, 0, 0};
    u32x4 codes[RT], x[2][4];
    uint32_t byte[RT];
    const auto load_codes = [&](int c) {
#pragma unroll
        for (int t = 0; t < RT; ++t) {
            codes[t] = w4_codes(tile[t], c, lane);
            byte[t] = w4_scale(tile[t], a.s.chunks, c, lane);
        }
    };
    const int last = a.s.chunks - 1;
    if (wave <= last) {
        load_codes(wave);
        in[0].load(x[0], wave, lane, a.s.n_in);
    }
    for (int first = wave; first <= last; first += 2 * waves) {
#pragma unroll
        for (int b = 0; b < 2; ++b) {
            const int c = first + b * waves, next = min(c + waves, last);  // past the end: again what is there
            if (c > last) break;
            bf16x8 w[RT][4];
#pragma unroll
            for (int t = 0; t < RT; ++t)
#pragma unroll
                for (int s = 0; s < 4; ++s) w[t][s] = w4_operand(codes[t], kv4_scale(byte[t]), s);
#pragma unroll
            for (int i = 0; i < C; ++i) {
                u32x4(&now)[4] = x[(b * C + i) & 1];
                in[(i + 1) % C].load(x[(b * C + i + 1) & 1], i + 1 < C ? c : next, lane, a.s.n_in);
                if (i == 0) load_codes(next);
                stage.turn(now, c, a.s.n_in);
#pragma unroll
                for (int s = 0; s < 4; ++s)
#pragma unroll
                    for (int t = 0; t < RT; ++t) acc[t][i] = w4_product(w[t][s], now[s], acc[t][i]);
            }
        }
    }
    join_waves<RT, C>(a, acc, part, tile0, token0);
}

template <int RT>
const void *pick_linear(int columns) {
    return columns == 1   ? reinterpret_cast<const void *>(&k_w4_linear<RT, 1>)
           : columns == 2 ? reinterpret_cast<const void *>(&k_w4_linear<RT, 2>)
           : columns == 3 ? reinterpret_cast<const void *>(&k_w4_linear<RT, 3>)
                          : reinterpret_cast<const void *>(&k_w4_linear<RT, 4>);
}

const void *pick_held(int tiles) {
    return tiles == 4   ? reinterpret_cast<const void *>(&k_w4_linear_held<4>)
           : tiles == 3 ? reinterpret_cast<const void *>(&k_w4_linear_held<3>)
           : tiles == 2 ? reinterpret_cast<const void *>(&k_w4_linear_held<2>)
                        : reinterpret_cast<const void *>(&k_w4_linear_held<1>);
}

RowsArg matrix(const void *p, int64_t stride, int64_t rows, int columns) {
    return RowsArg{ar_rows{const_cast<void *>(p), rows > 1 ? stride : 0, 0}, rows, 1, columns};
}

}  // namespace
}  // namespace ar

using namespace ar;

extern "C" {

int64_t ar_w4_bytes(int64_t n_out, int64_t n_in) {
    W4Shape s;
    return w4_shape(n_out, n_in, &s) ? s.bytes() : AR_EINVAL;
}

int ar_w4_pack(const void *w, int64_t row_stride, void *packed, int64_t n_out, int64_t n_in, void *stream) {
    PackArgs a = {};
    if (!w4_shape(n_out, n_in, &a.s)) return AR_EINVAL;
    const RowsArg rw = matrix(w, row_stride, n_out, (int)n_in);
    if (!rw.valid() || !packed || !aligned_to(packed, 16)) return AR_EINVAL;
    if (overlap(rw.span(), Span{addr(packed), (uintptr_t)a.s.bytes()})) return AR_EALIAS;
    a.w = static_cast<const uint16_t *>(w), a.row_stride = rw.r.token_stride, a.packed = static_cast<uint8_t *>(packed);
    const int64_t items = (int64_t)a.s.tiles * 16 * ((a.s.chunks + 3) / 4 * 4 * kW4Chunk / 8);
    const int64_t blocks = (items + kThreads - 1) / kThreads;
    if (blocks > 0x7FFFFFFF / kThreads) return AR_EINVAL;
    return launch(reinterpret_cast<const void *>(&k_w4_pack), (unsigned)blocks, kThreads, a, stream);
}

int ar_w4_unpack(const void *packed, void *w, int64_t row_stride, int64_t n_out, int64_t n_in, void *stream) {
    UnpackArgs a = {};
    if (!w4_shape(n_out, n_in, &a.s)) return AR_EINVAL;
    const RowsArg rw = matrix(w, row_stride, n_out, (int)n_in);
    if (!rw.valid() || rw.self_overlap() || !packed || !aligned_to(packed, 16)) return AR_EINVAL;
    if (overlap(rw.span(), Span{addr(packed), (uintptr_t)a.s.bytes()})) return AR_EALIAS;
    a.w = static_cast<uint16_t *>(w), a.row_stride = rw.r.token_stride, a.packed = static_cast<const uint8_t *>(packed);
    const int64_t blocks = (n_out * (n_in / 8) + kThreads - 1) / kThreads;
    if (blocks > 0x7FFFFFFF / kThreads) return AR_EINVAL;
    return launch(reinterpret_cast<const void *>(&k_w4_unpack), (unsigned)blocks, kThreads, a, stream);
}

int ar_w4_linear(ar_rows x, const void *packed, ar_rows out, int64_t tokens, int64_t n_out, int64_t n_in, void *stream) {
    W4Shape shape;
    if (!w4_shape(n_out, n_in, &shape) || tokens < 0 || tokens > 1 << 20) return AR_EINVAL;
    if (tokens == 0) return AR_OK;
    const RowsArg rx = matrix(x.p, x.token_stride, tokens, (int)n_in), ro = matrix(out.p, out.token_stride, tokens, (int)n_out);
    if (!rx.valid() || !ro.valid() || ro.self_overlap() || !packed || !aligned_to(packed, 16)) return AR_EINVAL;
    if (ro.overlaps(rx) || overlap(ro.span(), Span{addr(packed), (uintptr_t)shape.bytes()})) return AR_EALIAS;
    LinearArgs a = {static_cast<const uint8_t *>(packed), static_cast<const uint16_t *>(x.p), static_cast<uint16_t *>(out.p),
                    rx.r.token_stride, ro.r.token_stride, (int)n_out, (int)n_in, (int)tokens};
    const int columns = tokens <= 16 ? 1 : tokens <= 32 ? 2 : tokens <= 48 ? 3 : 4;
    const int64_t groups = (tokens + 16 * columns - 1) / (16 * columns);
    // The time of the compute unit that has most to do: for each chunk its
    // tiles' codes, and the inputs, which cost as much as two tiles for every 16
    // tokens however many tiles share them.  (64 tokens x 7168 x 7168 take 28.7, 18.9,
    // 21.7 and 23.6 us with one to four tiles, x 5120 x 10240 33.8, 27.1, 17.9 and 19.2,
    // x 8192 x 28672 106.8, 77.7, 66.1 and 51.8.)
    int tiles = 1;
    int64_t least = 0;
    for (int n = 1; n <= 4; ++n) {
        const int64_t time = ((shape.tiles + n - 1) / n * groups + kCus - 1) / kCus * (n + 2 * columns);
        if (n == 1 || time < least) least = time, tiles = n;
    }
    const int64_t blocks = (shape.tiles + tiles - 1) / tiles;
    const bool shared = blocks * groups > kCus;  // compute units get more than one workgroup
    const int64_t held_bytes = tokens * held_row(shape) * 2;
    const bool held = tokens <= (tiles == 1 ? 4 : 2) && (tiles < 4 || shared) && held_bytes <= kHeldBytes;
    const bool few = !held && tokens <= 8 && tiles == 4;
    // Four waves where compute units get more than one workgroup: 64 tokens x 8192 x
    // 28672 take 51.8 us, and 54.1 with eight; x 5120 x 17408, three tiles, 31.6 and
    // 34.3.  With one, eight: one token x 4096 x 14336 8.6, and 10.8 with four.  Where the
    // inputs are held, eight in both (one token x 8192 x 28672 24.4, and 25.7 with four),
    // and sixteen to single tiles of more than 16 chunks (x 7168 x 2112 4.2, 4.6 with
    // eight; x 2048 x 2048 3.3 and 3.0).
    const int waves = held ? (tiles == 1 && shape.chunks > 16 ? 16 : 8) : shared ? 4 : 8;
    const int sums = 1024 * (columns * tiles < kJoin ? columns * tiles : kJoin);
    const int inputs = held ? (int)held_bytes : few ? 0 : waves * kStage * 16;
    const unsigned lds = inputs > waves * sums ? inputs : waves * sums;
    void *args[] = {&a};
    const void *fn = held         ? pick_held(tiles)
                     : few        ? reinterpret_cast<const void *>(&k_w4_linear_few)
                     : tiles == 4 ? pick_linear<4>(columns)
                     : tiles == 3 ? pick_linear<3>(columns)
                     : tiles == 2 ? pick_linear<2>(columns)
                                  : pick_linear<1>(columns);
    return hipLaunchKernel(fn, dim3((unsigned)blocks, (unsigned)groups), dim3(64 * waves), args, lds,
                           static_cast<hipStream_t>(stream)) == hipSuccess
               ? AR_OK
               : AR_ELAUNCH;
}

}  // extern "C"
