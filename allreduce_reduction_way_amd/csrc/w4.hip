// w4.hip -- weights of 4 bits: packed from bf16 and unpacked, and a few tokens'
// products with them.
//
// out = x W^T with W's codes turned into bf16, which is exact, and products added
// up in binary32 by the matrix unit.  For up to some 64 tokens it is bound by the
// weights' bytes, 17/32 of one each, or by latency where there are few of those.
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
// byte is written: what lies past the matrix becomes zeros.
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
    if (c < a.s.chunks) *reinterpret_cast<uint32_t *>(tile + w4_code_at(c, lane) + k % 32 / 2) = codes;
    if (k % 32 == 0) tile[w4_scale_at(a.s.chunks, c, lane)] = (uint8_t)byte;
}

struct UnpackArgs {
    W4Shape s;
    const uint8_t *packed;
    uint16_t *w;
    int64_t row_stride;
};

__global__ __launch_bounds__(kThreads) void k_w4_unpack(UnpackArgs a) {
    const int octets = a.s.n_in / 8;
    const int64_t item = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    const int64_t n = item / octets;
    const int k = (int)(item % octets) * 8;
    if (n >= a.s.n_out) return;
    const uint8_t *tile = a.packed + n / 16 * a.s.tile_bytes;
    const int c = k / kW4Chunk, lane = k % kW4Chunk / 32 * 16 + (int)(n % 16);
    const uint32_t codes = *reinterpret_cast<const uint32_t *>(tile + w4_code_at(c, lane) + k % 32 / 2);
    *reinterpret_cast<u32x4_any *>(a.w + n * a.row_stride + k) = kv4_dequantise(codes, tile[w4_scale_at(a.s.chunks, c, lane)]);
}

struct LinearArgs {
    W4Shape s;
    const uint8_t *packed;
    Rows x, out;
    int64_t tokens;
};

// A workgroup computes RT tiles of outputs for C times 16 tokens.  Its waves take
// the chunks in turn, each with sums of its own, and join them through LDS.  U:
// chunks that a wave has on their way at once.
template <int RT, int C, int U>
__global__ __launch_bounds__(512) void k_w4_linear(LinearArgs a) {
    extern __shared__ f32x4 part[];  // [waves][min(RT C, 4)][64]
    const int lane = threadIdx.x % 64, r = lane % 16, q = lane / 16;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64), waves = blockDim.x / 64;
    const int tile0 = blockIdx.x * RT;
    const int64_t token0 = (int64_t)blockIdx.y * (16 * C);
    const uint8_t *tile[RT];
    const uint16_t *row[C];
#pragma unroll
    for (int t = 0; t < RT; ++t) tile[t] = a.packed + min(tile0 + t, a.s.tiles - 1) * a.s.tile_bytes;
    // a column past the tokens is not stored; it takes the last token's row
#pragma unroll
    for (int c = 0; c < C; ++c) row[c] = a.x.p + min(token0 + c * 16 + r, a.tokens - 1) * a.x.ts;
    f32x4 acc[RT][C];
#pragma unroll
    for (int t = 0; t < RT; ++t)
#pragma unroll
        for (int c = 0; c < C; ++c) acc[t][c] = f32x4{0, 0, 0, 0};

    const auto step = [&](int first, auto count) {
        constexpr int N = decltype(count)::value;
        u32x4 codes[N][RT], x[N][C][4];
        uint32_t byte[N][RT];
#pragma unroll
        for (int u = 0; u < N; ++u) {
            const int c = first + u * waves;
#pragma unroll
            for (int t = 0; t < RT; ++t) {
                codes[u][t] = *reinterpret_cast<const u32x4 *>(tile[t] + w4_code_at(c, lane));
                byte[u][t] = tile[t][w4_scale_at(a.s.chunks, c, lane)];
            }
#pragma unroll
            for (int i = 0; i < C; ++i) load_inputs(x[u][i], row[i], c * kW4Chunk + q * 32, a.s.n_in);
        }
#pragma unroll
        for (int u = 0; u < N; ++u)
#pragma unroll
            for (int s = 0; s < 4; ++s)
#pragma unroll
                for (int t = 0; t < RT; ++t) {
                    const bf16x8 w = w4_operand(codes[u][t], kv4_scale(byte[u][t]), s);
#pragma unroll
                    for (int i = 0; i < C; ++i) acc[t][i] = w4_product(w, x[u][i][s], acc[t][i]);
                }
    };
    int c = wave;
    for (; c + (U - 1) * waves < a.s.chunks; c += U * waves) step(c, std::integral_constant<int, U>());
    for (; c < a.s.chunks; c += waves) step(c, std::integral_constant<int, 1>());

    // the waves' sums, some tiles of the output at a time
    constexpr int kTogether = RT * C < 4 ? RT * C : 4;
#pragma unroll
    for (int first = 0; first < RT * C; first += kTogether) {
        if (first) __syncthreads();
#pragma unroll
        for (int i = 0; i < kTogether; ++i) part[(wave * kTogether + i) * 64 + lane] = acc[(first + i) / C][(first + i) % C];
        __syncthreads();
        for (int item = threadIdx.x; item < kTogether * 64; item += blockDim.x) {
            f32x4 v = part[item];
            for (int w = 1; w < waves; ++w) v += part[w * kTogether * 64 + item];
            const int i = first + item / 64, at = item % 64;
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

template <int RT>
const void *pick_linear(int columns) {
    return columns == 1   ? reinterpret_cast<const void *>(&k_w4_linear<RT, 1, RT == 4 ? 2 : 4>)
           : columns == 2 ? reinterpret_cast<const void *>(&k_w4_linear<RT, 2, 2>)
                          : reinterpret_cast<const void *>(&k_w4_linear<RT, 4, 1>);
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
    LinearArgs a = {};
    if (!w4_shape(n_out, n_in, &a.s) || tokens < 0 || tokens > 1 << 20) return AR_EINVAL;
    if (tokens == 0) return AR_OK;
    const RowsArg rx = matrix(x.p, x.token_stride, tokens, (int)n_in), ro = matrix(out.p, out.token_stride, tokens, (int)n_out);
    if (!rx.valid() || !ro.valid() || ro.self_overlap() || !packed || !aligned_to(packed, 16)) return AR_EINVAL;
    if (ro.overlaps(rx) || overlap(ro.span(), Span{addr(packed), (uintptr_t)a.s.bytes()})) return AR_EALIAS;
    a.packed = static_cast<const uint8_t *>(packed);
    a.x = rows(rx), a.out = rows(ro), a.tokens = tokens;
    const int columns = tokens <= 16 ? 1 : tokens <= 32 ? 2 : 4;
    const int64_t groups = (tokens + 16 * columns - 1) / (16 * columns);
    const int tiles = a.s.tiles * groups >= 2048 ? 4 : a.s.tiles * groups >= 1024 ? 2 : 1;
    const int waves = columns == 4 && tiles == 4 ? 4 : 8;
    const unsigned lds = waves * (columns * tiles < 4 ? columns * tiles : 4) * 1024;
    void *args[] = {&a};
    const void *fn = tiles == 4 ? pick_linear<4>(columns) : tiles == 2 ? pick_linear<2>(columns) : pick_linear<1>(columns);
    return hipLaunchKernel(fn, dim3((a.s.tiles + tiles - 1) / tiles, (unsigned)groups), dim3(64 * waves), args, lds,
                           static_cast<hipStream_t>(stream)) == hipSuccess
               ? AR_OK
               : AR_ELAUNCH;
}

}  // extern "C"
