// experts.hip -- a mixture-of-experts layer for a few tokens, from the router to
// the weighted sum, with weights of 4 bits.
//
// For a token x: logits R x, of which the top_k largest are taken; their softmax
// p; for each of those experts a = silu(G x) * (U x), and
//     out = scale * sum_j p_j D_j a_j.
// For a few tokens it is bound by the bytes of the experts that some token takes,
// each read once however many tokens do.
//
// Four launches, each waiting for the one before:
// k_router: logits, with sums in 64 bits, so that what an expert's place among a
//   token's turns on is the logit and not the order of a sum.  Matrix
//   instructions for 64 bits; the inputs are split over many workgroups.
// k_choose: joins the splits, and a token's experts by counting how many come
//   before each.
// k_experts_up: a workgroup has one expert that is taken, some tiles of its gate
//   and the same of its up part, and all the tokens that take it as columns.  The
//   result goes on in two bf16 parts, whose sum is off by 2^-17 of it at most:
//   rounding it to one would add as much to the output's error as the output's
//   own rounding.
// k_experts_down: a workgroup has some outputs of all experts; its waves take
//   the experts' chunks in turn.  Eight tokens of an expert are a column tile,
//   first parts in columns 0 to 7, second parts in 8 to 15.  Each wave adds what
//   a token gets into rows of its own in LDS, so that no sum depends on which
//   wave is first.
#include "host.h"
#include "rows.h"
#include "w4.h"

namespace ar {
namespace {

constexpr int kMaxExperts = 512, kMaxTopK = 16;
constexpr int kTogether = 64;  // tokens of a pass
constexpr int kMaxPairs = kTogether * kMaxTopK;
constexpr int kLogits = 65536;  // partial logits of a pass, at most
constexpr int kRouterWaves = 4, kUpWaves = 8, kDownWaves = 8;

typedef double f64x4 __attribute__((ext_vector_type(4)));

struct ExpertsArgs {
    W4Shape up, down;
    const uint8_t *gate_up, *dn;
    const uint16_t *router;
    Rows x, out;
    double *logits;  // [splits][tokens][experts]
    int32_t *choice;
    float *weight;
    uint16_t *act;  // [tokens top_k][2][inner]
    int tokens, hidden, inner, experts, top_k, splits;
    float scale;
};

// Logits of 16 experts and 16 tokens over a part of the inputs.  A lane takes
// eight inputs of its expert and of its token at a time, and product s of eight
// takes the s-th of each lane's.
__global__ __launch_bounds__(64 * kRouterWaves) void k_router(ExpertsArgs a) {
    __shared__ double part[kRouterWaves][16][17];
    const int lane = threadIdx.x % 64, r = lane % 16, q = lane / 16, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
    const int expert0 = blockIdx.x * 16, token0 = blockIdx.y * 16;
    const uint16_t *w = a.router + (int64_t)min(expert0 + r, a.experts - 1) * a.hidden + q * 8;
    const uint16_t *x = a.x.p + min(token0 + r, a.tokens - 1) * a.x.ts + q * 8;
    const int units = a.hidden / 32, all = gridDim.z * kRouterWaves, mine = blockIdx.z * kRouterWaves + wave;
    const int begin = (int)((int64_t)units * mine / all), end = (int)((int64_t)units * (mine + 1) / all);
    f64x4 acc = {0, 0, 0, 0};
    for (int u = begin; u < end; ++u) {
        const u32x4 vw = load_vec8<false>(w + u * 32), vx = load_vec8<false>(x + u * 32);
        float fw[8], fx[8];
        widen(vw, fw);
        widen(vx, fx);
#pragma unroll
        for (int s = 0; s < 8; ++s) acc = __builtin_amdgcn_mfma_f64_16x16x4f64((double)fw[s], (double)fx[s], acc, 0, 0, 0);
    }
    // a lane has experts q, 4 + q, 8 + q, 12 + q of token r
#pragma unroll
    for (int i = 0; i < 4; ++i) part[wave][r][4 * i + q] = acc[i];
    __syncthreads();
    const int t = threadIdx.x / 16, e = threadIdx.x % 16;
    if (token0 + t >= a.tokens || expert0 + e >= a.experts) return;
    double v = part[0][t][e];
#pragma unroll
    for (int i = 1; i < kRouterWaves; ++i) v += part[i][t][e];
    a.logits[((int64_t)blockIdx.z * a.tokens + token0 + t) * a.experts + expert0 + e] = v;
}

// A token's experts.  The order is that of the logits from the largest, NaN
// before all numbers, and of two alike the lower index first: a total one, so
// that each place has one expert.
__global__ __launch_bounds__(kMaxExperts) void k_choose(ExpertsArgs a) {
    __shared__ uint32_t keys[kMaxExperts];
    __shared__ float top[kMaxTopK];
    const int token = blockIdx.x, e = threadIdx.x;
    double v = 0;
    if (e < a.experts)
        for (int s = 0; s < a.splits; ++s) v += a.logits[((int64_t)s * a.tokens + token) * a.experts + e];
    const float logit = (float)v + 0.0f;  // no negative zero
    const uint32_t bits = __float_as_uint(logit);
    // rising with the logit; nothing past the experts is taken
    const uint32_t key = e >= a.experts ? 0 : logit != logit ? 0xFFFFFFFFu : bits >> 31 ? ~bits : bits | 0x80000000u;
    keys[e] = key;
    __syncthreads();
    int place = 0;
    for (int i = 0; i < a.experts; ++i) {
        const uint32_t other = keys[i];
        place += other > key || (other == key && i < e);
    }
    const bool taken = e < a.experts && place < a.top_k;
    if (taken) {
        a.choice[token * a.top_k + place] = e;
        top[place] = logit;
    }
    __syncthreads();
    if (e >= a.top_k) return;
    float sum = 0;
    for (int i = 0; i < a.top_k; ++i) sum += expf(top[i] - top[0]);
    a.weight[token * a.top_k + e] = expf(top[e] - top[0]) / sum * a.scale;
}

// How many of the lower lanes are in the mask.
__device__ __forceinline__ int below(uint64_t mask) {
    return __builtin_amdgcn_mbcnt_hi((uint32_t)(mask >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)mask, 0));
}

// One expert's tiles [tile0, tile0 + N) of the gate and of the up part, for all
// tokens that take it.
template <int N, int U>
__global__ __launch_bounds__(64 * kUpWaves) void k_experts_up(ExpertsArgs a) {
    __shared__ int taken[kMaxExperts];
    __shared__ int list[kMaxPairs];  // the pairs (token, place) that take the expert
    __shared__ f32x4 part[kUpWaves][2 * N][64];
    const int lane = threadIdx.x % 64, r = lane % 16, q = lane / 16, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
    const int pairs = a.tokens * a.top_k;

    // the expert: the blockIdx.y-th of those that are taken
    for (int i = threadIdx.x; i < kMaxExperts; i += blockDim.x) taken[i] = 0;
    __syncthreads();
    for (int i = threadIdx.x; i < pairs; i += blockDim.x) taken[a.choice[i]] = 1;
    __syncthreads();
    int expert = -1, before = 0;
    for (int w = 0; w < a.experts; w += 64) {
        const uint64_t mask = __ballot(w + lane < a.experts && taken[min(w + lane, kMaxExperts - 1)]);
        const int at = (int)blockIdx.y - before, n = __popcll(mask);
        if (at < n) {
            expert = w + __builtin_ctzll(__ballot((mask >> lane & 1) && below(mask) == at));
            break;
        }
        before += n;
    }
    if (expert < 0) return;
    expert = __builtin_amdgcn_readfirstlane(expert);
    int count = 0;
    for (int p = 0; p < pairs; p += 64) {
        const bool mine = p + lane < pairs && a.choice[min(p + lane, pairs - 1)] == expert;
        const uint64_t mask = __ballot(mine);
        if (mine && wave == 0) list[count + below(mask)] = p + lane;
        count += __popcll(mask);
    }
    __syncthreads();

    const int half = a.inner / 16;  // tiles of the gate
    const int tile0 = blockIdx.x * N;
    const uint8_t *base = a.gate_up + expert * a.up.bytes();
    const uint8_t *tile[2 * N];
#pragma unroll
    for (int t = 0; t < N; ++t) {
        const int at = min(tile0 + t, half - 1);
        tile[t] = base + at * a.up.tile_bytes;
        tile[N + t] = base + (half + at) * a.up.tile_bytes;
    }
    for (int first = 0; first < count; first += 16) {
        const uint16_t *row = a.x.p + list[min(first + r, count - 1)] / a.top_k * a.x.ts;
        f32x4 acc[2 * N];
#pragma unroll
        for (int t = 0; t < 2 * N; ++t) acc[t] = f32x4{0, 0, 0, 0};
        const auto step = [&](int chunk, auto number) {
            constexpr int M = decltype(number)::value;
            u32x4 codes[M][2 * N], x[M][4];
            uint32_t byte[M][2 * N];
#pragma unroll
            for (int u = 0; u < M; ++u) {
                const int c = chunk + u * kUpWaves;
#pragma unroll
                for (int t = 0; t < 2 * N; ++t) {
                    codes[u][t] = *reinterpret_cast<const u32x4 *>(tile[t] + w4_code_at(c, lane));
                    byte[u][t] = tile[t][w4_scale_at(a.up.chunks, c, lane)];
                }
                load_inputs(x[u], row, c * kW4Chunk + q * 32, a.hidden);
            }
#pragma unroll
            for (int u = 0; u < M; ++u)
#pragma unroll
                for (int s = 0; s < 4; ++s)
#pragma unroll
                    for (int t = 0; t < 2 * N; ++t)
                        acc[t] = w4_product(w4_operand(codes[u][t], kv4_scale(byte[u][t]), s), x[u][s], acc[t]);
        };
        int c = wave;
        for (; c + (U - 1) * kUpWaves < a.up.chunks; c += U * kUpWaves) step(c, std::integral_constant<int, U>());
        for (; c < a.up.chunks; c += kUpWaves) step(c, std::integral_constant<int, 1>());
        if (first) __syncthreads();
#pragma unroll
        for (int t = 0; t < 2 * N; ++t) part[wave][t][lane] = acc[t];
        __syncthreads();
        for (int item = threadIdx.x; item < N * 64; item += blockDim.x) {
            const int t = item / 64, at = item % 64, column = first + at % 16;
            if (column >= count || tile0 + t >= half) continue;
            f32x4 g = part[0][t][at], u = part[0][N + t][at];
#pragma unroll
            for (int w = 1; w < kUpWaves; ++w) g += part[w][t][at], u += part[w][N + t][at];
            uint16_t *to = a.act + (int64_t)list[column] * 2 * a.inner + (tile0 + t) * 16 + at / 16 * 4;
            uint32_t hi[2], lo[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                float v[2], rest[2];
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const float z = g[2 * i + j];
                    v[j] = z / (1.0f + expf(-z)) * u[2 * i + j];
                }
                hi[i] = bf16_pair(v[0], v[1]);
                const float back[2] = {lo_f32(hi[i]), hi_f32(hi[i])};
#pragma unroll
                for (int j = 0; j < 2; ++j) rest[j] = fabsf(back[j]) < __builtin_inff() ? v[j] - back[j] : 0.0f;
                lo[i] = bf16_pair(rest[0], rest[1]);
            }
            *reinterpret_cast<uint2 *>(to) = uint2{hi[0], hi[1]};
            *reinterpret_cast<uint2 *>(to + a.inner) = uint2{lo[0], lo[1]};
        }
    }
}

// N tiles of the outputs.
template <int N>
__global__ __launch_bounds__(64 * kDownWaves) void k_experts_down(ExpertsArgs a) {
    extern __shared__ f32x4 sums[];  // [waves][tokens][4 N]
    __shared__ int counts[kMaxExperts], starts[kMaxExperts];
    __shared__ int expert_of[kMaxExperts], used;
    __shared__ int list[kMaxPairs];
    __shared__ float weights[kMaxPairs];
    const int lane = threadIdx.x % 64, r = lane % 16, q = lane / 16, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
    const int pairs = a.tokens * a.top_k;

    // The pairs by expert.  Their order within one is left open: it says which
    // column a token is in, and no more.
    for (int i = threadIdx.x; i < kMaxExperts; i += blockDim.x) counts[i] = 0;
    for (int i = threadIdx.x; i < kDownWaves * a.tokens * 4 * N; i += blockDim.x) sums[i] = f32x4{0, 0, 0, 0};
    __syncthreads();
    constexpr int kEach = kMaxPairs / (64 * kDownWaves);
    int place[kEach], expert[kEach];
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
        const int p = threadIdx.x + i * 64 * kDownWaves;
        expert[i] = p < pairs ? a.choice[p] : -1;
        if (expert[i] >= 0) place[i] = atomicAdd(&counts[expert[i]], 1);
    }
    __syncthreads();
    if (wave == 0) {
        int start = 0, slot = 0;
        for (int w = 0; w < a.experts; w += 64) {
            const int e = w + lane, n = e < a.experts ? counts[min(e, kMaxExperts - 1)] : 0;
            int sum = n;
#pragma unroll
            for (int d = 1; d < 64; d *= 2) {
                const int left = __shfl_up(sum, d);
                if (lane >= d) sum += left;
            }
            const uint64_t mask = __ballot(n > 0);
            if (n > 0) {
                expert_of[slot + below(mask)] = e;
                starts[e] = start + sum - n;
            }
            start += __shfl(sum, 63);
            slot += __popcll(mask);
        }
        if (lane == 0) used = slot;
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
        const int p = threadIdx.x + i * 64 * kDownWaves;
        if (expert[i] >= 0) {
            list[starts[expert[i]] + place[i]] = p;
            weights[starts[expert[i]] + place[i]] = a.weight[p];
        }
    }
    __syncthreads();

    const int tile0 = blockIdx.x * N, chunks = a.down.chunks, items = used * chunks;
    f32x4 *mine = sums + wave * a.tokens * 4 * N;
    for (int item = wave; item < items; item += kDownWaves) {
        const int e = __builtin_amdgcn_readfirstlane(expert_of[item / chunks]), c = item % chunks;
        const int start = __builtin_amdgcn_readfirstlane(starts[e]), count = __builtin_amdgcn_readfirstlane(counts[e]);
        const uint8_t *base = a.dn + e * a.down.bytes();
        u32x4 codes[N];
        uint32_t byte[N];
#pragma unroll
        for (int t = 0; t < N; ++t) {
            const uint8_t *tile = base + min(tile0 + t, a.down.tiles - 1) * a.down.tile_bytes;
            codes[t] = *reinterpret_cast<const u32x4 *>(tile + w4_code_at(c, lane));
            byte[t] = tile[w4_scale_at(chunks, c, lane)];
        }
        for (int first = 0; first < count; first += 8) {
            const int at = start + min(first + r % 8, count - 1), pair = list[at];
            u32x4 x[4];
            load_inputs(x, a.act + ((int64_t)pair * 2 + r / 8) * a.inner, c * kW4Chunk + q * 32, a.inner);
            const float weight = weights[at];
            const int token = pair / a.top_k;
#pragma unroll
            for (int t = 0; t < N; ++t) {
                f32x4 d = {0, 0, 0, 0};
#pragma unroll
                for (int s = 0; s < 4; ++s) d = w4_product(w4_operand(codes[t], kv4_scale(byte[t]), s), x[s], d);
#pragma unroll
                for (int i = 0; i < 4; ++i) d[i] = dpp_add<0x128, 0xf>(d[i]);  // the two parts
                if (r < 8 && first + r < count) {
                    f32x4 &to = mine[(token * N + t) * 4 + q];
                    to += weight * d;
                }
                // the next expert's columns are others: its lanes read what these wrote
                __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
            }
        }
    }
    __syncthreads();
    for (int i = threadIdx.x; i < a.tokens * 4 * N; i += blockDim.x) {
        f32x4 v = sums[i];
        for (int w = 1; w < kDownWaves; ++w) v += sums[w * a.tokens * 4 * N + i];
        const int token = i / (4 * N);
        const int64_t n = (int64_t)tile0 * 16 + i % (4 * N) * 4;
        if (n >= a.hidden) continue;  // n_out is a multiple of 32
        uint16_t *to = const_cast<uint16_t *>(a.out.p) + token * a.out.ts + n;
        typedef uint32_t u32x2_any __attribute__((ext_vector_type(2), aligned(2)));
        *reinterpret_cast<u32x2_any *>(to) = u32x2_any{bf16_pair(v[0], v[1]), bf16_pair(v[2], v[3])};
    }
}

int launch3(const void *fn, dim3 grid, unsigned block, unsigned lds, ExpertsArgs &a, void *stream) {
    void *args[] = {&a};
    return hipLaunchKernel(fn, grid, dim3(block), args, lds, static_cast<hipStream_t>(stream)) == hipSuccess ? AR_OK : AR_ELAUNCH;
}

bool valid_sizes(int64_t tokens, int64_t hidden, int64_t inner, int experts, int top_k, W4Shape *up, W4Shape *down) {
    return tokens >= 0 && tokens <= 1 << 20 && inner >= 32 && inner <= 1 << 19 && experts >= 1 && experts <= kMaxExperts && top_k >= 1 &&
           top_k <= kMaxTopK && top_k <= experts && w4_shape(2 * inner, hidden, up) && w4_shape(hidden, inner, down);
}

}  // namespace
}  // namespace ar

using namespace ar;

extern "C" {

int64_t ar_w4_experts_workspace(int64_t tokens, int64_t hidden, int64_t inner, int experts, int top_k) {
    W4Shape up, down;
    if (!valid_sizes(tokens, hidden, inner, experts, top_k, &up, &down)) return AR_EINVAL;
    const int64_t pairs = (tokens < kTogether ? tokens : kTogether) * top_k;
    return kLogits * 8 + pairs * 4 * inner;
}

int ar_w4_experts(ar_rows x, const void *router, const void *gate_up, const void *down, ar_rows out, void *choice, void *weight,
                  void *workspace, int64_t tokens, int64_t hidden, int64_t inner, int experts, int top_k, float scale, void *stream) {
    ExpertsArgs a = {};
    if (!valid_sizes(tokens, hidden, inner, experts, top_k, &a.up, &a.down) || !(scale >= -3.0e38f && scale <= 3.0e38f)) return AR_EINVAL;
    if (tokens == 0) return AR_OK;
    const auto row_arg = [&](ar_rows r) { return RowsArg{ar_rows{r.p, tokens > 1 ? r.token_stride : 0, 0}, tokens, 1, (int)hidden}; };
    const RowsArg rx = row_arg(x), ro = row_arg(out);
    if (!rx.valid() || !ro.valid() || ro.self_overlap() || !router || !aligned_to(router, 2) || !gate_up || !aligned_to(gate_up, 16) ||
        !down || !aligned_to(down, 16) || !choice || !aligned_to(choice, 4) || !weight || !aligned_to(weight, 4) || !workspace ||
        !aligned_to(workspace, 16))
        return AR_EINVAL;
    const Span reads[] = {rx.span(), {addr(router), (uintptr_t)(2 * experts * hidden)}, {addr(gate_up), (uintptr_t)(experts * a.up.bytes())},
                          {addr(down), (uintptr_t)(experts * a.down.bytes())}};
    const Span writes[] = {ro.span(), {addr(choice), (uintptr_t)(4 * tokens * top_k)}, {addr(weight), (uintptr_t)(4 * tokens * top_k)},
                           {addr(workspace), (uintptr_t)ar_w4_experts_workspace(tokens, hidden, inner, experts, top_k)}};
    for (int i = 0; i < 4; ++i) {
        for (int j = 0; j < 4; ++j)
            if ((j < i && overlap(writes[i], writes[j])) || (!(i == 0 && j == 0) && overlap(writes[i], reads[j]))) return AR_EALIAS;
    }
    if (ro.overlaps(rx)) return AR_EALIAS;
    a.gate_up = static_cast<const uint8_t *>(gate_up), a.dn = static_cast<const uint8_t *>(down);
    a.router = static_cast<const uint16_t *>(router);
    a.logits = static_cast<double *>(workspace);
    a.act = reinterpret_cast<uint16_t *>(static_cast<uint8_t *>(workspace) + kLogits * 8);
    a.hidden = (int)hidden, a.inner = (int)inner, a.experts = experts, a.top_k = top_k, a.scale = scale;
    for (int64_t at = 0; at < tokens; at += kTogether) {
        a.tokens = (int)(tokens - at < kTogether ? tokens - at : kTogether);
        a.x = rows(rx), a.out = rows(ro);
        a.x.p += at * a.x.ts, a.out.p += at * a.out.ts;
        a.choice = static_cast<int32_t *>(choice) + at * top_k, a.weight = static_cast<float *>(weight) + at * top_k;
        const int expert_tiles = (experts + 15) / 16, token_tiles = (a.tokens + 15) / 16, units = (int)hidden / 32;
        a.splits = 256 / (expert_tiles * token_tiles);
        if (a.splits > (units + kRouterWaves - 1) / kRouterWaves) a.splits = (units + kRouterWaves - 1) / kRouterWaves;
        if (a.splits < 1) a.splits = 1;
        int rc = launch3(reinterpret_cast<const void *>(&k_router), dim3(expert_tiles, token_tiles, a.splits), 64 * kRouterWaves, 0, a, stream);
        if (rc != AR_OK) return rc;
        rc = launch3(reinterpret_cast<const void *>(&k_choose), dim3(a.tokens), (unsigned)round_up(experts, 64), 0, a, stream);
        if (rc != AR_OK) return rc;
        const int slots = a.tokens * top_k < experts ? a.tokens * top_k : experts;
        const int half = (int)inner / 16;
        const bool wide = (int64_t)slots * half >= 2048;
        rc = launch3(wide ? reinterpret_cast<const void *>(&k_experts_up<2, 2>) : reinterpret_cast<const void *>(&k_experts_up<1, 4>),
                     dim3(wide ? (half + 1) / 2 : half, slots), 64 * kUpWaves, 0, a, stream);
        if (rc != AR_OK) return rc;
        const int n = 1;
        rc = launch3(reinterpret_cast<const void *>(&k_experts_down<1>), dim3((a.down.tiles + n - 1) / n), 64 * kDownWaves,
                     kDownWaves * a.tokens * 64 * n, a, stream);
        if (rc != AR_OK) return rc;
    }
    return AR_OK;
}

}  // extern "C"
