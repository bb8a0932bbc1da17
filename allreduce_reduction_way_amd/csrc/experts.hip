// experts.hip -- a mixture-of-experts layer for a few tokens, from the router to
// the weighted sum, with weights of 4 bits.
//
// For a token x: logits R x, of which the top_k largest are taken; their softmax
// p; for each of those experts a = silu(G x) * (U x), and
//     out = scale * sum_j p_j D_j a_j.
// For a few tokens it is bound by the bytes of the experts that some token takes.  An
// expert's weights are read again for every 16 of its tokens in the first product and for
// every five or ten in the second, from the caches where they last: 64 tokens x 5120
// through 128 experts of 768 take 183 us (4.3 TB/s of weights read once), five x 7168
// through 256 of 256 44 us (2.6 TB/s; 40 where the caches hold some), one x 5120 through
// 64 of 192, which is latency, 16.8 us.  All 64 taking the same eight of the 128 take 100
// us, ten times those weights' bytes: the work on an expert stays in as many workgroups
// as it has tiles.
//
// Three to five launches, each waiting for the one before:
// k_router: logits, with sums in 64 bits, so that what an expert's place among a
//   token's turns on is the logit and not the order of a sum.  Matrix
//   instructions for 64 bits; the inputs are split over many workgroups.
// k_choose: joins the splits, and takes a token's experts from the largest logit
//   down.  For a small router k_route does both.
// k_experts_up: a workgroup has one expert that is taken, some tiles of its gate
//   and the same of its up part, and all the tokens that take it as columns.  The
//   result goes on in three bf16 parts, whose sum is the binary32 number: with
//   two, 16 of its 24 bits, one output in a thousand came out as its neighbour.
//   Up to five tokens of an expert are a group, which lies in memory as the next
//   product takes it: first parts in columns 0 to 4, second parts in 5 to 9,
//   third parts in 10 to 14.  (Eight tokens, with the third parts in an operand of
//   their own, are twice the instructions for up to five: five tokens x 7168 through
//   256 experts of 256 took 42.1 us so, 40.4 with this, 64 x 5120 through 128 of 768
//   182.9 and 183.1.  Two parts, of 16 bits, took 39.7 and 171.7.)
// k_experts_down: a workgroup has one expert, some tiles of its outputs, and its
//   groups one or two at a time in LDS.  Each token's result is left in binary32.
// k_experts_sum: a token's results by weight, in the order of its experts.
// Where the chunks are few, k_experts_down_few (up to five tokens) or
// k_experts_down_all makes products and sums at once.
#include <math.h>

#include "host.h"
#include "rows.h"
#include "w4.h"

namespace ar {
namespace {

constexpr int kMaxExperts = 512, kMaxTopK = 16;
constexpr int kTogether = 64;  // tokens of a pass
constexpr int kMaxPairs = kTogether * kMaxTopK;
constexpr int kRouterParts = 512;           // workgroups of the router, but for the smallest and largest sizes
constexpr int kRouteAlone = 1 << 15;          // weights of a router whose logits one workgroup makes
constexpr int kLogits = kRouterParts * 256;  // partial logits of a pass, at most
constexpr int kRouterWaves = 4, kChooseWaves = 8, kRouteWaves = 16, kUpWaves = 8, kDownWaves = 8, kFewWaves = 16;
constexpr int kFewChunks = 128;  // see k_experts_down_few, k_experts_down_all
constexpr int kColumns = 5, kParts = 3;  // tokens of a group; of a 16-column operand the parts take all but one
constexpr int kCus = 256;

typedef double f64x4 __attribute__((ext_vector_type(4)));

// The numbers of a pass in one word.
struct Sizes {
    uint32_t word;

    static Sizes of(int tokens, int top_k, int experts, bool few, bool all) {
        return Sizes{(uint32_t)tokens | (uint32_t)top_k << 7 | (uint32_t)experts << 12 | (uint32_t)few << 22 | (uint32_t)all << 23};
    }
    __device__ __forceinline__ int tokens() const { return word & 127; }
    __device__ __forceinline__ int top_k() const { return word >> 7 & 31; }
    __device__ __forceinline__ int experts() const { return word >> 12 & 1023; }
    // up to kColumns tokens, whose columns are the same in every expert
    __device__ __forceinline__ int few() const { return word >> 22 & 1; }
    // more, and few chunks of all groups: `taken` has an entry for each group
    __device__ __forceinline__ int all() const { return word >> 23 & 1; }
};

// The workspace: logits, the experts that are taken, the groups' pairs, what goes
// into the second product, and what comes out.  `most`: groups, at most.
struct Places {
    int64_t used, taken, pair, act, y;
    __host__ __device__ Places(int64_t most, int chunks)
        : used((int64_t)kLogits * 8), taken(used + 16), pair(taken + most * 16), act(pair + (most * kColumns * 4 + 15) / 16 * 16), y(act + most * chunks * 4 * 64 * 16) {}
};

// Arguments of the launches, up to 64 bytes each: with more a launch costs its
// caller 3.3 us (three tokens x 608 through 8 experts of 64 take 10.3 us so, and 10.5 with
// 250 bytes).
struct RouteArgs {
    const uint16_t *router, *x;
    int64_t x_stride;
    double *logits;
    int32_t *choice;
    float *weight;
    int hidden, splits;
    float scale;
    Sizes sizes;
};

struct UpArgs {
    const uint8_t *gate_up;
    const uint16_t *x;
    int64_t x_stride;
    const int32_t *choice;
    const float *weight;
    uint8_t *workspace;
    int hidden, inner, most;
    Sizes sizes;
};

struct DownArgs {
    const uint8_t *down;
    const float *weight;
    uint16_t *out;
    int64_t out_stride;
    uint8_t *workspace;
    int hidden, inner, most;
    Sizes sizes;
};
static_assert(sizeof(RouteArgs) <= 64 && sizeof(UpArgs) <= 64 && sizeof(DownArgs) <= 64, "arguments of a cheap launch");

// The same as the kernels take them.
struct ExpertsArgs {
    W4Shape up, down;
    const uint8_t *gate_up, *dn;
    const uint16_t *router;
    Rows x, out;
    double *logits;  // [splits][tokens][experts]
    int32_t *choice;
    float *weight;
    int32_t *used;        // how many experts are taken
    int4 *taken;          // each of them: expert, first group, tokens, and a bit for each token where there are few
    int32_t *group_pair;  // the pairs (token, place) of each group
    float *group_weight;  // where there are few, in its place: what each token weighs
    uint16_t *act;        // [groups][chunks of inner][4 steps][64 lanes][8], columns from kParts kColumns on of anything
    float *y;             // [pairs][hidden]
    int tokens, hidden, inner, experts, top_k, splits, few, all;
    float scale;

    __device__ __forceinline__ void take(Sizes s) {
        tokens = s.tokens(), top_k = s.top_k(), experts = s.experts(), few = s.few(), all = s.all();
    }
    __device__ __forceinline__ void place(uint8_t *workspace, int most) {
        const Places at(most, down.chunks);
        used = reinterpret_cast<int32_t *>(workspace + at.used), taken = reinterpret_cast<int4 *>(workspace + at.taken);
        group_pair = reinterpret_cast<int32_t *>(workspace + at.pair), group_weight = reinterpret_cast<float *>(workspace + at.pair);
        act = reinterpret_cast<uint16_t *>(workspace + at.act), y = reinterpret_cast<float *>(workspace + at.y);
    }
    __device__ __forceinline__ explicit ExpertsArgs(const RouteArgs &r)
        : router(r.router), x{r.x, r.x_stride, 0}, logits(r.logits), choice(r.choice), weight(r.weight), hidden(r.hidden), splits(r.splits), scale(r.scale) {
        take(r.sizes);
    }
    __device__ __forceinline__ explicit ExpertsArgs(const UpArgs &u)
        : up(w4_shape_of(2 * u.inner, u.hidden)), down(w4_shape_of(u.hidden, u.inner)), gate_up(u.gate_up), x{u.x, u.x_stride, 0},
          choice(const_cast<int32_t *>(u.choice)), weight(const_cast<float *>(u.weight)), hidden(u.hidden), inner(u.inner) {
        take(u.sizes);
        place(u.workspace, u.most);
    }
    __device__ __forceinline__ explicit ExpertsArgs(const DownArgs &d)
        : down(w4_shape_of(d.hidden, d.inner)), dn(d.down), out{d.out, d.out_stride, 0}, weight(const_cast<float *>(d.weight)), hidden(d.hidden), inner(d.inner) {
        take(d.sizes);
        place(d.workspace, d.most);
    }
};

// Logits of 16 experts and 16 tokens over a part of the inputs.  A lane takes
// eight inputs of its expert and of its token at a time, and product s of eight
// takes the s-th of each lane's.
__global__ __launch_bounds__(64 * kRouterWaves) void k_router(RouteArgs args) {
    const ExpertsArgs a(args);
    __shared__ double part[kRouterWaves][16][17];
    const int lane = threadIdx.x % 64, r = lane % 16, q = lane / 16, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
    const int expert0 = blockIdx.x * 16, token0 = blockIdx.y * 16;
    const uint16_t *w = a.router + (int64_t)min(expert0 + r, a.experts - 1) * a.hidden + q * 8;
    const uint16_t *x = a.x.p + min(token0 + r, a.tokens - 1) * a.x.ts + q * 8;
    const int units = a.hidden / 32, all = gridDim.z * kRouterWaves, mine = blockIdx.z * kRouterWaves + wave;
    const int begin = (int)((int64_t)units * mine / all), end = (int)((int64_t)units * (mine + 1) / all);
    f64x4 acc = {0, 0, 0, 0};
    for (int first = begin; first < end; first += 4) {
        u32x4 vw[4], vx[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int u = min(first + i, end - 1);
            vw[i] = load_vec8<false>(w + u * 32);
            vx[i] = load_vec8<false>(x + u * 32);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (first + i >= end) break;
            float fw[8], fx[8];
            widen(vw[i], fw);
            widen(vx[i], fx);
#pragma unroll
            for (int s = 0; s < 8; ++s) acc = __builtin_amdgcn_mfma_f64_16x16x4f64((double)fw[s], (double)fx[s], acc, 0, 0, 0);
        }
    }
    // a lane has experts q, 4 + q, 8 + q, 12 + q of token r
#pragma unroll
    for (int i = 0; i < 4; ++i) part[wave][r][4 * i + q] = acc[i];
    __syncthreads();
    const int t = threadIdx.x / 16, e = threadIdx.x % 16;
    if (t >= 16 || token0 + t >= a.tokens || expert0 + e >= a.experts) return;
    double v = part[0][t][e];
#pragma unroll
    for (int i = 1; i < kRouterWaves; ++i) v += part[i][t][e];
    a.logits[((int64_t)blockIdx.z * a.tokens + token0 + t) * a.experts + expert0 + e] = v;
}

// v of lane l + N of the sixteen; lanes without one get 0.
template <int N>
__device__ __forceinline__ float lane_after(float v) {
    return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0x100 + N, 0xf, 0xf, true));
}

// The parts of columns 0 to kColumns - 1 added up, there.
__device__ __forceinline__ f32x4 parts_sum(f32x4 d) {
#pragma unroll
    for (int i = 0; i < 4; ++i) d[i] += lane_after<kColumns>(d[i]) + lane_after<2 * kColumns>(d[i]);
    return d;
}

// How many of the lower lanes are in the mask.
__device__ __forceinline__ int below(uint64_t mask) {
    return __builtin_amdgcn_mbcnt_hi((uint32_t)(mask >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)mask, 0));
}

// The largest of the wave's values.
__device__ __forceinline__ uint32_t wave_max(uint32_t v) {
    v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x128, 0xf, 0xf, false));
    v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x124, 0xf, 0xf, false));
    v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x122, 0xf, 0xf, false));
    v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x121, 0xf, 0xf, false));
    uint32_t r = __builtin_amdgcn_readlane((int)v, 0);
    r = max(r, (uint32_t)__builtin_amdgcn_readlane((int)v, 16));
    r = max(r, (uint32_t)__builtin_amdgcn_readlane((int)v, 32));
    return max(r, (uint32_t)__builtin_amdgcn_readlane((int)v, 48));
}

// A token's experts are taken from the largest logit down, NaN before all numbers,
// and of two alike the lower index first: a total order, so that each is taken once.
// By one wave, whose lane l has the logits of experts l, 64 + l, ...
constexpr int kEach = kMaxExperts / 64;

struct Keys {
    uint32_t of[kEach];  // rise with the logits

    __device__ __forceinline__ void set(int w, bool there, double sum) {
        of[w] = 0;  // past the experts: below every logit's
        if (!there) return;
        const float logit = (float)sum + 0.0f;  // no negative zero
        const uint32_t bits = __float_as_uint(logit);
        of[w] = logit != logit ? 0xFFFFFFFFu : bits >> 31 ? ~bits : bits | 0x80000000u;
    }
    __device__ __forceinline__ void choose(const ExpertsArgs &a, int token, int lane) {
        int expert = 0;
        uint32_t mine = 0;
        for (int j = 0; j < a.top_k; ++j) {
            uint32_t top = 0;
#pragma unroll
            for (int w = 0; w < kEach; ++w) top = max(top, of[w]);
            top = wave_max(top);
            int found = -1;
#pragma unroll
            for (int w = 0; w < kEach; ++w) {
                if (w * 64 >= a.experts) break;
                const uint64_t mask = __ballot(of[w] == top);
                if (found < 0 && mask) {
                    const int at = __builtin_ctzll(mask);
                    found = w * 64 + at;
                    if (lane == at) of[w] = 0;
                }
            }
            if (lane == j) expert = found, mine = top;
        }
        const float logit = mine == 0xFFFFFFFFu ? __builtin_nanf("") : __uint_as_float(mine >> 31 ? mine & 0x7FFFFFFFu : ~mine);
        const float first = __uint_as_float(__builtin_amdgcn_readfirstlane(__float_as_int(logit)));
        const float e = lane < a.top_k ? expf(logit - first) : 0.0f;
        const float weight = e / row16_sum(e) * a.scale;  // kMaxTopK lanes side by side
        if (lane < a.top_k) {
            a.choice[token * a.top_k + lane] = expert;
            a.weight[token * a.top_k + lane] = weight;
        }
    }
};

// Joins the splits.  A workgroup to a token: its waves add them up, the first one
// chooses.
__global__ __launch_bounds__(64 * kChooseWaves) void k_choose(RouteArgs args) {
    const ExpertsArgs a(args);
    __shared__ double part[kChooseWaves][64];
    const int lane = threadIdx.x % 64, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64), token = blockIdx.x;
    // a wave has 64 experts, and a part of the splits where there are fewer words
    // of 64 than waves
    const int words = a.experts <= 64 ? 1 : a.experts <= 128 ? 2 : a.experts <= 256 ? 4 : 8, parts = kChooseWaves / words;
    const int64_t step = (int64_t)a.tokens * a.experts;
    const double *p = a.logits + (int64_t)token * a.experts + min(wave % words * 64 + lane, a.experts - 1);
    double sum = 0;
    for (int s = wave / words; s < a.splits; s += 8 * parts) {
        double t[8];  // all on their way at once
#pragma unroll
        for (int i = 0; i < 8; ++i) t[i] = p[min(s + i * parts, a.splits - 1) * step];
#pragma unroll
        for (int i = 0; i < 8; ++i) sum += s + i * parts < a.splits ? t[i] : 0.0;
    }
    part[wave][lane] = sum;
    __syncthreads();
    if (wave) return;
    Keys keys;
#pragma unroll
    for (int w = 0; w < kEach; ++w) {
        const bool there = w * 64 + lane < a.experts;
        double v = 0;
        if (there) {
            v = part[w][lane];
            for (int i = 1; i < parts; ++i) v += part[w + i * words][lane];
        }
        keys.set(w, there, v);
    }
    keys.choose(a, token, lane);
}

__device__ __forceinline__ double dpp_sum16(double v) {
    const auto step = [](double v, auto control) {
        constexpr int C = decltype(control)::value;
        const uint64_t b = __builtin_bit_cast(uint64_t, v);
        const uint32_t lo = __builtin_amdgcn_update_dpp(0, (int)(uint32_t)b, C, 0xf, 0xf, false);
        const uint32_t hi = __builtin_amdgcn_update_dpp(0, (int)(uint32_t)(b >> 32), C, 0xf, 0xf, false);
        return v + __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
    };
    v = step(v, std::integral_constant<int, 0x128>());
    v = step(v, std::integral_constant<int, 0x124>());
    v = step(v, std::integral_constant<int, 0x122>());
    return step(v, std::integral_constant<int, 0x121>());
}

// Logits and choice at once, where the router is small.  A workgroup to a token: a
// wave takes experts in turn, or parts of their inputs where there are fewer experts
// than waves.
__global__ __launch_bounds__(64 * kRouteWaves) void k_route(RouteArgs args) {
    const ExpertsArgs a(args);
    __shared__ double part[kMaxExperts][4];
    const int lane = threadIdx.x % 64, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64), token = blockIdx.x;
    const int parts = a.experts >= kRouteWaves ? 1 : kRouteWaves / a.experts;
    const uint16_t *x = a.x.p + token * a.x.ts;
    for (int item = wave; item < a.experts * parts; item += kRouteWaves) {
        const uint16_t *w = a.router + (int64_t)(item / parts) * a.hidden;
        double sum = 0;
        for (int k = (item % parts * 64 + lane) * 8; k < a.hidden; k += parts * 512) {
            const u32x4 vw = load_vec8<false>(w + k), vx = load_vec8<false>(x + k);
            float fw[8], fx[8];
            widen(vw, fw);
            widen(vx, fx);
#pragma unroll
            for (int i = 0; i < 8; ++i) sum = __builtin_fma((double)fw[i], (double)fx[i], sum);
        }
        sum = dpp_sum16(sum);
        if (lane % 16 == 0) part[item][lane / 16] = sum;
    }
    __syncthreads();
    if (wave) return;
    Keys keys;
#pragma unroll
    for (int w = 0; w < kEach; ++w) {
        const int expert = w * 64 + lane;
        double v = 0;
        if (expert < a.experts) {
            for (int i = expert * parts; i < (expert + 1) * parts; ++i) v += (part[i][0] + part[i][1]) + (part[i][2] + part[i][3]);
        }
        keys.set(w, expert < a.experts, v);
    }
    keys.choose(a, token, lane);
}

// One expert's tiles of the gate and of the up part, N each at a time, for all tokens
// that take it.  U: chunks that a wave has on their way at once, one or two side
// by side, whose scales come in one load (with a load for each, five tokens x 7168
// through 256 experts of 256 took 1.4 us more).
template <int N, int U>
__global__ __launch_bounds__(64 * kUpWaves) void k_experts_up(UpArgs args) {
    const ExpertsArgs a(args);
    __shared__ int chosen[kMaxPairs], counts[kMaxExperts];
    __shared__ int list[kTogether];  // the pairs (token, place) that take the expert
    __shared__ f32x4 part[kUpWaves][2 * N][64];
    const int lane = threadIdx.x % 64, r = lane % 16, q = lane / 16, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
    const int pairs = a.tokens * a.top_k;

    // the expert: the blockIdx.y-th of those that are taken, and the groups before its
    for (int i = threadIdx.x; i < kMaxExperts; i += blockDim.x) counts[i] = 0;
    __syncthreads();
    for (int i = threadIdx.x; i < pairs; i += blockDim.x) {
        const int e = a.choice[i];
        chosen[i] = e;
        atomicAdd(&counts[e], 1);
    }
    __syncthreads();
    int expert = -1, base = 0, before = 0, groups = 0;
    for (int w = 0; w < a.experts; w += 64) {
        const int n = w + lane < a.experts ? counts[min(w + lane, kMaxExperts - 1)] : 0, g = (n + kColumns - 1) / kColumns;
        const uint64_t mask = __ballot(n > 0);
        int left = 0, sum = 0;  // groups of the lanes below, of all lanes
#pragma unroll
        for (int b = 0; b < 4; ++b) {  // at most 13, ceil(kTogether / kColumns), to an expert
            const uint64_t bit = __ballot(g >> b & 1);
            left += below(bit) << b;
            sum += __popcll(bit) << b;
        }
        const int at = (int)blockIdx.y - before;
        if (at >= 0 && at < (int)__popcll(mask)) {
            const int l = __builtin_ctzll(__ballot((mask >> lane & 1) && below(mask) == at));
            expert = w + l;
            base = groups + __builtin_amdgcn_readlane(left, l);
        }
        before += __popcll(mask);
        groups += sum;
    }
    if (expert < 0) return;
    int count = 0;
    for (int p = 0; p < pairs; p += 64) {
        const bool mine = p + lane < pairs && chosen[min(p + lane, pairs - 1)] == expert;
        const uint64_t mask = __ballot(mine);
        if (mine && wave == 0) list[count + below(mask)] = p + lane;
        count += __popcll(mask);
    }
    __syncthreads();
    if (blockIdx.x == 0 && (int)threadIdx.x < count) {
        const int pair = list[threadIdx.x], token = pair / a.top_k;
        if (a.few) a.group_weight[base * kColumns + token] = a.weight[pair];
        else a.group_pair[base * kColumns + threadIdx.x] = pair;
        if (a.all) {
            if ((int)threadIdx.x == count - 1)
                for (int i = count; i % kColumns; ++i) a.group_pair[base * kColumns + i] = -1;
            if (threadIdx.x % kColumns == 0) a.taken[base + threadIdx.x / kColumns] = int4{expert, 0, 0, 0};
            if (blockIdx.y == 0 && threadIdx.x == 0) *a.used = groups;
        } else if (wave == 0) {
            int tokens = 0;  // few tokens are in one wave
            for (int t = 0; a.few && t < a.tokens; ++t) tokens |= (__ballot(token == t) != 0) << t;
            if (lane == 0) {
                a.taken[blockIdx.y] = int4{expert, base, count, tokens};
                if (blockIdx.y == 0) *a.used = before;
            }
        }
    }

    const int half = a.inner / 16;  // tiles of the gate
    const uint8_t *from = a.gate_up + expert * a.up.bytes();
    bool again = false;
    for (int tile0 = blockIdx.x * N; tile0 < half; tile0 += gridDim.x * N) {
        const uint8_t *tile[2 * N];
#pragma unroll
        for (int t = 0; t < N; ++t) {
            const int at = min(tile0 + t, half - 1);
            tile[t] = from + at * a.up.tile_bytes;
            tile[N + t] = from + (half + at) * a.up.tile_bytes;
        }
        for (int first = 0; first < count; first += 16) {
            const bool mine = first + r < count;
            const uint16_t *row = a.x.p + list[min(first + r, count - 1)] / a.top_k * a.x.ts + q * 32;
            f32x4 acc[2 * N];
#pragma unroll
            for (int t = 0; t < 2 * N; ++t) acc[t] = f32x4{0, 0, 0, 0};
            const auto step = [&](int chunk, auto number) {
                constexpr int M = decltype(number)::value;
                u32x4 codes[M][2 * N], x[M][4];
                uint32_t byte[M][2 * N];
#pragma unroll
                for (int u = 0; u < M; ++u) {
                    const int c = chunk + u;
#pragma unroll
                    for (int t = 0; t < 2 * N; ++t) {
                        codes[u][t] = w4_codes(tile[t], c, lane);
                        byte[u][t] = M == 1 ? w4_scale(tile[t], a.up.chunks, c, lane) : u ? byte[0][t] >> 8 : w4_two_scales(tile[t], a.up.chunks, c, lane);
                    }
                    const int at = min(c * kW4Chunk, a.hidden - 32 - q * 32);  // past the row: inside it
                    load_few_inputs(x[u], row + at, 8, mine);
                }
#pragma unroll
                for (int u = 0; u < M; ++u) {
                    const int c = chunk + u;
                    if ((c + 1) * kW4Chunk > a.hidden && c * kW4Chunk + q * 32 >= a.hidden) {
#pragma unroll
                        for (int s = 0; s < 4; ++s) x[u][s] = u32x4{0, 0, 0, 0};
                    }
#pragma unroll
                    for (int s = 0; s < 4; ++s)
#pragma unroll
                        for (int t = 0; t < 2 * N; ++t)
                            acc[t] = w4_product(w4_operand(codes[u][t], kv4_scale(byte[u][t] & 255), s), x[u][s], acc[t]);
                }
            };
            int c = U * wave;
            for (; c + U <= a.up.chunks; c += U * kUpWaves) step(c, std::integral_constant<int, U>());
            if (U > 1 && c < a.up.chunks) step(c, std::integral_constant<int, 1>());
            if (again) __syncthreads();
            again = true;
#pragma unroll
            for (int t = 0; t < 2 * N; ++t) part[wave][t][lane] = acc[t];
            __syncthreads();
            for (int item = threadIdx.x; item < N * 64; item += 64 * kUpWaves) {
                const int t = item / 64, at = item % 64, column = first + at % 16;
                if (column >= count || tile0 + t >= half) continue;
                f32x4 g = part[0][t][at], u = part[0][N + t][at];
#pragma unroll
                for (int w = 1; w < kUpWaves; ++w) g += part[w][t][at], u += part[w][N + t][at];
                // element k of chunk c is one of step s of lane (column, k's 32)
                const int k = (tile0 + t) * 16 + at / 16 * 4, c = k / kW4Chunk, s = k % 32 / 8;
                const int place = a.few ? list[column] / a.top_k : column % kColumns;
                uint16_t *to = a.act + ((((int64_t)(base + column / kColumns) * a.down.chunks + c) * 4 + s) * 64 +
                                        k % kW4Chunk / 32 * 16 + place) * 8 + k % 8;
                // each part is the eight bits that come next: no part of a number is infinite
                uint32_t bits[kParts][4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    float v = g[i] / (1.0f + expf(-g[i])) * u[i];
                    const bool number = fabsf(v) < __builtin_inff();
#pragma unroll
                    for (int p = 0; p < kParts; ++p) {
                        bits[p][i] = __float_as_uint(v) >> 16;
                        v = number ? v - __uint_as_float(bits[p][i] << 16) : 0.0f;
                    }
                }
#pragma unroll
                for (int p = 0; p < kParts; ++p)
                    *reinterpret_cast<uint2 *>(to + p * kColumns * 8) = uint2{bits[p][0] | bits[p][1] << 16, bits[p][2] | bits[p][3] << 16};
            }
        }
    }
}

// One expert's tiles, N to a wave, for up to G groups at a time.  Chunks come to LDS
// in blocks of kBlock / G.
constexpr int kBlock = 16;

template <int N, int G>
__global__ __launch_bounds__(64 * kDownWaves) void k_experts_down(DownArgs args) {
    const ExpertsArgs a(args);
    extern __shared__ u32x4 act[];  // [groups][chunks of a block][4 steps][64 lanes]
    if ((int)blockIdx.y >= *a.used) return;
    const int lane = threadIdx.x % 64, r = lane % 16, q = lane / 16, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
    const int4 mine = a.taken[blockIdx.y];
    const int expert = __builtin_amdgcn_readfirstlane(mine.x), base = __builtin_amdgcn_readfirstlane(mine.y), count = __builtin_amdgcn_readfirstlane(mine.z);
    const int chunks = a.down.chunks, groups = (count + kColumns - 1) / kColumns;
    const int tile0 = (blockIdx.x * kDownWaves + wave) * N;
    const uint8_t *tile[N];
#pragma unroll
    for (int t = 0; t < N; ++t) tile[t] = a.dn + expert * a.down.bytes() + min(tile0 + t, a.down.tiles - 1) * a.down.tile_bytes;
    u32x4 codes[2][N];
    uint32_t byte[2][N];
    const auto load = [&](int b, int c) {
#pragma unroll
        for (int t = 0; t < N; ++t) {
            codes[b][t] = w4_codes(tile[t], c, lane);
            byte[b][t] = w4_scale(tile[t], chunks, c, lane);
        }
    };
    for (int first = 0; first < groups; first += G) {
        f32x4 acc[N][G];
#pragma unroll
        for (int t = 0; t < N; ++t)
#pragma unroll
            for (int g = 0; g < G; ++g) acc[t][g] = f32x4{0, 0, 0, 0};
        for (int block = 0; block < chunks; block += kBlock / G) {
            const int some = min(chunks - block, kBlock / G);
            load(0, block);
            if (first + block) __syncthreads();
#pragma unroll
            for (int g = 0; g < G; ++g) {
                const u32x4 *from = reinterpret_cast<const u32x4 *>(a.act) + ((int64_t)(base + min(first + g, groups - 1)) * chunks + block) * 256;
                for (int i = threadIdx.x; i < some * 256; i += 64 * kDownWaves) {
                    const int k = (block + i / 256) * kW4Chunk + i % 64 / 16 * 32;
                    act[g * (some * 256) + i] = k < a.inner ? from[i] : u32x4{0, 0, 0, 0};  // nothing was written past it
                }
            }
            __syncthreads();
            for (int at = 0; at < some; at += 2) {
#pragma unroll
                for (int b = 0; b < 2; ++b) {
                    const int c = at + b;
                    if (c >= some) break;
                    load(1 - b, block + min(c + 1, some - 1));  // past the end: again what is there
#pragma unroll
                    for (int s = 0; s < 4; ++s) {
                        u32x4 x[G];
#pragma unroll
                        for (int g = 0; g < G; ++g) x[g] = act[(g * some + c) * 256 + s * 64 + lane];
#pragma unroll
                        for (int t = 0; t < N; ++t) {
                            const bf16x8 w = w4_operand(codes[b][t], kv4_scale(byte[b][t]), s);
#pragma unroll
                            for (int g = 0; g < G; ++g) acc[t][g] = w4_product(w, x[g], acc[t][g]);
                        }
                    }
                }
            }
        }
#pragma unroll
        for (int g = 0; g < G; ++g) {
            const int column = (first + g) * kColumns + r;
            const bool store = r < kColumns && column < count;
            const int pair = a.group_pair[base * kColumns + (store ? column : 0)];
#pragma unroll
            for (int t = 0; t < N; ++t) {
                const f32x4 d = parts_sum(acc[t][g]);
                if (store && tile0 + t < a.down.tiles)  // hidden is a multiple of 32
                    *reinterpret_cast<f32x4 *>(a.y + (int64_t)pair * a.hidden + (tile0 + t) * 16 + q * 4) = d;
            }
        }
    }
}

// Up to five tokens: a workgroup has N tiles of outputs of all experts that are taken,
// whose chunks its waves take in turn.  Each expert is one
// group, with the same columns for the same tokens: what an expert gives a token
// that does not take it is left out, whatever it is.  Each tile reads all the
// activations, four times the weights' bytes with five tokens, and where the chunks
// are many, those weigh more than a launch: five tokens x 7168 through 256 experts of 256
// (80 chunks) take 40.6 us in all, 44.2 with k_experts_down and k_experts_sum, four x
// 4096 through 8 of 1536 (96) 22.0 and 25.2, but five x 2624 through 16 of 1504 (192)
// 31.5 and 31.1, five x 2048 through 64 of 1408 (440) 66.0 and 49.9.  A single token
// takes a fifth of them.  (Two and four chunks on their way with eight waves took 0.9 and
// 1.8 us more.)
template <int N>
__global__ __launch_bounds__(64 * kFewWaves) void k_experts_down_few(DownArgs args) {
    const ExpertsArgs a(args);
    __shared__ f32x4 part[kFewWaves][N][4][kColumns];
    const int lane = threadIdx.x % 64, r = lane % 16, q = lane / 16, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
    const int chunks = a.down.chunks, token = r % kColumns, tile0 = blockIdx.x * N;
    const int items = *a.used * chunks;
    f32x4 sum[N];
#pragma unroll
    for (int t = 0; t < N; ++t) sum[t] = f32x4{0, 0, 0, 0};
    for (int item = wave; item < items; item += kFewWaves) {
        const int slot = item / chunks, c = item - slot * chunks;  // a group to a slot
        const int4 taken = a.taken[slot];
        const uint8_t *from = a.dn + __builtin_amdgcn_readfirstlane(taken.x) * a.down.bytes();
        const float weight = a.group_weight[slot * kColumns + token];
        u32x4 x[4], codes[N];
        uint32_t byte[N];
        load_few_inputs(x, a.act + ((int64_t)slot * chunks + c) * 4 * 64 * 8 + lane * 8, 64 * 8, token < a.tokens);
#pragma unroll
        for (int t = 0; t < N; ++t) {
            const uint8_t *tile = from + min(tile0 + t, a.down.tiles - 1) * a.down.tile_bytes;
            codes[t] = w4_codes(tile, c, lane);
            byte[t] = w4_scale(tile, chunks, c, lane);
        }
        if (c * kW4Chunk + q * 32 >= a.inner) {  // nothing was written there
#pragma unroll
            for (int s = 0; s < 4; ++s) x[s] = u32x4{0, 0, 0, 0};
        }
#pragma unroll
        for (int t = 0; t < N; ++t) {
            f32x4 d = {0, 0, 0, 0};
#pragma unroll
            for (int s = 0; s < 4; ++s) d = w4_product(w4_operand(codes[t], kv4_scale(byte[t]), s), x[s], d);
#pragma unroll
            for (int i = 0; i < 4; ++i) sum[t][i] += taken.w >> token & 1 ? weight * d[i] : 0.0f;
        }
    }
#pragma unroll
    for (int t = 0; t < N; ++t) {
        sum[t] = parts_sum(sum[t]);
        if (r < kColumns) part[wave][t][q][r] = sum[t];
    }
    __syncthreads();
    const int tile = tile0 + (int)threadIdx.x / (4 * kColumns), n = threadIdx.x / kColumns % 4, to_token = threadIdx.x % kColumns;
    if ((int)threadIdx.x >= N * 4 * kColumns || to_token >= a.tokens || tile >= a.down.tiles) return;
    f32x4 v = part[0][tile - tile0][n][to_token];
#pragma unroll
    for (int w = 1; w < kFewWaves; ++w) v += part[w][tile - tile0][n][to_token];
    typedef uint32_t u32x2_any __attribute__((ext_vector_type(2), aligned(2)));
    uint16_t *to = const_cast<uint16_t *>(a.out.p) + to_token * a.out.ts + tile * 16 + n * 4;  // hidden is a multiple of 32
    *reinterpret_cast<u32x2_any *>(to) = u32x2_any{bf16_pair(v[0], v[1]), bf16_pair(v[2], v[3])};
}

// More tokens, but few chunks of all groups: products and sums at once as well.  A
// wave has sums of its own of all tokens in LDS, to which it adds what a group's
// columns are.  (15 tokens x 736 through 8 experts of 224, 64 chunks, take 15.4 us in all,
// 18.8 with k_experts_down and k_experts_sum, 6 x 1568 through 8 of 1088 (90) 17.9 and
// 18.8, 20 x 2048 through 16 of 512 (128) 21.6 and 21.7, 13 x 2208 through 16 of 1088 (189)
// 28.0 and 25.0.  With more tiles than compute units it takes half as many: 6 x 7168 through
// 64 of 128 (64) 26.0 and 28.6, 8 x 5120 through 64 of 192 (96) 28.6 and 27.8.)
__global__ __launch_bounds__(64 * kFewWaves) void k_experts_down_all(DownArgs args) {
    const ExpertsArgs a(args);
    extern __shared__ f32x4 sums[];  // [waves][tokens][4, and one for the banks]
    const int lane = threadIdx.x % 64, r = lane % 16, q = lane / 16, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
    const int chunks = a.down.chunks, items = *a.used * chunks, size = a.tokens * 5;
    f32x4 *mine = sums + wave * size;
    for (int i = lane; i < size; i += 64) mine[i] = f32x4{0, 0, 0, 0};
    for (int item = wave; item < items; item += kFewWaves) {
        const int group = item / chunks, c = item - group * chunks;
        const uint8_t *tile = a.dn + __builtin_amdgcn_readfirstlane(a.taken[group].x) * a.down.bytes() + blockIdx.x * a.down.tile_bytes;
        const int pair = a.group_pair[group * kColumns + r % kColumns];  // below zero: no token's
        u32x4 x[4];
        load_few_inputs(x, a.act + ((int64_t)group * chunks + c) * 4 * 64 * 8 + lane * 8, 64 * 8, pair >= 0);
        const float weight = pair >= 0 ? a.weight[pair] : 0.0f;
        const u32x4 codes = w4_codes(tile, c, lane);
        const uint32_t byte = w4_scale(tile, chunks, c, lane);
        if (c * kW4Chunk + q * 32 >= a.inner) {  // nothing was written there
#pragma unroll
            for (int s = 0; s < 4; ++s) x[s] = u32x4{0, 0, 0, 0};
        }
        f32x4 d = {0, 0, 0, 0};
#pragma unroll
        for (int s = 0; s < 4; ++s) d = w4_product(w4_operand(codes, kv4_scale(byte), s), x[s], d);
        d = parts_sum(d);
        if (r < kColumns && pair >= 0) mine[pair / a.top_k * 5 + q] += weight * d;
    }
    __syncthreads();
    for (int i = threadIdx.x; i < a.tokens * 4; i += 64 * kFewWaves) {
        const int n = i % 4, token = i / 4;
        const f32x4 *p = sums + token * 5 + n;
        f32x4 v = p[0];
#pragma unroll
        for (int w = 1; w < kFewWaves; ++w) v += p[w * size];
        typedef uint32_t u32x2_any __attribute__((ext_vector_type(2), aligned(2)));
        uint16_t *to = const_cast<uint16_t *>(a.out.p) + token * a.out.ts + blockIdx.x * 16 + n * 4;  // hidden is a multiple of 32
        *reinterpret_cast<u32x2_any *>(to) = u32x2_any{bf16_pair(v[0], v[1]), bf16_pair(v[2], v[3])};
    }
}

// Four outputs of a token to a lane.
__global__ __launch_bounds__(kThreads) void k_experts_sum(DownArgs args) {
    const ExpertsArgs a(args);
    const int n = (blockIdx.x * kThreads + threadIdx.x) * 4, token = blockIdx.y;
    if (n >= a.hidden) return;
    const float *y = a.y + (int64_t)token * a.top_k * a.hidden + n;
    f32x4 v = {0, 0, 0, 0};
    for (int j = 0; j < a.top_k; ++j) v += a.weight[token * a.top_k + j] * *reinterpret_cast<const f32x4 *>(y + (int64_t)j * a.hidden);
    typedef uint32_t u32x2_any __attribute__((ext_vector_type(2), aligned(2)));
    uint16_t *to = const_cast<uint16_t *>(a.out.p) + token * a.out.ts + n;
    *reinterpret_cast<u32x2_any *>(to) = u32x2_any{bf16_pair(v[0], v[1]), bf16_pair(v[2], v[3])};
}

template <typename Args>
int launch3(const void *fn, dim3 grid, unsigned block, unsigned lds, Args a, void *stream) {
    void *args[] = {&a};
    return hipLaunchKernel(fn, grid, dim3(block), args, lds, static_cast<hipStream_t>(stream)) == hipSuccess ? AR_OK : AR_ELAUNCH;
}

// Groups of a pass, at most: one for every pair, and for every expert one that is
// not full.
int64_t most_groups(int64_t tokens, int experts, int top_k) {
    const int64_t pairs = (tokens < kTogether ? tokens : kTogether) * top_k, full = experts + pairs / kColumns;
    return pairs < full ? pairs : full;
}

template <int N>
const void *pick_down(bool two) {
    return two ? reinterpret_cast<const void *>(&k_experts_down<N, 2>) : reinterpret_cast<const void *>(&k_experts_down<N, 1>);
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
    return Places(most_groups(tokens, experts, top_k), down.chunks).y + pairs * hidden * 4;
}

int ar_w4_experts(ar_rows x, const void *router, const void *gate_up, const void *down, ar_rows out, void *choice, void *weight,
                  void *workspace, int64_t tokens, int64_t hidden, int64_t inner, int experts, int top_k, float scale, void *stream) {
    W4Shape up, dn;
    if (!valid_sizes(tokens, hidden, inner, experts, top_k, &up, &dn) || !(scale >= -3.0e38f && scale <= 3.0e38f)) return AR_EINVAL;
    if (tokens == 0) return AR_OK;
    const auto row_arg = [&](ar_rows r) { return RowsArg{ar_rows{r.p, tokens > 1 ? r.token_stride : 0, 0}, tokens, 1, (int)hidden}; };
    const RowsArg rx = row_arg(x), ro = row_arg(out);
    if (!rx.valid() || !ro.valid() || ro.self_overlap() || !router || !aligned_to(router, 2) || !gate_up || !aligned_to(gate_up, 16) ||
        !down || !aligned_to(down, 16) || !choice || !aligned_to(choice, 4) || !weight || !aligned_to(weight, 4) || !workspace ||
        !aligned_to(workspace, 16))
        return AR_EINVAL;
    const Span reads[] = {rx.span(), {addr(router), (uintptr_t)(2 * experts * hidden)}, {addr(gate_up), (uintptr_t)(experts * up.bytes())},
                          {addr(down), (uintptr_t)(experts * dn.bytes())}};
    const Span writes[] = {ro.span(), {addr(choice), (uintptr_t)(4 * tokens * top_k)}, {addr(weight), (uintptr_t)(4 * tokens * top_k)},
                           {addr(workspace), (uintptr_t)ar_w4_experts_workspace(tokens, hidden, inner, experts, top_k)}};
    for (int i = 0; i < 4; ++i) {
        for (int j = 0; j < 4; ++j)
            if ((j < i && overlap(writes[i], writes[j])) || (!(i == 0 && j == 0) && overlap(writes[i], reads[j]))) return AR_EALIAS;
    }
    if (ro.overlaps(rx)) return AR_EALIAS;
    const Rows xs = rows(rx), outs = rows(ro);
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    const int most = (int)most_groups(tokens, experts, top_k);
    for (int64_t at = 0; at < tokens; at += kTogether) {
        const int some = (int)(tokens - at < kTogether ? tokens - at : kTogether);
        int32_t *const choices = static_cast<int32_t *>(choice) + at * top_k;
        float *const weights = static_cast<float *>(weight) + at * top_k;
        const int slots = some * top_k < experts ? some * top_k : experts;
        // see k_experts_down_few, k_experts_down_all
        const bool few = some == 1 || (some <= kColumns && slots * dn.chunks <= kFewChunks);
        const bool all = some > kColumns && most_groups(some, experts, top_k) * dn.chunks <= (dn.tiles > kCus ? kFewChunks / 2 : kFewChunks);
        const Sizes sizes = Sizes::of(some, top_k, experts, few, all);
        RouteArgs r = {static_cast<const uint16_t *>(router), xs.p + at * xs.ts, xs.ts, reinterpret_cast<double *>(ws), choices, weights, (int)hidden, 0, scale,
                       sizes};
        const UpArgs u = {static_cast<const uint8_t *>(gate_up), r.x, xs.ts, choices, weights, ws, (int)hidden, (int)inner, most, sizes};
        const DownArgs d = {static_cast<const uint8_t *>(down), weights, const_cast<uint16_t *>(outs.p) + at * outs.ts, outs.ts, ws, (int)hidden, (int)inner,
                            most, sizes};
        int rc;
        // A small router's logits are made where the choice is: four tokens x 2048 through
        // 16 experts of 64 take 12.2 us in all, 13.7 with a launch for each; x 7392 through 8,
        // where it no longer does, would take 16.4 and take 16.6.
        if ((int64_t)experts * hidden <= kRouteAlone) {
            rc = launch3(reinterpret_cast<const void *>(&k_route), dim3(some), 64 * kRouteWaves, 0, r, stream);
            if (rc != AR_OK) return rc;
        } else {
            const int expert_tiles = (experts + 15) / 16, token_tiles = (some + 15) / 16, units = (int)hidden / 32;
            // 40 tokens x 7168 through 256 experts of 256: 135.4 us in all with 512, 137.5 with
            // 256, 147.1 with 128.
            r.splits = kRouterParts / (expert_tiles * token_tiles);
            if (r.splits > (units + kRouterWaves - 1) / kRouterWaves) r.splits = (units + kRouterWaves - 1) / kRouterWaves;
            if (r.splits < 1) r.splits = 1;
            rc = launch3(reinterpret_cast<const void *>(&k_router), dim3(expert_tiles, token_tiles, r.splits), 64 * kRouterWaves, 0, r, stream);
            if (rc != AR_OK) return rc;
            rc = launch3(reinterpret_cast<const void *>(&k_choose), dim3(some), 64 * kChooseWaves, 0, r, stream);
            if (rc != AR_OK) return rc;
        }
        const int half = (int)inner / 16;
        // Two tiles of each where that leaves the chip full, or where an expert has
        // several tokens, whose inputs weigh more than its weights.  (5 tokens x 7168, 256
        // experts of 256: 40.3 us in all with one, 42.3 with two; 8 x 5120, 128 of 768:
        // 88.2 and 83.3; 64 x 2048, 64 of 1408: 122.9 and 100.5.)
        const bool two_up = (int64_t)slots * half >= 1024 || some * top_k >= 8 * experts;
        // Where a wave has no more than one chunk, finding the expert weighs as much, and
        // two workgroups to a compute unit take tiles in turn.  They are counted by the
        // experts that tokens take which choose apart from each other, and 7% more, since
        // one workgroup too many is a whole turn more: 64 x 512 through 128 experts
        // of 1024 51.8 us in all, 68.2 with a workgroup to each; 64 x 5120 through 128 of
        // 768, with five chunks to a wave, took 9 us more in turn.
        int up_blocks = two_up ? (half + 1) / 2 : half;
        if (up.chunks <= kUpWaves && (int64_t)up_blocks * slots >= 4 * kCus) {
            const double used = fmin(slots, 1.07 * experts * (1.0 - pow(1.0 - (double)top_k / experts, some)));
            up_blocks = used < 2 * kCus ? (int)(2 * kCus / used) : 1;
        }
        rc = launch3(two_up ? reinterpret_cast<const void *>(&k_experts_up<2, 1>) : reinterpret_cast<const void *>(&k_experts_up<1, 2>),
                     dim3(up_blocks, slots), 64 * kUpWaves, 0, u, stream);
        if (rc != AR_OK) return rc;
        if (few) {
            // Two tiles where there are more than compute units: five tokens x 7168
            // through 256 experts of 256 take 40.3 us in all, 44.0 with one; five x 1568
            // through 8 of 1088 17.1 and 16.0.
            const int n = dn.tiles > kCus ? 2 : 1;
            rc = launch3(n == 2 ? reinterpret_cast<const void *>(&k_experts_down_few<2>) : reinterpret_cast<const void *>(&k_experts_down_few<1>),
                         dim3((dn.tiles + n - 1) / n), 64 * kFewWaves, 0, d, stream);
            if (rc != AR_OK) return rc;
            continue;
        }
        if (all) {
            rc = launch3(reinterpret_cast<const void *>(&k_experts_down_all), dim3(dn.tiles), 64 * kFewWaves, kFewWaves * some * 5 * 16, d, stream);
            if (rc != AR_OK) return rc;
            continue;
        }
        // Two tiles to a wave from some 32 to a compute unit on (16 tokens x 2048, 64
        // experts of 1024: 61.2 us in all, 62.1 with one; 12 x 4096, 8 of 1536: 35.5 and 34.1),
        // and two groups where experts have more than five tokens on average (64 x 2048,
        // 64 of 1408: 100.4, 109.3 with one; 12 x 4096, 8 of 1536: 34.1 and 35.2; 64 x 5120,
        // 128 of 768 and four experts to a token 156.5 and 148.9).
        const bool wide = (int64_t)slots * dn.tiles >= 8192;
        const bool two = some * top_k > 5 * experts;
        const int per = (wide ? 2 : 1) * kDownWaves;
        const int block = dn.chunks < kBlock / (two ? 2 : 1) ? dn.chunks : kBlock / (two ? 2 : 1);
        rc = launch3(wide ? pick_down<2>(two) : pick_down<1>(two), dim3((dn.tiles + per - 1) / per, slots),
                     64 * kDownWaves, block * (two ? 2 : 1) * 4096, d, stream);
        if (rc != AR_OK) return rc;
        rc = launch3(reinterpret_cast<const void *>(&k_experts_sum), dim3(((int)hidden + 4 * kThreads - 1) / (4 * kThreads), some), kThreads, 0, d, stream);
        if (rc != AR_OK) return rc;
    }
    return AR_OK;
}

}  // extern "C"
