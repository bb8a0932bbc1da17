// block_norm.hip -- from a block's partial sums to the next block's input: the
// ranks' parts added up, the norm after the block, its gate, the residual
// stream, and the norm before the next block, in one pass; and the gradient.
//
// For one token's row of `dim` channels, with parts y_r, stream x, gate g:
//     y = y_0 + y_1 + ...,  u = y / sqrt(mean(y^2) + eps) * post,
//     h = a x + g u,        z = h / sqrt(mean(h^2) + eps) * pre.
// Backwards, with n1 = y r1 and n2 = h r2 the rows that the norms make:
//     q = dz pre,  e = dh + r2 (q - n2 mean(q n2)),  dx = a e,  dg = e u,
//     p = e g post,  dy = r1 (p - n1 mean(p n1)),
//     dpost = sum of e g n1 over tokens,  dpre = sum of dz n2.
//
// Both are bound by memory: each row is read and written once, in binary32 between,
// but for gradients beyond 8192 channels, which read it once more for what tokens share
// (twice where dx or dy take its place).  A row lies in one workgroup, eight channels to a
// lane, or twice eight (beyond 6144 channels backwards, and forwards for up to four parts;
// always beyond 8192), so that both norms' sums are exchanges within it.
// Eight parts of 440 x 5120 take 9.7 to 10.0 us (5.0 TB/s), 8191 x 7169 with a gate for
// each token 124 us (4.7 TB/s), the gradient of 4096 x 7168 89.2 us (5.3 TB/s)
// and of 440 x 5120, whose three sums one after another are latency, 15.6 us.
#include "host.h"
#include "rows.h"
#include "wave.h"

namespace ar {
namespace {

constexpr int kMaxDim = 1 << 14;
constexpr int kMaxThreads = 1024;
// Tokens whose terms a lane adds up one after another in binary32, at most: their sum is
// off by 95 x 2^-24 of the terms.  (Of 2^22 equal terms 4096 one after another gave
// 2^-14.)
constexpr int kChain = 96;
// Above this many bytes, rows are read and written past the caches: 8191 tokens of
// 7168 take 87.8 us with it, 105 without.
constexpr int64_t kStreamBytes = (int64_t)128 << 20;

struct BlockArgs {
    const uint16_t *part[AR_MAX_P];
    Rows x, gate, h, z;      // h, z: outputs, or what comes in for them (backwards)
    Rows dx, dy, dgate;      // backwards only
    const uint16_t *post, *pre;
    float *sums[3];          // backwards: sums over a workgroup's tokens for the gate, the norm after, the norm before
                             // (null: none), 3 dim floats from a workgroup's to the next one's
    float *roots;            // backwards, beyond kSumDim: a token's r1, r2 and r2 mean(q n2)
    int64_t part_stride, tokens;
    int dim;
    int slots;               // backwards: places for sums, one or more of each workgroup
    int roots_only;          // backwards, beyond kSumDim: nothing but the roots is written
    float scale, eps;
};

template <bool NT>
__device__ __forceinline__ void store_vec8(uint16_t *p, const float (&f)[8]) {
    const u32x4 v = {bf16_pair(f[0], f[1]), bf16_pair(f[2], f[3]), bf16_pair(f[4], f[5]), bf16_pair(f[6], f[7])};
    u32x4_any *to = reinterpret_cast<u32x4_any *>(p);
    if (NT) __builtin_nontemporal_store(v, to);
    else *to = v;
}

// Sums over the workgroup of N values, in the same order each time; every lane
// gets them.  `part` is not used for another sum before the next barrier.
template <int N>
__device__ __forceinline__ void block_sum(float (&v)[N], float (&part)[N][kMaxThreads / 64]) {
#pragma unroll
    for (int n = 0; n < N; ++n) v[n] = wave_sum(v[n]);
    const int waves = blockDim.x / 64;
    if (waves == 1) return;
    if (threadIdx.x % 64 == 0) {
#pragma unroll
        for (int n = 0; n < N; ++n) part[n][threadIdx.x / 64] = v[n];
    }
    __syncthreads();
#pragma unroll
    for (int n = 0; n < N; ++n) {
        const float p = threadIdx.x % 16 < (unsigned)waves ? part[n][threadIdx.x % 16] : 0.0f;
        v[n] = row16_sum(p);
    }
}

// Where a lane's eight channels lie.  Past the row's last eight it takes those, and of
// them as its own what no lane before it has: no load stands behind a branch (with loads
// of single channels behind branches the gradient's registers ran over, and 7439 rows of
// 286 took 10.5 us forwards, 6.3 this way).  What it has of another lane's channels is
// masked, whatever that lane has written there meanwhile where a result takes a row's
// place.  Rows shorter than eight channels are one lane's, channel by channel.
template <bool SHORT>
struct Eight {
    int at, own;  // the first channel, and of the eight the first own one

    Eight() = default;
    __device__ __forceinline__ Eight(int first, int dim) {
        at = SHORT ? first : min(first, dim - 8);
        own = SHORT ? 0 : min(first - at, 8);
    }
    // Of the own ones.
    __device__ __forceinline__ u32x4 mask() const {
        u32x4 m;
#pragma unroll
        for (int i = 0; i < 4; ++i) m[i] = (2 * i >= own ? 0xFFFFu : 0) | (2 * i + 1 >= own ? 0xFFFF0000u : 0);
        return m;
    }
    template <bool NT>
    __device__ __forceinline__ u32x4 load(const uint16_t *row, int dim) const {
        return SHORT ? load_few(row + at, dim - at) : load_vec8<NT>(further(row, 2u * at));
    }
    template <bool NT>
    __device__ __forceinline__ void store(uint16_t *row, const float (&f)[8], int dim) const {
        if (!SHORT && own == 0) {
            store_vec8<NT>(further(row, 2u * at), f);
        } else {
#pragma unroll
            for (int c = 0; c < 8; ++c)
                if (c >= own && at + c < dim) row[at + c] = (uint16_t)bf16_pair(f[c], 0.0f);
        }
    }
};

// P parts; V times eight channels to a lane.
template <int P, int V, bool NT>
__global__ __launch_bounds__(kMaxThreads) void k_block_norm(BlockArgs a) {
    __shared__ float part1[1][kMaxThreads / 64], part2[1][kMaxThreads / 64];
    const int64_t token = blockIdx.x;
    const bool all = a.dim == V * 8 * (int)blockDim.x;  // every lane has eight of its own
    u32x4 y[V][P], x[V], g[V], w1[V], w2[V];
    Eight<false> at[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
        at[i] = Eight<false>((threadIdx.x + i * blockDim.x) * 8, a.dim);
        const u32x4 none = {0, 0, 0, 0};
#pragma unroll
        for (int p = 0; p < P; ++p) y[i][p] = at[i].template load<NT>(a.part[p] + token * a.part_stride, a.dim);
        x[i] = at[i].template load<NT>(a.x.p + token * a.x.ts, a.dim);
        g[i] = a.gate.p ? at[i].template load<false>(a.gate.p + token * a.gate.ts, a.dim) : none;
        w1[i] = a.post ? at[i].template load<false>(a.post, a.dim) : none;
        if (V == 1) w2[i] = a.pre ? at[i].template load<false>(a.pre, a.dim) : none;
    }
    if (!all) {  // zeros for channels that are another lane's: they add nothing to a sum
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const u32x4 mask = at[i].mask();
#pragma unroll
            for (int p = 0; p < P; ++p) y[i][p] &= mask;
            x[i] &= mask, g[i] &= mask, w1[i] &= mask;
        }
    }
    float f[V][8];
#pragma unroll
    for (int i = 0; i < V; ++i) {
        widen(y[i][0], f[i]);
#pragma unroll
        for (int p = 1; p < P; ++p) {
            float t[8];
            widen(y[i][p], t);
#pragma unroll
            for (int e = 0; e < 8; ++e) f[i][e] += t[e];
        }
    }
    const float by = 1.0f / a.dim;
    if (a.post) {
        float s[1] = {0};
#pragma unroll
        for (int i = 0; i < V; ++i)
#pragma unroll
            for (int e = 0; e < 8; ++e) s[0] += f[i][e] * f[i][e];
        block_sum(s, part1);
        const float r = rsqrtf(s[0] * by + a.eps);
#pragma unroll
        for (int i = 0; i < V; ++i) {
            float w[8];
            widen(w1[i], w);
#pragma unroll
            for (int e = 0; e < 8; ++e) f[i][e] = f[i][e] * r * w[e];
        }
    }
    float s[1] = {0};
#pragma unroll
    for (int i = 0; i < V; ++i) {
        float t[8], w[8];
        widen(x[i], t);
        widen(g[i], w);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            f[i][e] = a.scale * t[e] + (a.gate.p ? f[i][e] * w[e] : f[i][e]);
            s[0] += f[i][e] * f[i][e];
        }
        at[i].template store<NT>(const_cast<uint16_t *>(a.h.p) + token * a.h.ts, f[i], a.dim);
    }
    if (!a.pre) return;
    // Sixteen channels to a lane have this weight no earlier: with it 65 registers
    // left one row to a compute unit.
    if (V > 1) {
#pragma unroll
        for (int i = 0; i < V; ++i) w2[i] = at[i].template load<false>(a.pre, a.dim);
    }
    block_sum(s, part2);
    const float r = rsqrtf(s[0] * by + a.eps);
#pragma unroll
    for (int i = 0; i < V; ++i) {
        float w[8];
        widen(w2[i], w);
#pragma unroll
        for (int e = 0; e < 8; ++e) f[i][e] = f[i][e] * r * w[e];
        at[i].template store<NT>(const_cast<uint16_t *>(a.z.p) + token * a.z.ts, f[i], a.dim);
    }
}

// Rows shorter than eight channels: one to a lane.
__global__ __launch_bounds__(kThreads) void k_block_norm_short(BlockArgs a, int parts) {
    const int64_t token = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    if (token >= a.tokens) return;
    const auto at = [&](const uint16_t *row, int c) { return lo_f32(row[c]); };
    float f[7], s = 0;
#pragma unroll
    for (int c = 0; c < 7; ++c) {
        f[c] = 0;
        if (c >= a.dim) continue;
        for (int p = 0; p < parts; ++p) f[c] += at(a.part[p] + token * a.part_stride, c);
        s += f[c] * f[c];
    }
    const float r1 = a.post ? rsqrtf(s / a.dim + a.eps) : 1.0f;
    s = 0;
#pragma unroll
    for (int c = 0; c < 7; ++c) {
        if (c >= a.dim) continue;
        if (a.post) f[c] = f[c] * r1 * at(a.post, c);
        f[c] = a.scale * at(a.x.p + token * a.x.ts, c) + (a.gate.p ? f[c] * at(a.gate.p + token * a.gate.ts, c) : f[c]);
        s += f[c] * f[c];
    }
    const float r2 = a.pre ? rsqrtf(s / a.dim + a.eps) : 0.0f;
#pragma unroll
    for (int c = 0; c < 7; ++c) {
        if (c >= a.dim) continue;
        (const_cast<uint16_t *>(a.h.p) + token * a.h.ts)[c] = (uint16_t)bf16_pair(f[c], 0.0f);
        if (a.pre) (const_cast<uint16_t *>(a.z.p) + token * a.z.ts)[c] = (uint16_t)bf16_pair(f[c] * r2 * at(a.pre, c), 0.0f);
    }
}

// What a lane holds of one token's rows backwards.  What is not there is zeros, or
// ones for a gate, so that nothing asks for it again.
constexpr uint32_t kOnes = 0x3F803F80u;

template <bool NT, bool SHORT>
struct GradRow {
    u32x4 x, y, dh, dz, g;
    __device__ __forceinline__ void load(const BlockArgs &a, int64_t token, const Eight<SHORT> &at) {
        const u32x4 none = {0, 0, 0, 0}, ones = {kOnes, kOnes, kOnes, kOnes};
        y = at.template load<NT>(a.part[0] + token * a.part_stride, a.dim);
        x = at.template load<NT>(a.x.p + token * a.x.ts, a.dim);
        dh = a.h.p ? at.template load<NT>(a.h.p + token * a.h.ts, a.dim) : none;
        dz = a.pre ? at.template load<NT>(a.z.p + token * a.z.ts, a.dim) : none;
        g = a.gate.p ? at.template load<false>(a.gate.p + token * a.gate.ts, a.dim) : ones;
    }
    // Zeros for channels that are another lane's: they add nothing to a sum.  (The gate's
    // too, and the weights': an infinity there times 0 would be NaN.)
    __device__ __forceinline__ GradRow own(const Eight<SHORT> &at, bool all) const {
        if (SHORT || all) return *this;
        const u32x4 mask = at.mask();
        return GradRow{x & mask, y & mask, dh & mask, dz & mask, g & mask};
    }
};

typedef float f32x4_any __attribute__((ext_vector_type(4), aligned(4)));

__device__ __forceinline__ void store_floats(float *to, const float (&f)[8]) {
    f32x4_any *v = reinterpret_cast<f32x4_any *>(to);
    v[0] = f32x4_any{f[0], f[1], f[2], f[3]};
    v[1] = f32x4_any{f[4], f[5], f[6], f[7]};
}

// A lane's sums into a slot.
template <bool SHORT>
__device__ __forceinline__ void store_sums(const BlockArgs &a, int64_t slot, const Eight<SHORT> &at, const float (&sg)[8], const float (&s1)[8],
                                           const float (&s2)[8]) {
    const int64_t to = slot * 3 * a.dim + at.at;
    if (!SHORT && at.own == 0) {
        if (a.sums[0]) store_floats(a.sums[0] + to, sg);
        if (a.sums[1]) store_floats(a.sums[1] + to, s1);
        if (a.sums[2]) store_floats(a.sums[2] + to, s2);
        return;
    }
#pragma unroll
    for (int c = 0; c < 8; ++c)
        if (c >= at.own && at.at + c < a.dim) {
            if (a.sums[0]) a.sums[0][to + c] = sg[c];
            if (a.sums[1]) a.sums[1][to + c] = s1[c];
            if (a.sums[2]) a.sums[2][to + c] = s2[c];
        }
}

// Backwards.  Without a norm after the block its weight and root are 1 and what its
// mean takes off is 0; without one before the next block the root is 0.  The rows that
// those factors would meet are put to 0 there: an infinity times 0 is NaN.
//
// SUMS: a workgroup takes tokens in turn, the next one's rows on their way while it
// works on one, and each lane keeps its channels' sums over them; a second launch adds
// the workgroups' up.  CHAINS: over kChain of its tokens at a time (440 tokens of 5120
// take 16.4 us so, 15.6 without).  For longer rows there are not registers enough for the
// sums: a workgroup to a token leaves its roots, and k_block_norm_columns makes the
// sums from the rows again.
// T: lanes, at most.
template <int V, int T, bool NT, bool SUMS, bool CHAINS, bool SHORT>
__global__ __launch_bounds__(T) void k_block_norm_grad(BlockArgs a) {
    __shared__ float part1[1][kMaxThreads / 64], part2[2][kMaxThreads / 64], part3[1][kMaxThreads / 64];
    const float by = 1.0f / a.dim;
    const bool all = a.dim == V * 8 * (int)blockDim.x;  // every lane has eight of its own
    constexpr int kSums = SUMS ? V : 1;
    float sg[kSums][8] = {}, s1[kSums][8] = {}, s2[kSums][8] = {};
    u32x4 w1[V], w2[V];
    Eight<SHORT> at[V];
    // Sixteen channels to a lane leave no room for rows in binary32 from one sum to
    // the next, and 1024 lanes (128 registers each) none for the weights, which the
    // caches hold.
    constexpr bool kLean = V > 1, kHeld = T < 1024;
    const auto weights = [&](int i) {
        w1[i] = a.post ? at[i].template load<false>(a.post, a.dim) : u32x4{kOnes, kOnes, kOnes, kOnes};
        w2[i] = a.pre ? at[i].template load<false>(a.pre, a.dim) : u32x4{0, 0, 0, 0};
        if (!SHORT && !all) w1[i] &= at[i].mask(), w2[i] &= at[i].mask();
    };
#pragma unroll
    for (int i = 0; i < V; ++i) {
        at[i] = Eight<SHORT>((threadIdx.x + i * blockDim.x) * 8, a.dim);
        if (kHeld) weights(i);
    }
    constexpr bool kAhead = SUMS;
    GradRow<NT, SHORT> next[V];
    if (kAhead) {
#pragma unroll
        for (int i = 0; i < V; ++i) next[i].load(a, blockIdx.x, at[i]);
    }
    int slot = blockIdx.x, chain = 0;
    const auto leave_sums = [&] {
#pragma unroll
        for (int i = 0; i < V; ++i) {
            store_sums(a, slot, at[i], sg[i % kSums], s1[i % kSums], s2[i % kSums]);
#pragma unroll
            for (int c = 0; c < 8; ++c) sg[i % kSums][c] = s1[i % kSums][c] = s2[i % kSums][c] = 0.0f;
        }
        slot += gridDim.x;
    };
    for (int64_t token = blockIdx.x; token < a.tokens; token += gridDim.x) {
        if (CHAINS && chain++ == kChain) leave_sums(), chain = 1;
        GradRow<NT, SHORT> row[V];
#pragma unroll
        for (int i = 0; i < V; ++i) {
            if (!kAhead) next[i].load(a, token, at[i]);
            row[i] = next[i].own(at[i], all);
            if (!kHeld) weights(i);
        }
        if (kAhead && token + gridDim.x < a.tokens) {
#pragma unroll
            for (int i = 0; i < V; ++i) next[i].load(a, token + gridDim.x, at[i]);
        }
        float r1 = 1.0f;
        if (a.post) {
            float s[1] = {0};
#pragma unroll
            for (int i = 0; i < V; ++i)
#pragma unroll
                for (int c = 0; c < 8; ++c) s[0] += at8(row[i].y, c) * at8(row[i].y, c);
            block_sum(s, part1);
            r1 = rsqrtf(s[0] * by + a.eps);
        }
        float h[V][8];
        float s[2] = {0, 0};
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const u32x4 y = kLean ? again(row[i].y) : row[i].y, u1 = kLean ? again(w1[i]) : w1[i], u2 = kLean ? again(w2[i]) : w2[i];
#pragma unroll
            for (int c = 0; c < 8; ++c) {
                h[i][c] = a.scale * at8(row[i].x, c) + at8(row[i].g, c) * (at8(y, c) * r1 * at8(u1, c));
                s[0] += h[i][c] * h[i][c];
                s[1] += at8(row[i].dz, c) * at8(u2, c) * h[i][c];
            }
        }
        float r2 = 0.0f, along2 = 0.0f;
        if (a.pre) {
            block_sum(s, part2);
            r2 = rsqrtf(s[0] * by + a.eps);
            along2 = s[1] * by * r2;
        } else {
#pragma unroll
            for (int i = 0; i < V; ++i)
#pragma unroll
                for (int c = 0; c < 8; ++c) h[i][c] = 0.0f;
        }
        if (!SUMS && threadIdx.x == 0) a.roots[token * 3] = r1, a.roots[token * 3 + 1] = r2, a.roots[token * 3 + 2] = along2;
        if (!SUMS && a.roots_only) {
            __syncthreads();
            continue;
        }
        float d[1] = {0};
        float(&e)[V][8] = h;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            float t[8];
            const u32x4 z = kLean ? again(row[i].dz) : row[i].dz, u2 = kLean ? again(w2[i]) : w2[i];
#pragma unroll
            for (int c = 0; c < 8; ++c) {
                const float n2 = h[i][c] * r2;
                if (SUMS) s2[i % kSums][c] += at8(z, c) * n2;
                e[i][c] = at8(row[i].dh, c) + r2 * (at8(z, c) * at8(u2, c) - n2 * along2);
                t[c] = a.scale * e[i][c];
            }
            at[i].template store<NT>(const_cast<uint16_t *>(a.dx.p) + token * a.dx.ts, t, a.dim);
            const u32x4 y = kLean ? again(row[i].y) : row[i].y, g = kLean ? again(row[i].g) : row[i].g, u1 = kLean ? again(w1[i]) : w1[i];
#pragma unroll
            for (int c = 0; c < 8; ++c) t[c] = e[i][c] * (at8(y, c) * r1 * at8(u1, c));
            if (a.dgate.p) at[i].template store<NT>(const_cast<uint16_t *>(a.dgate.p) + token * a.dgate.ts, t, a.dim);
#pragma unroll
            for (int c = 0; c < 8; ++c) {
                if (SUMS) sg[i % kSums][c] += t[c];
                e[i][c] *= at8(g, c);
                if (SUMS) s1[i % kSums][c] += e[i][c] * (at8(y, c) * r1);
                e[i][c] *= at8(u1, c);
                d[0] += e[i][c] * at8(y, c);
            }
        }
        float along1 = 0.0f;
        if (a.post) {
            block_sum(d, part3);
            along1 = d[0] * by * r1 * r1;
        } else {
#pragma unroll
            for (int i = 0; i < V; ++i) row[i].y = u32x4{0, 0, 0, 0};
        }
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const u32x4 y = kLean ? again(row[i].y) : row[i].y;
#pragma unroll
            for (int c = 0; c < 8; ++c) e[i][c] = r1 * (e[i][c] - at8(y, c) * along1);
            at[i].template store<NT>(const_cast<uint16_t *>(a.dy.p) + token * a.dy.ts, e[i], a.dim);
        }
        // Each sum's part is written again after the barrier of another one.
        // Where there is one sum alone, after this one.
        if (!a.post) __syncthreads();
    }
    if (SUMS) leave_sums();
    while (CHAINS && slot < a.slots) leave_sums();  // zeros, where other workgroups had one token more
}

// The sums over tokens from the rows and each token's roots: a wave has 512
// channels, and the waves of a workgroup take its tokens in turn.
__global__ __launch_bounds__(kThreads) void k_block_norm_columns(BlockArgs a) {
    constexpr int kWaves = kThreads / 64;
    __shared__ float part[kWaves][3][512];
    const int lane = threadIdx.x % 64, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64), lane8 = (blockIdx.x * 64 + lane) * 8;
    const Eight<false> at(lane8, a.dim);
    float sg[8] = {}, s1[8] = {}, s2[8] = {}, w1[8], w2[8];
    widen(a.post ? at.load<false>(a.post, a.dim) : u32x4{kOnes, kOnes, kOnes, kOnes}, w1);
    widen(a.pre ? at.load<false>(a.pre, a.dim) : u32x4{0, 0, 0, 0}, w2);
    const int64_t begin = a.tokens * blockIdx.y / gridDim.y, end = a.tokens * (blockIdx.y + 1) / gridDim.y;
    for (int64_t token = begin + wave; token < end; token += kWaves) {
        GradRow<false, false> row;
        row.load(a, token, at);
        row = row.own(at, a.dim % 512 == 0);
        const float r1 = a.roots[token * 3], r2 = a.roots[token * 3 + 1], along2 = a.roots[token * 3 + 2];
        float y[8], x[8], dh[8], q[8], g[8];
        widen(row.y, y);
        widen(row.x, x);
        widen(row.dh, dh);
        widen(row.dz, q);
        widen(row.g, g);
#pragma unroll
        for (int c = 0; c < 8; ++c) {
            const float n1 = y[c] * r1, u = n1 * w1[c], n2 = a.pre ? (a.scale * x[c] + g[c] * u) * r2 : 0.0f;
            const float e = dh[c] + r2 * (q[c] * w2[c] - n2 * along2);
            sg[c] += e * u;
            s1[c] += e * g[c] * n1;
            s2[c] += q[c] * n2;
        }
    }
#pragma unroll
    for (int c = 0; c < 8; ++c) part[wave][0][c * 64 + lane] = sg[c], part[wave][1][c * 64 + lane] = s1[c], part[wave][2][c * 64 + lane] = s2[c];
    __syncthreads();
    if (wave) return;
#pragma unroll
    for (int c = 0; c < 8; ++c) {
        sg[c] = (part[0][0][c * 64 + lane] + part[1][0][c * 64 + lane]) + (part[2][0][c * 64 + lane] + part[3][0][c * 64 + lane]);
        s1[c] = (part[0][1][c * 64 + lane] + part[1][1][c * 64 + lane]) + (part[2][1][c * 64 + lane] + part[3][1][c * 64 + lane]);
        s2[c] = (part[0][2][c * 64 + lane] + part[1][2][c * 64 + lane]) + (part[2][2][c * 64 + lane] + part[3][2][c * 64 + lane]);
    }
    store_sums(a, blockIdx.y, at, sg, s1, s2);
}

struct SumArgs {
    const float *slots;
    float *out[3];  // of the gate, the norm after, the norm before; null: not wanted
    int dim, blocks;
};

// Adds the workgroups' sums up: 64 columns to a workgroup, its 16 waves taking every
// sixteenth slot.  Sixteen slots, and the waves, are added up in binary32, and in 64
// bits what grows with the tokens.
constexpr int kSumWaves = 16;

__global__ __launch_bounds__(64 * kSumWaves) void k_block_norm_sums(SumArgs a) {
    __shared__ float part[kSumWaves][64];
    const int per = (a.dim + 63) / 64, which = blockIdx.x / per, lane = threadIdx.x % 64, wave = threadIdx.x / 64;
    const int c = blockIdx.x % per * 64 + lane;
    float *out = a.out[which];
    if (!out) return;
    float t = 0;
    double all = 0;
    if (c < a.dim) {
        const float *p = a.slots + (int64_t)which * a.dim + c;
        for (int s = wave; s < a.blocks; s += kSumWaves * 16) {
            float v[16];  // all on their way at once
#pragma unroll
            for (int k = 0; k < 16; ++k) v[k] = p[(int64_t)min(s + kSumWaves * k, a.blocks - 1) * 3 * a.dim];
            float some = 0;
#pragma unroll
            for (int k = 0; k < 16; ++k) some += s + kSumWaves * k < a.blocks ? v[k] : 0.0f;
            all += some;
        }
    }
    part[wave][lane] = t = (float)all;
    __syncthreads();
    if (wave || c >= a.dim) return;
#pragma unroll
    for (int w = 1; w < kSumWaves; ++w) t += part[w][lane];
    out[c] = t;
}

template <int P>
const void *pick_parts(bool wide, bool stream) {
    return wide ? (stream ? reinterpret_cast<const void *>(&k_block_norm<P, 2, true>) : reinterpret_cast<const void *>(&k_block_norm<P, 2, false>))
                : (stream ? reinterpret_cast<const void *>(&k_block_norm<P, 1, true>) : reinterpret_cast<const void *>(&k_block_norm<P, 1, false>));
}

const void *pick(int P, bool wide, bool stream) {
    switch (P) {
        case 1: return pick_parts<1>(wide, stream);
        case 2: return pick_parts<2>(wide, stream);
        case 3: return pick_parts<3>(wide, stream);
        case 4: return pick_parts<4>(wide, stream);
        case 5: return pick_parts<5>(wide, stream);
        case 6: return pick_parts<6>(wide, stream);
        case 7: return pick_parts<7>(wide, stream);
        default: return pick_parts<8>(wide, stream);
    }
}

// Eight channels to a lane up to 6144, sixteen beyond that.  (8192 tokens of 5120 take
// 99 us with eight and 110 with sixteen; 4096 of 7168, whose 896 lanes with eight
// would have 128 registers each, 79 us with sixteen and 94 with eight.)
constexpr int kSumDim = 8 * kMaxThreads;

// Rows beyond kSumDim are read again by k_block_norm_columns: they stay in the caches.
template <bool NT, bool CHAINS>
const void *pick_sums(int dim) {
    return dim < 8       ? reinterpret_cast<const void *>(&k_block_norm_grad<1, 64, false, true, CHAINS, true>)
           : dim <= 6144 ? reinterpret_cast<const void *>(&k_block_norm_grad<1, 768, NT, true, CHAINS, false>)
                         : reinterpret_cast<const void *>(&k_block_norm_grad<2, 512, NT, true, CHAINS, false>);
}

const void *pick_grad(int dim, bool stream, bool chains) {
    return dim > kSumDim ? reinterpret_cast<const void *>(&k_block_norm_grad<2, 1024, false, false, false, false>)
           : stream      ? (chains ? pick_sums<true, true>(dim) : pick_sums<true, false>(dim))
                         : (chains ? pick_sums<false, true>(dim) : pick_sums<false, false>(dim));
}

// Sixteen channels to a lane: rows of more than 8192, and of more than 6144 and up to
// four parts.  (8191 tokens of 7169: 106 us, 116 with eight; 3000 of 7168 and four parts
// 53.5 and 54.9; 1000 of 8192 and two 13.7 and 15.0.  2100 of 8191 and eight parts 89.2,
// 87.3 with eight; 8200 of 4104 53.2 and 50.3; 440 of 5120 and eight parts 10.2 and 9.8.)
bool is_wide(int dim, int P) { return dim > 8 * kMaxThreads || (dim > 6144 && P <= 4); }

unsigned threads_of(int dim, bool wide) {
    const int vecs = (dim + 7) / 8, lanes = wide ? (vecs + 1) / 2 : vecs;
    return (unsigned)round_up(lanes, 64);
}

bool valid_shape(int64_t tokens, int dim) { return tokens >= 0 && tokens <= (int64_t)1 << 28 && dim >= 1 && dim <= kMaxDim; }

bool valid_numbers(float scale, float eps) { return scale >= -3.0e38f && scale <= 3.0e38f && eps >= 0 && eps <= 3.0e38f; }

// The rows of a call, with a weight's bytes where there is one.
struct Buffers {
    RowsArg rows[8];
    int count = 0;
    Span small[3];
    int smalls = 0;

    void add(const RowsArg &r) { rows[count++] = r; }
    void weight(const void *p, int dim) {
        if (p) small[smalls++] = Span{addr(p), (uintptr_t)(2 * dim)};
    }
};

RowsArg row_arg(ar_rows r, int64_t tokens, int dim) {
    r.head_stride = 0;
    if (tokens <= 1) r.token_stride = 0;
    return RowsArg{r, tokens, 1, dim};
}

// Outputs: apart from each other and from all that is read, but for an output
// that is exactly one of the rows read and allowed to be.
int check_output(const RowsArg &out, const Buffers &in, unsigned may_be) {
    if (!out.valid() || out.self_overlap()) return AR_EINVAL;
    for (int i = 0; i < in.smalls; ++i)
        if (overlap(out.span(), in.small[i])) return AR_EALIAS;
    for (int i = 0; i < in.count; ++i)
        if (!((may_be >> i & 1) && out.same(in.rows[i])) && out.overlaps(in.rows[i])) return AR_EALIAS;
    return AR_OK;
}

bool half_aligned(const void *p) { return aligned_to(p, 2); }

int lanes_of_grad(int dim) {
    const int each = dim <= 6144 ? 8 : 16;
    return (int)round_up((dim + each - 1) / each, 64);
}

// Workgroups whose rows of sums the workspace has room for.  Its size never falls as
// tokens or channels grow: 2^20 channels of rows, or 256 rows, or one for each token; and
// beyond 256 chains a row for each chain more.
int64_t slot_rows(int64_t tokens, int dim) {
    const int64_t rows = (1 << 20) / dim > 256 ? (1 << 20) / dim : 256;
    return tokens < 1 ? 1 : tokens < rows ? tokens : rows;
}

int64_t slot_channels(int64_t tokens, int dim) {
    const int64_t all = (tokens < 1 ? 1 : tokens) * dim, most = (int64_t)256 * dim > 1 << 20 ? (int64_t)256 * dim : 1 << 20;
    return (all < most ? all : most) + (tokens > 256 * kChain ? tokens / kChain * dim : 0);
}

// Workgroups with sums of their own: one to each of 256 compute units, or for short
// rows as many as leave eight waves to each and four tokens to a workgroup (4096
// tokens of 1024 take 28.8 us with 256, 20.7 with 1024; 440 take 9.9 with 256, 11.4
// with one each, whose sums take longer to join).
//
// A few tokens' sums stay in one workgroup and are the gradients, without a launch to
// join them: one token of 5120 takes 5.7 us (8.2), two 7.9 (8.2), but two of 8192 10.5
// (10.2); 32 of 16384, whose rows are read again, 14.7 (20.8), 64 17.9 (18.6).
int sum_groups(int64_t tokens, int dim) {
    if (tokens <= (dim > kSumDim ? 32 : dim <= 6144 ? 2 : 1)) return 1;
    const int waves = lanes_of_grad(dim) / 64;
    int64_t most = dim > kSumDim ? 32 : dim > 4096 ? 256 : waves <= 2 ? 1024 : 2048 / waves;
    if (most > 256 && most > tokens / 4) most = tokens / 4 > 256 ? tokens / 4 : 256;
    if (most > slot_rows(tokens, dim)) most = slot_rows(tokens, dim);
    if (tokens <= most) return (int)tokens;
    const int64_t each = (tokens + most - 1) / most;  // of the workgroup with most: no more workgroups than that needs
    return (int)((tokens + each - 1) / each);
}

// Their rows of sums.  Beyond kSumDim a workgroup's four waves have a chain each.
int64_t sum_slots(int64_t tokens, int dim) {
    const int64_t groups = sum_groups(tokens, dim);
    if (dim > kSumDim) {
        const int64_t chains = (tokens + 4 * kChain - 1) / (4 * kChain);
        return chains > 65535 ? 65535 : chains > groups ? chains : groups;  // a launch has no more
    }
    const int64_t each = (tokens + groups - 1) / groups;
    return groups * ((each + kChain - 1) / kChain);
}

}  // namespace
}  // namespace ar

using namespace ar;

extern "C" {

int ar_block_norm(ar_ptrs parts, int64_t part_stride, int P, ar_rows x, const void *post_weight, ar_rows gate,
                  const void *pre_weight, ar_rows h, ar_rows z, int64_t tokens, int dim, float residual_scale, float eps,
                  void *stream) {
    if (!valid_shape(tokens, dim) || !valid_numbers(residual_scale, eps) || P < 1 || P > AR_MAX_P) return AR_EINVAL;
    if (tokens == 0) return AR_OK;
    if (tokens >= 1 << 21) return AR_EINVAL;  // a workgroup each, of up to 1024 lanes
    if (!half_aligned(post_weight) || !half_aligned(pre_weight)) return AR_EINVAL;
    Buffers in;
    const RowsArg rx = row_arg(x, tokens, dim);
    in.weight(post_weight, dim);
    in.weight(pre_weight, dim);
    // a gate that all tokens share is one row
    const RowsArg rg = row_arg(gate, gate.token_stride ? tokens : 1, dim);
    if (!rx.valid() || (gate.p && !rg.valid())) return AR_EINVAL;
    in.add(rx);
    if (gate.p) in.add(rg);
    BlockArgs a = {};
    for (int p = 0; p < P; ++p) {
        const RowsArg r = row_arg(ar_rows{parts.p[p], part_stride, 0}, tokens, dim);
        if (!r.valid()) return AR_EINVAL;
        a.part[p] = static_cast<const uint16_t *>(parts.p[p]);
        a.part_stride = r.r.token_stride;
    }
    const RowsArg rh = row_arg(h, tokens, dim), rz = row_arg(z, tokens, dim);
    const RowsArg *outs[] = {&rh, &rz};
    for (int o = 0; o < (pre_weight ? 2 : 1); ++o) {
        if (const int rc = check_output(*outs[o], in, o == 0)) return rc;
        for (int p = 0; p < P; ++p)
            if (outs[o]->overlaps(row_arg(ar_rows{parts.p[p], part_stride, 0}, tokens, dim))) return AR_EALIAS;
    }
    if (pre_weight && rh.overlaps(rz)) return AR_EALIAS;
    a.x = rows(rx), a.h = rows(rh);
    if (gate.p) a.gate = rows(rg);
    if (pre_weight) a.z = rows(rz);
    a.post = static_cast<const uint16_t *>(post_weight), a.pre = static_cast<const uint16_t *>(pre_weight);
    a.tokens = tokens, a.dim = dim, a.scale = residual_scale, a.eps = eps;
    if (dim < 8) {
        void *args[] = {&a, &P};
        return hipLaunchKernel(reinterpret_cast<const void *>(&k_block_norm_short), dim3((unsigned)((tokens + kThreads - 1) / kThreads)), dim3(kThreads), args, 0,
                               static_cast<hipStream_t>(stream)) == hipSuccess
                   ? AR_OK
                   : AR_ELAUNCH;
    }
    const int64_t bytes = 2 * tokens * dim * (P + 3);
    const bool past = bytes > kStreamBytes, wide = is_wide(dim, P);
    return launch(pick(P, wide, past), (unsigned)tokens, threads_of(dim, wide), a, stream);
}

int64_t ar_block_norm_bwd_workspace(int64_t tokens, int dim) {
    if (!valid_shape(tokens, dim)) return AR_EINVAL;
    return round_up(slot_channels(tokens, dim) * 12, 16) + (dim > kSumDim ? round_up(tokens * 12, 16) : 0);
}

int ar_block_norm_bwd(ar_rows h_grad, ar_rows z_grad, ar_rows y, ar_rows x, const void *post_weight, ar_rows gate,
                      const void *pre_weight, ar_rows dx, ar_rows dy, ar_rows gate_grad, void *post_grad, void *pre_grad,
                      void *workspace, int64_t tokens, int dim, float residual_scale, float eps, void *stream) {
    if (!valid_shape(tokens, dim) || !valid_numbers(residual_scale, eps)) return AR_EINVAL;
    const bool shared = gate.p && gate.token_stride == 0;
    void *sums[3] = {shared ? gate_grad.p : nullptr, post_weight ? post_grad : nullptr, pre_weight ? pre_grad : nullptr};
    const bool wanted = sums[0] || sums[1] || sums[2];
    if (!workspace || !aligned_to(workspace, 16) || !half_aligned(post_weight) || !half_aligned(pre_weight)) return AR_EINVAL;
    Span apart[4] = {{addr(workspace), (uintptr_t)ar_block_norm_bwd_workspace(tokens, dim)}};
    int aparts = 1;
    for (void *p : sums) {
        if (!aligned_to(p, 4)) return AR_EINVAL;
        if (p) apart[aparts++] = Span{addr(p), (uintptr_t)(4 * dim)};
    }
    Buffers in;
    const RowsArg rx = row_arg(x, tokens, dim), ry = row_arg(y, tokens, dim), rdh = row_arg(h_grad, tokens, dim),
                  rdz = row_arg(z_grad, tokens, dim), rg = row_arg(gate, shared ? 1 : tokens, dim);
    const RowsArg rdx = row_arg(dx, tokens, dim), rdy = row_arg(dy, tokens, dim), rdg = row_arg(gate_grad, tokens, dim);
    in.weight(post_weight, dim);
    in.weight(pre_weight, dim);
    const bool gate_rows = gate.p && !shared && gate_grad.p;
    if (tokens > 0) {
        in.add(rx), in.add(ry);
        if (h_grad.p) in.add(rdh);
        if (pre_weight) in.add(rdz);
        const unsigned rows_read = (1u << in.count) - 1;
        if (gate.p) in.add(rg);
        for (int i = 0; i < in.count; ++i)
            if (!in.rows[i].valid()) return AR_EINVAL;
        if (const int rc = check_output(rdx, in, rows_read)) return rc;
        if (const int rc = check_output(rdy, in, rows_read)) return rc;
        if (rdx.overlaps(rdy)) return AR_EALIAS;
        if (gate_rows) {
            if (const int rc = check_output(rdg, in, 0)) return rc;
            if (rdg.overlaps(rdx) || rdg.overlaps(rdy)) return AR_EALIAS;
        }
    }
    for (int i = 0; i < aparts; ++i) {
        for (int j = 0; j < i; ++j)
            if (overlap(apart[i], apart[j])) return AR_EALIAS;
        for (int j = 0; j < in.smalls; ++j)
            if (overlap(apart[i], in.small[j])) return AR_EALIAS;
        for (int j = 0; j < in.count; ++j)
            if (overlap(apart[i], in.rows[j].span())) return AR_EALIAS;
        if (tokens > 0 && (overlap(apart[i], rdx.span()) || overlap(apart[i], rdy.span()) ||
                           (gate_rows && overlap(apart[i], rdg.span()))))
            return AR_EALIAS;
    }
    const int64_t slots = tokens ? sum_slots(tokens, dim) : 0;
    SumArgs sum = {static_cast<const float *>(workspace),
                   {static_cast<float *>(sums[0]), static_cast<float *>(sums[1]), static_cast<float *>(sums[2])},
                   dim,
                   (int)slots};
    if (tokens > 0) {
        BlockArgs a = {};
        a.part[0] = static_cast<const uint16_t *>(y.p), a.part_stride = ry.r.token_stride;
        a.x = rows(rx), a.dx = rows(rdx), a.dy = rows(rdy);
        if (h_grad.p) a.h = rows(rdh);
        if (pre_weight) a.z = rows(rdz);
        if (gate.p) a.gate = rows(rg);
        if (gate_rows) a.dgate = rows(rdg);
        a.post = static_cast<const uint16_t *>(post_weight), a.pre = static_cast<const uint16_t *>(pre_weight);
        // a single workgroup's sums are the gradients
        float *const ws = static_cast<float *>(workspace);
        for (int i = 0; i < 3; ++i) a.sums[i] = !sums[i] ? nullptr : slots == 1 ? static_cast<float *>(sums[i]) : ws + i * dim;
        a.roots = ws + slots * 3 * dim;
        a.slots = (int)slots;
        a.tokens = tokens, a.dim = dim, a.scale = residual_scale, a.eps = eps;
        const bool own = dim <= kSumDim;
        const unsigned blocks = own ? sum_groups(tokens, dim) : tokens < 512 ? tokens : 512, lanes = lanes_of_grad(dim);
        const void *fn = pick_grad(dim, 2 * tokens * dim * 6 > kStreamBytes, slots > blocks);
        const auto columns = [&] {
            void *args[] = {&a};
            return hipLaunchKernel(reinterpret_cast<const void *>(&k_block_norm_columns), dim3((dim + 511) / 512, (unsigned)slots), dim3(kThreads), args, 0,
                                   static_cast<hipStream_t>(stream)) == hipSuccess
                       ? AR_OK
                       : AR_ELAUNCH;
        };
        // k_block_norm_columns needs the rows as they came in: where dx or dy take
        // one's place it goes before them, with roots from a pass of their own.
        bool before = false;
        for (int i = 0; !own && wanted && i < in.count; ++i) before = before || rdx.overlaps(in.rows[i]) || rdy.overlaps(in.rows[i]);
        int rc = AR_OK;
        if (before) {
            a.roots_only = 1;
            rc = launch(fn, blocks, lanes, a, stream);
            a.roots_only = 0;
            if (rc == AR_OK) rc = columns();
        }
        if (rc == AR_OK) rc = launch(fn, blocks, lanes, a, stream);
        if (rc == AR_OK && !own && wanted && !before) rc = columns();
        if (rc != AR_OK) return rc;
    }
    if (!wanted || (tokens > 0 && slots == 1)) return AR_OK;
    return launch(reinterpret_cast<const void *>(&k_block_norm_sums), (unsigned)(3 * ((dim + 63) / 64)), 64 * kSumWaves, sum, stream);
}

}  // extern "C"
