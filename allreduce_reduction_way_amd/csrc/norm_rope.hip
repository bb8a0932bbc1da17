// norm_rope.hip -- norms of queries and keys for each head with the position
// rotation in the same pass, and its gradient.
//
// For one row x of D channels (a token's head), weight w, and the token's
// cosines and sines:
//     r = 1 / sqrt(mean(x^2) + eps),   z = x r w,
//     y_a = z_a cos - z_b sin,  y_b = z_b cos + z_a sin   on each pair (a, b),
// and y = z on the channels that do not turn.  Backwards, with g the rotation
// of the incoming gradient by the opposite angle, n = x r and h = g w:
//     dx = r (h - n mean(h n)),   dw = sum over tokens and heads of g n.
//
// Both are bound by memory: 4 bytes (6 backwards) per element against some ten
// (twenty) operations.  A row lies in D/8 lanes of one wave, 16 bytes each, so
// a wave works on 512/D rows at once, the sums over a row are exchanges
// between its lanes, and the two channels of a pair are either in one lane
// (pairs side by side) or in two lanes of the row, which exchange the packed
// bf16 words (half the exchanges of the widened values).  The heads of one
// token share the wave's cosines and sines, so a wave stays on one token and
// takes several steps of rows.
#include "host.h"
#include "join.h"
#include "rows.h"

namespace ar {
namespace {

constexpr int kMaxHeads = 1 << 16;
constexpr int kSteps = 4;      // steps of rows that a wave has in flight, forward
constexpr int kGradSteps = 2;  // the same backwards (two loads a row)

struct NormArgs {
    Rows q, k, gq, gk, oq, ok;  // gq, gk: incoming gradients (backwards only)
    const uint16_t *wq, *wk;
    const float *cs;
    const int64_t *pos;
    float *dwq, *dwk;  // backwards only
    float *slots;      // backwards: partial sums of dw, 2 D floats for each workgroup
    uint32_t *counters;
    int64_t tokens, table;
    int hq, heads;  // query heads, and query + key heads
    int rotated, interleaved;
    int steps, parts;  // steps of rows a token takes; waves that share a token (forward)
    float eps;
};

template <bool VEC, int N>
__device__ __forceinline__ void loadf(const float *p, float (&r)[N]) {
#pragma unroll
    for (int i = 0; i < N; i += 4) {
        if (VEC) {
            const float4 t = *reinterpret_cast<const float4 *>(p + i);
            r[i] = t.x, r[i + 1] = t.y, r[i + 2] = t.z, r[i + 3] = t.w;
        } else {
            for (int j = 0; j < 4; ++j) r[i + j] = p[i + j];
        }
    }
}

__device__ __forceinline__ void widen(u32x4 v, float (&f)[8]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) f[2 * i] = lo_f32(v[i]), f[2 * i + 1] = hi_f32(v[i]);
}

// Sum over the D/8 lanes of a row; every lane gets it.
template <int LANES>
__device__ __forceinline__ float row_sum(float v) {
#pragma unroll
    for (int m = 1; m < LANES; m *= 2) v += __shfl_xor(v, m);
    return v;
}

// What a lane needs of its token: the factors of its eight channels in
// y_c = z_c cos_c + z_mate(c) sin_c (the sign of the sine folded in), and
// where the mates are.
template <int D, bool VEC>
struct Turn {
    float c[8], s[8];
    bool turns;   // whether this lane's channels turn at all
    int mate;     // the lane that holds the mates (this one where pairs lie side by side)
    bool within;  // pairs side by side

    __device__ __forceinline__ void place(const NormArgs &a, int lane) {
        constexpr int kLanes = D / 8;
        const int li = lane % kLanes, half = a.rotated / 16;
        turns = li < 2 * half;
        within = a.interleaved != 0;
        mate = within || !turns ? lane : li < half ? lane + half : lane - half;
    }
    __device__ __forceinline__ void load(const NormArgs &a, int lane, const float *row) {
        constexpr int kLanes = D / 8;
        const int li = lane % kLanes, half = a.rotated / 16;
        if (within) {
            float cc[4] = {1, 1, 1, 1}, ss[4] = {0, 0, 0, 0};
            if (turns) {
                loadf<VEC>(row + li * 4, cc);
                loadf<VEC>(row + a.rotated / 2 + li * 4, ss);
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) c[e] = cc[e / 2], s[e] = e % 2 ? ss[e / 2] : -ss[e / 2];
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) c[e] = 1, s[e] = 0;
            if (turns) {
                const int at = (li < half ? li : li - half) * 8;
                loadf<VEC>(row + at, c);
                loadf<VEC>(row + a.rotated / 2 + at, s);
                if (li < half) {
#pragma unroll
                    for (int e = 0; e < 8; ++e) s[e] = -s[e];
                }
            }
        }
    }
    // The words of the mates of a lane's four words.
    __device__ __forceinline__ u32x4 mates(u32x4 v) const {
        u32x4 r;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            r[i] = within ? (v[i] >> 16) | (v[i] << 16) : (uint32_t)__shfl((int)v[i], mate);
        return r;
    }
};

template <int D, bool VEC>
__global__ __launch_bounds__(kThreads) void k_norm_rope(NormArgs a) {
    constexpr int kLanes = D / 8, kRows = 64 / kLanes;
    const int lane = threadIdx.x % 64, li = lane % kLanes;
    const int64_t item = (int64_t)blockIdx.x * (kThreads / 64) + threadIdx.x / 64;
    const int64_t token = item / a.parts;
    if (token >= a.tokens) return;
    const int first = (int)(item % a.parts) * kSteps;

    u32x4 x[kSteps];
#pragma unroll
    for (int u = 0; u < kSteps; ++u) {
        const int h = (first + u) * kRows + lane / kLanes;
        if (h < a.heads) {
            const bool isq = h < a.hq;
            const uint16_t *p = isq ? a.q.p + token * a.q.ts + h * a.q.hs
                                    : a.k.p + token * a.k.ts + (h - a.hq) * a.k.hs;
            x[u] = load8<VEC>(p + li * 8);
        } else {
            x[u] = u32x4{0, 0, 0, 0};
        }
    }
    Turn<D, VEC> turn;
    turn.place(a, lane);
    const int64_t pos = a.pos[token];
    const bool known = pos >= 0 && pos < a.table;
    turn.load(a, lane, a.cs + (known ? pos : 0) * a.rotated);
    u32x4 wq = {0, 0, 0, 0}, wk = {0, 0, 0, 0};
    if (a.hq > 0) wq = load8<VEC>(a.wq + li * 8);
    if (a.heads > a.hq) wk = load8<VEC>(a.wk + li * 8);
    const u32x4 wqm = turn.mates(wq), wkm = turn.mates(wk);

#pragma unroll
    for (int u = 0; u < kSteps; ++u) {
        const int h = (first + u) * kRows + lane / kLanes;
        const bool isq = h < a.hq;
        const u32x4 xm = turn.mates(x[u]);
        float f[8], m[8], w[8], wm[8];
        widen(x[u], f);
        widen(xm, m);
        widen(isq ? wq : wk, w);
        widen(isq ? wqm : wkm, wm);
        float ss = 0;
#pragma unroll
        for (int e = 0; e < 8; ++e) ss += f[e] * f[e];
        const float r = rsqrtf(row_sum<kLanes>(ss) * (1.0f / D) + a.eps);
        float y[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float z = f[e] * r * w[e];
            const float t = z * turn.c[e] + m[e] * r * wm[e] * turn.s[e];
            y[e] = !known ? __uint_as_float(0x7FC00000u) : turn.turns ? t : z;
        }
        if (h < a.heads) {
            uint16_t *p = const_cast<uint16_t *>(isq ? a.oq.p + token * a.oq.ts + h * a.oq.hs
                                                     : a.ok.p + token * a.ok.ts + (h - a.hq) * a.ok.hs);
            u32x4 o;
#pragma unroll
            for (int i = 0; i < 4; ++i) o[i] = pack_bf16x2(y[2 * i], y[2 * i + 1]);
            store8<VEC>(p + li * 8, o);
        }
    }
}

// Backwards.  Each lane keeps the sums of g n of its channels over all rows
// that it meets (binary32; rows, lanes, waves, workgroups and groups of
// workgroups are joined as a tree in a fixed order, so the sums do not depend
// on which workgroup ends last).
template <int D, bool VEC>
__global__ __launch_bounds__(kThreads) void k_norm_rope_grad(NormArgs a) {
    constexpr int kLanes = D / 8, kRows = 64 / kLanes, kWaves = kThreads / 64;
    const int lane = threadIdx.x % 64, li = lane % kLanes, wave = threadIdx.x / 64;
    Turn<D, VEC> turn;
    turn.place(a, lane);
    u32x4 wq = {0, 0, 0, 0}, wk = {0, 0, 0, 0};
    if (a.tokens > 0 && a.hq > 0) wq = load8<VEC>(a.wq + li * 8);
    if (a.tokens > 0 && a.heads > a.hq) wk = load8<VEC>(a.wk + li * 8);
    float dq[8] = {}, dk[8] = {};

    for (int64_t token = (int64_t)blockIdx.x * kWaves + wave; token < a.tokens;
         token += (int64_t)gridDim.x * kWaves) {
        const int64_t pos = a.pos[token];
        const bool known = pos >= 0 && pos < a.table;
        turn.load(a, lane, a.cs + (known ? pos : 0) * a.rotated);
        for (int first = 0; first < a.steps; first += kGradSteps) {
            u32x4 x[kGradSteps], gy[kGradSteps];
#pragma unroll
            for (int u = 0; u < kGradSteps; ++u) {
                const int h = (first + u) * kRows + lane / kLanes;
                x[u] = gy[u] = u32x4{0, 0, 0, 0};
                if (h < a.heads) {
                    const bool isq = h < a.hq;
                    const int hh = isq ? h : h - a.hq;
                    x[u] = load8<VEC>((isq ? a.q.p + token * a.q.ts + hh * a.q.hs
                                           : a.k.p + token * a.k.ts + hh * a.k.hs) + li * 8);
                    gy[u] = load8<VEC>((isq ? a.gq.p + token * a.gq.ts + hh * a.gq.hs
                                            : a.gk.p + token * a.gk.ts + hh * a.gk.hs) + li * 8);
                }
            }
#pragma unroll
            for (int u = 0; u < kGradSteps; ++u) {
                const int h = (first + u) * kRows + lane / kLanes;
                const bool isq = h < a.hq;
                float f[8], g[8], m[8], w[8];
                widen(x[u], f);
                widen(gy[u], g);
                widen(turn.mates(gy[u]), m);
                widen(isq ? wq : wk, w);
                float ss = 0;
#pragma unroll
                for (int e = 0; e < 8; ++e) ss += f[e] * f[e];
                const float r = rsqrtf(row_sum<kLanes>(ss) * (1.0f / D) + a.eps);
                float along = 0;
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const float t = g[e] * turn.c[e] - m[e] * turn.s[e];
                    g[e] = !known ? __uint_as_float(0x7FC00000u) : turn.turns ? t : g[e];
                    f[e] *= r;
                    along += g[e] * w[e] * f[e];
                }
                along = row_sum<kLanes>(along) * (1.0f / D);
                if (h < a.heads) {
                    u32x4 o;
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        o[i] = pack_bf16x2(r * (g[2 * i] * w[2 * i] - f[2 * i] * along),
                                           r * (g[2 * i + 1] * w[2 * i + 1] - f[2 * i + 1] * along));
                    const int hh = isq ? h : h - a.hq;
                    store8<VEC>(const_cast<uint16_t *>(isq ? a.oq.p + token * a.oq.ts + hh * a.oq.hs
                                                           : a.ok.p + token * a.ok.ts + hh * a.ok.hs) + li * 8, o);
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const float t = g[e] * f[e];
                        if (isq) dq[e] += t;
                        else dk[e] += t;
                    }
                }
            }
        }
    }

    // the rows of a wave, then the waves of the workgroup
    __shared__ float part[kWaves][2 * D];
    __shared__ uint32_t order;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
#pragma unroll
        for (int m = kLanes; m < 64; m *= 2) {
            dq[e] += __shfl_xor(dq[e], m);
            dk[e] += __shfl_xor(dk[e], m);
        }
        if (lane < kLanes) {
            part[wave][li * 8 + e] = dq[e];
            part[wave][D + li * 8 + e] = dk[e];
        }
    }
    __syncthreads();
    float *slot = a.slots + (int64_t)blockIdx.x * 2 * D;
    for (int c = threadIdx.x; c < 2 * D; c += kThreads) {
        float t = part[0][c];
#pragma unroll
        for (int i = 1; i < kWaves; ++i) t += part[i][c];
        store_shared(slot + c, t);
    }
    // groups of kJoin workgroups, then the groups: whoever comes last in a
    // group adds its slots up into the group's first, whoever comes last of
    // the groups adds those
    const int groups = (int)((gridDim.x + kJoin - 1) / kJoin), mine = (int)(blockIdx.x / kJoin);
    const int size = min(kJoin, (int)gridDim.x - mine * kJoin);
    if (!arrive_last(a.counters + 1 + mine, size, &order)) return;
    float *base = a.slots + (int64_t)mine * kJoin * 2 * D;
    for (int c = threadIdx.x; c < 2 * D; c += kThreads) {
        float t = 0;
#pragma unroll 8
        for (int i = 0; i < size; ++i) t += load_shared(base + (int64_t)i * 2 * D + c);
        store_shared(base + c, t);
    }
    if (!arrive_last(a.counters, groups, &order)) return;
    for (int c = threadIdx.x; c < 2 * D; c += kThreads) {
        float t = 0;
#pragma unroll 8
        for (int i = 0; i < groups; ++i) t += load_shared(a.slots + (int64_t)i * kJoin * 2 * D + c);
        if (c < D) {
            if (a.dwq) a.dwq[c] = t;
        } else if (a.dwk) {
            a.dwk[c - D] = t;
        }
    }
}

template <bool GRAD>
const void *pick(int dim, bool vec) {
#define AR_PICK(D_)                                                                        \
    case D_:                                                                               \
        if (GRAD)                                                                          \
            return vec ? reinterpret_cast<const void *>(&k_norm_rope_grad<D_, true>)       \
                       : reinterpret_cast<const void *>(&k_norm_rope_grad<D_, false>);     \
        return vec ? reinterpret_cast<const void *>(&k_norm_rope<D_, true>)                \
                   : reinterpret_cast<const void *>(&k_norm_rope<D_, false>);
    switch (dim) {
        AR_PICK(64)
        AR_PICK(128)
        AR_PICK(256)
    }
#undef AR_PICK
    return nullptr;
}

// Workgroups of the backward pass: a token to each wave, as long as the slots
// of the partial sums last.
int grad_blocks(int64_t tokens) {
    const int64_t blocks = (tokens + kThreads / 64 - 1) / (kThreads / 64);
    return (int)(blocks < kJoin * kJoin ? blocks : kJoin * kJoin);
}

bool valid_shape(int64_t tokens, int heads, int kv_heads, int dim) {
    return tokens >= 0 && tokens <= (int64_t)1 << 28 && heads >= 0 && kv_heads >= 0 &&
           heads <= kMaxHeads && kv_heads <= kMaxHeads && (dim == 64 || dim == 128 || dim == 256);
}

int check(const RowsArg *const *reads, int nreads, const RowsArg *const *writes, int nwrites,
          const void *wq, const void *wk, const void *cs, const void *pos, int64_t tokens, int heads,
          int kv_heads, int dim, int rotated, int64_t table, float eps) {
    if (!valid_shape(tokens, heads, kv_heads, dim) || rotated < 16 || rotated > dim ||
        rotated % 16 || table < 1 || table > (int64_t)1 << 31 || !(eps >= 0) || !(eps <= 3.0e38f))
        return AR_EINVAL;
    if (tokens == 0 || heads + kv_heads == 0) return AR_OK;
    for (int i = 0; i < nreads; ++i)
        if (!reads[i]->valid()) return AR_EINVAL;
    for (int i = 0; i < nwrites; ++i)
        if (!writes[i]->valid() || writes[i]->self_overlap()) return AR_EINVAL;
    if ((heads && (!wq || !aligned_to(wq, 2))) || (kv_heads && (!wk || !aligned_to(wk, 2))) || !cs ||
        !aligned_to(cs, 4) || !pos || !aligned_to(pos, 8))
        return AR_EINVAL;
    const Span small[] = {{addr(wq), (uintptr_t)(heads ? 2 * dim : 0)},
                          {addr(wk), (uintptr_t)(kv_heads ? 2 * dim : 0)},
                          {addr(cs), (uintptr_t)(4 * table * rotated)},
                          {addr(pos), (uintptr_t)(8 * tokens)}};
    for (int o = 0; o < nwrites; ++o) {
        for (const Span &s : small)
            if (overlap(writes[o]->span(), s)) return AR_EALIAS;
        for (int i = 0; i < nreads; ++i)
            // in place: queries over queries, keys over keys, row by row
            if (!(i % 2 == o && writes[o]->same(*reads[i])) && writes[o]->overlaps(*reads[i]))
                return AR_EALIAS;
        for (int j = o + 1; j < nwrites; ++j)
            if (writes[o]->overlaps(*writes[j])) return AR_EALIAS;
    }
    return AR_OK;
}

}  // namespace
}  // namespace ar

using namespace ar;

extern "C" {

int ar_qk_norm_rope(ar_rows q, ar_rows k, const void *q_weight, const void *k_weight,
                    const void *cos_sin, const void *positions, ar_rows q_out, ar_rows k_out,
                    int64_t tokens, int heads, int kv_heads, int dim, int rotated, int64_t table,
                    float eps, int interleaved, void *stream) {
    const RowsArg rq{q, tokens, heads, dim}, rk{k, tokens, kv_heads, dim},
        oq{q_out, tokens, heads, dim}, ok{k_out, tokens, kv_heads, dim};
    const RowsArg *reads[] = {&rq, &rk}, *writes[] = {&oq, &ok};
    const int rc = check(reads, 2, writes, 2, q_weight, k_weight, cos_sin, positions, tokens, heads,
                         kv_heads, dim, rotated, table, eps);
    if (rc != AR_OK || tokens == 0 || heads + kv_heads == 0) return rc;
    NormArgs a = {};
    a.q = rows(rq), a.k = rows(rk), a.oq = rows(oq), a.ok = rows(ok);
    a.wq = static_cast<const uint16_t *>(q_weight), a.wk = static_cast<const uint16_t *>(k_weight);
    a.cs = static_cast<const float *>(cos_sin), a.pos = static_cast<const int64_t *>(positions);
    a.tokens = tokens, a.table = table, a.hq = heads, a.heads = heads + kv_heads;
    a.rotated = rotated, a.interleaved = interleaved != 0, a.eps = eps;
    const int per = 512 / dim;  // rows a wave works on at once
    a.steps = (a.heads + per - 1) / per;
    a.parts = (a.steps + kSteps - 1) / kSteps;
    const bool vec = rq.vec() && rk.vec() && oq.vec() && ok.vec() && aligned_to(q_weight, 16) &&
                     aligned_to(k_weight, 16) && aligned_to(cos_sin, 16);
    const int64_t blocks = (tokens * a.parts + kThreads / 64 - 1) / (kThreads / 64);
    if (blocks > 0x7FFFFFFF / kThreads) return AR_EINVAL;
    return launch(pick<false>(dim, vec), (unsigned)blocks, kThreads, a, stream);
}

int64_t ar_qk_norm_rope_bwd_workspace(int64_t tokens, int heads, int kv_heads, int dim) {
    if (!valid_shape(tokens, heads, kv_heads, dim)) return AR_EINVAL;
    return 4 * (int64_t)kJoinCounters + (int64_t)grad_blocks(tokens) * 2 * dim * 4;
}

int ar_qk_norm_rope_bwd(ar_rows q_grad, ar_rows k_grad, ar_rows q, ar_rows k, const void *q_weight,
                        const void *k_weight, const void *cos_sin, const void *positions, ar_rows dq,
                        ar_rows dk, void *dq_weight, void *dk_weight, void *workspace,
                        int64_t tokens, int heads, int kv_heads, int dim, int rotated, int64_t table,
                        float eps, int interleaved, void *stream) {
    const RowsArg rq{q, tokens, heads, dim}, rk{k, tokens, kv_heads, dim},
        gq{q_grad, tokens, heads, dim}, gk{k_grad, tokens, kv_heads, dim},
        oq{dq, tokens, heads, dim}, ok{dk, tokens, kv_heads, dim};
    const RowsArg *reads[] = {&rq, &rk, &gq, &gk}, *writes[] = {&oq, &ok};
    const int rc = check(reads, 4, writes, 2, q_weight, k_weight, cos_sin, positions, tokens, heads,
                         kv_heads, dim, rotated, table, eps);
    if (rc != AR_OK) return rc;
    if (heads + kv_heads == 0) return AR_OK;
    // the weights' gradients and the workspace are apart from everything else
    const Span outs[] = {{addr(dq_weight), (uintptr_t)(heads ? 4 * dim : 0)},
                         {addr(dk_weight), (uintptr_t)(kv_heads ? 4 * dim : 0)},
                         {addr(workspace), (uintptr_t)ar_qk_norm_rope_bwd_workspace(tokens, heads, kv_heads, dim)}};
    if ((heads && !dq_weight) || (kv_heads && !dk_weight) || !workspace ||
        !aligned_to(dq_weight, 4) || !aligned_to(dk_weight, 4) || !aligned_to(workspace, 16))
        return AR_EINVAL;
    const Span others[] = {rq.span(), rk.span(), gq.span(), gk.span(), oq.span(), ok.span(),
                           {addr(q_weight), (uintptr_t)(heads ? 2 * dim : 0)},
                           {addr(k_weight), (uintptr_t)(kv_heads ? 2 * dim : 0)},
                           {addr(cos_sin), (uintptr_t)(4 * table * rotated)},
                           {addr(positions), (uintptr_t)(8 * tokens)}};
    for (int i = 0; i < 3; ++i) {
        for (const Span &s : others)
            if (overlap(outs[i], s)) return AR_EALIAS;
        for (int j = i + 1; j < 3; ++j)
            if (overlap(outs[i], outs[j])) return AR_EALIAS;
    }
    NormArgs a = {};
    a.q = rows(rq), a.k = rows(rk), a.gq = rows(gq), a.gk = rows(gk), a.oq = rows(oq), a.ok = rows(ok);
    a.wq = static_cast<const uint16_t *>(q_weight), a.wk = static_cast<const uint16_t *>(k_weight);
    a.cs = static_cast<const float *>(cos_sin), a.pos = static_cast<const int64_t *>(positions);
    a.dwq = heads ? static_cast<float *>(dq_weight) : nullptr;
    a.dwk = kv_heads ? static_cast<float *>(dk_weight) : nullptr;
    a.counters = static_cast<uint32_t *>(workspace);
    a.slots = reinterpret_cast<float *>(a.counters + kJoinCounters);
    a.tokens = tokens, a.table = table, a.hq = heads, a.heads = heads + kv_heads;
    a.rotated = rotated, a.interleaved = interleaved != 0, a.eps = eps;
    const int per = 512 / dim;
    a.steps = (a.heads + per - 1) / per;
    const bool vec = rq.vec() && rk.vec() && gq.vec() && gk.vec() && oq.vec() && ok.vec() &&
                     aligned_to(q_weight, 16) && aligned_to(k_weight, 16) && aligned_to(cos_sin, 16);
    // no tokens: one workgroup still writes the weights' gradients, zeros
    const int blocks = tokens ? grad_blocks(tokens) : 1;
    return launch(pick<true>(dim, vec), (unsigned)blocks, kThreads, a, stream);
}

}  // extern "C"
