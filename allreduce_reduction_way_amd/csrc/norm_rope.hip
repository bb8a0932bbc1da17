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
// takes several steps of rows.  Measured: 8192 tokens of 64 heads of 128 in 49
// us, 5.5 TB/s; the gradient of 4096 tokens of 72 heads in 49.6 us, 4.6 TB/s,
// 4.6 us of them the sums of the weights' gradients.
#include "host.h"
#include "rows.h"

namespace ar {
namespace {

constexpr int kMaxHeads = 1 << 16;
// Above this many bytes, rows are read and written past the caches (as the
// reduce kernels do): 268 MB forward take 49.2 us with it and 53.6 without, 226
// MB backwards 49.9 and 53.9 (before its rows were loaded a step ahead: 45.3
// now); rows of 0.5 to 12 MB take up to 0.7 us longer with it.
constexpr int64_t kStreamBytes = (int64_t)128 << 20;
struct NormArgs {
    Rows q, k, gq, gk, oq, ok;  // gq, gk: incoming gradients (backwards only)
    const uint16_t *wq, *wk;
    const float *cs;
    const int64_t *pos;
    float *dwq, *dwk;  // backwards only
    float *slots;      // backwards: partial sums of dw, 2 D floats for each workgroup
    int64_t tokens, table;
    int hq, hk;  // query heads and key heads
    int rotated, interleaved;
    int qsteps, steps, per, parts;  // steps of rows: of a token's queries, of it all, of a wave; waves that share a token
    int blocks;             // backwards: workgroups, each with a slot
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
    __device__ __forceinline__ void load(const NormArgs &a, int lane, int64_t pos) {
        const bool known = pos >= 0 && pos < a.table;
        const float *row = a.cs + (known ? pos : 0) * a.rotated;
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
        if (!known) {  // NaN rows
#pragma unroll
            for (int e = 0; e < 8; ++e) c[e] = __uint_as_float(0x7FC00000u);
        }
    }
    // The words of the mates of a lane's four words; zeros where it does not
    // turn.
    __device__ __forceinline__ u32x4 mates(u32x4 v) const {
        u32x4 r;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t w = within ? (v[i] >> 16) | (v[i] << 16) : (uint32_t)__shfl((int)v[i], mate);
            r[i] = turns ? w : 0;
        }
        return r;
    }
};

__device__ __forceinline__ uint32_t bf16_pair(float lo, float hi) {
    typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
    bf16x2 r;
    r[0] = (__bf16)lo;
    r[1] = (__bf16)hi;
    return __builtin_bit_cast(uint32_t, r);
}

__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }

// A token's rows of queries, or of keys, and its steps [begin, end) that a
// wave takes: a step is kRows heads.
struct Share {
    const uint16_t *x;
    uint16_t *out;
    const uint16_t *w;
    int64_t in_hs, out_hs;
    int heads, begin, end;
};

// VEC and NT: 16-byte accesses, non-temporal ones.
template <bool VEC, bool NT>
__device__ __forceinline__ u32x4 load_row(const uint16_t *p) {
    return NT ? __builtin_nontemporal_load(reinterpret_cast<const u32x4 *>(p)) : load8<VEC>(p);
}

template <bool VEC, bool NT>
__device__ __forceinline__ void store_row(uint16_t *p, u32x4 v) {
    if (NT) __builtin_nontemporal_store(v, reinterpret_cast<u32x4 *>(p));
    else store8<VEC>(p, v);
}

// U: steps of rows that a wave has in flight.  A step is of queries or of
// keys, so that all that depends on that is the same in a wave's lanes, and
// the weights are multiplied into the cosines and sines once.
template <int D, bool VEC, int U, bool NT>
__global__ __launch_bounds__(kThreads) void k_norm_rope(NormArgs a) {
    constexpr int kLanes = D / 8, kRows = 64 / kLanes;
    const int lane = threadIdx.x % 64, li = lane % kLanes;
    const int item = uniform(blockIdx.x * (kThreads / 64) + threadIdx.x / 64);
    const int64_t token = item / a.parts;
    if (token >= a.tokens) return;
    const int begin = item % a.parts * a.per, end = min(begin + a.per, a.steps);
    const int64_t pos = a.pos[token];
    Turn<D, VEC> turn;
    turn.place(a, lane);

    const auto go = [&](const Share &sh) {
        if (sh.begin >= sh.end) return;
        const auto at = [&](int first, int u) { return (first + u) * kRows + lane / kLanes; };
        u32x4 x[U];
        const auto load = [&](int first) {
#pragma unroll
            for (int u = 0; u < U; ++u) {
                x[u] = u32x4{0, 0, 0, 0};
                if (at(first, u) < sh.heads) x[u] = load_row<VEC, NT>(sh.x + at(first, u) * sh.in_hs + li * 8);
            }
        };
        load(sh.begin);
        const u32x4 weight = load8<VEC>(sh.w + li * 8);
        turn.load(a, lane, pos);
        float own[8], mate[8];  // y_c = r (x_c own_c + x_mate mate_c)
        widen(weight, own);
        widen(turn.mates(weight), mate);
#pragma unroll
        for (int e = 0; e < 8; ++e) own[e] *= turn.c[e], mate[e] *= turn.s[e];
        for (int first = sh.begin; first < sh.end; first += U) {
            if (first != sh.begin) load(first);
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if (first + u >= sh.end) break;
                float f[8], m[8];
                widen(x[u], f);
                widen(turn.mates(x[u]), m);
                float ss = 0;
#pragma unroll
                for (int e = 0; e < 8; ++e) ss += f[e] * f[e];
                const float r = rsqrtf(row_sum<kLanes>(ss) * (1.0f / D) + a.eps);
#pragma unroll
                for (int e = 0; e < 8; ++e) f[e] = (f[e] * own[e] + m[e] * mate[e]) * r;
                if (at(first, u) < sh.heads) {
                    const u32x4 o = {bf16_pair(f[0], f[1]), bf16_pair(f[2], f[3]), bf16_pair(f[4], f[5]), bf16_pair(f[6], f[7])};
                    store_row<VEC, NT>(sh.out + at(first, u) * sh.out_hs + li * 8, o);
                }
            }
        }
    };
    go(Share{a.q.p + token * a.q.ts, const_cast<uint16_t *>(a.oq.p) + token * a.oq.ts, a.wq, a.q.hs, a.oq.hs, a.hq, begin,
             min(end, a.qsteps)});
    go(Share{a.k.p + token * a.k.ts, const_cast<uint16_t *>(a.ok.p) + token * a.ok.ts, a.wk, a.k.hs, a.ok.hs, a.hk,
             max(begin - a.qsteps, 0), end - a.qsteps});
}

// Backwards.  Each lane keeps the sums of g n of its channels over all rows
// that it meets (binary32; rows, lanes, waves and workgroups are joined as a
// tree in a fixed order, so the sums are the same each time).  Each workgroup
// leaves its own in the workspace, and a second launch adds them up: with the
// last workgroup to arrive doing that, 440 tokens of 6 heads took 10.4 us where
// the two launches take 8.3.
template <int D, bool VEC, bool NT>
__global__ __launch_bounds__(kThreads) void k_norm_rope_grad(NormArgs a) {
    constexpr int kLanes = D / 8, kRows = 64 / kLanes, kWaves = kThreads / 64;
    const int lane = threadIdx.x % 64, li = lane % kLanes, wave = uniform(threadIdx.x / 64);
    Turn<D, VEC> turn;
    turn.place(a, lane);
    float dq[8] = {}, dk[8] = {};

    for (int64_t item = (int64_t)blockIdx.x * kWaves + wave; item < a.tokens * a.parts;
         item += (int64_t)gridDim.x * kWaves) {
        const int64_t token = item / a.parts;
        const int begin = (int)(item % a.parts) * a.per, end = min(begin + a.per, a.steps);
        turn.load(a, lane, a.pos[token]);
        const auto go = [&](const Share &sh, const uint16_t *gy, int64_t gy_hs, float(&dw)[8]) {
            if (sh.begin >= sh.end) return;
            u32x4 x, gx;  // of the step that comes next
            const auto load = [&](int step) {
                const int h = step * kRows + lane / kLanes;
                x = gx = u32x4{0, 0, 0, 0};
                if (h < sh.heads) {
                    x = load_row<VEC, NT>(sh.x + h * sh.in_hs + li * 8);
                    gx = load_row<VEC, NT>(gy + h * gy_hs + li * 8);
                }
            };
            load(sh.begin);
            float w[8];
            widen(load8<VEC>(sh.w + li * 8), w);
            for (int step = sh.begin; step < sh.end; ++step) {
                const int h = step * kRows + lane / kLanes;
                float n[8], g[8], m[8];
                widen(x, n);
                widen(gx, g);
                widen(turn.mates(gx), m);
                if (step + 1 < sh.end) load(step + 1);
                float ss = 0;
#pragma unroll
                for (int e = 0; e < 8; ++e) ss += n[e] * n[e];
                const float r = rsqrtf(row_sum<kLanes>(ss) * (1.0f / D) + a.eps);
                float along = 0;
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    n[e] *= r;
                    g[e] = g[e] * turn.c[e] - m[e] * turn.s[e];
                    if (h < sh.heads) dw[e] += g[e] * n[e];
                    g[e] *= w[e];
                    along += g[e] * n[e];
                }
                along = row_sum<kLanes>(along) * (1.0f / D);
                if (h < sh.heads) {
#pragma unroll
                    for (int e = 0; e < 8; ++e) g[e] = r * (g[e] - n[e] * along);
                    const u32x4 o = {bf16_pair(g[0], g[1]), bf16_pair(g[2], g[3]), bf16_pair(g[4], g[5]), bf16_pair(g[6], g[7])};
                    store_row<VEC, NT>(sh.out + h * sh.out_hs + li * 8, o);
                }
            }
        };
        go(Share{a.q.p + token * a.q.ts, const_cast<uint16_t *>(a.oq.p) + token * a.oq.ts, a.wq, a.q.hs, a.oq.hs, a.hq, begin,
                 min(end, a.qsteps)},
           a.gq.p + token * a.gq.ts, a.gq.hs, dq);
        go(Share{a.k.p + token * a.k.ts, const_cast<uint16_t *>(a.ok.p) + token * a.ok.ts, a.wk, a.k.hs, a.ok.hs, a.hk,
                 max(begin - a.qsteps, 0), end - a.qsteps},
           a.gk.p + token * a.gk.ts, a.gk.hs, dk);
    }

    // the rows of a wave, then the waves of the workgroup
    __shared__ float part[kWaves][2 * D];
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
        slot[c] = t;
    }
}

// Adds the workgroups' sums up: eight columns to a workgroup, 32 slots of each
// at a time.
__global__ __launch_bounds__(256) void k_norm_rope_weights(NormArgs a, int dim) {
    __shared__ float part[32][8];
    const int c = blockIdx.x * 8 + threadIdx.x % 8, s0 = threadIdx.x / 8;
    float t = 0;
    for (int s = s0; s < a.blocks; s += 32 * 16) {
        float v[16];  // all on their way at once
#pragma unroll
        for (int k = 0; k < 16; ++k) v[k] = a.slots[(int64_t)min(s + 32 * k, a.blocks - 1) * 2 * dim + c];
#pragma unroll
        for (int k = 0; k < 16; ++k) t += s + 32 * k < a.blocks ? v[k] : 0.0f;
    }
    part[s0][threadIdx.x % 8] = t;
    __syncthreads();
    if (s0 > 0) return;
#pragma unroll
    for (int s = 1; s < 32; ++s) t += part[s][threadIdx.x];
    if (c < dim) {
        if (a.dwq) a.dwq[c] = t;
    } else if (a.dwk) {
        a.dwk[c - dim] = t;
    }
}

template <int D>
const void *pick_dim(bool grad, bool vec, bool few, bool stream) {
    if (grad)
        return !vec     ? reinterpret_cast<const void *>(&k_norm_rope_grad<D, false, false>)
               : stream ? reinterpret_cast<const void *>(&k_norm_rope_grad<D, true, true>)
                        : reinterpret_cast<const void *>(&k_norm_rope_grad<D, true, false>);
    return !vec     ? reinterpret_cast<const void *>(&k_norm_rope<D, false, 1, false>)
           : few    ? reinterpret_cast<const void *>(&k_norm_rope<D, true, 1, false>)
           : stream ? reinterpret_cast<const void *>(&k_norm_rope<D, true, 4, true>)
                    : reinterpret_cast<const void *>(&k_norm_rope<D, true, 4, false>);
}

const void *pick(int dim, bool grad, bool vec, bool few, bool stream) {
    return dim == 64    ? pick_dim<64>(grad, vec, few, stream)
           : dim == 128 ? pick_dim<128>(grad, vec, few, stream)
                        : pick_dim<256>(grad, vec, few, stream);
}

void count_steps(NormArgs &a, int dim) {
    const int per = 512 / dim;  // rows that a wave works on at once
    a.qsteps = (a.hq + per - 1) / per;
    a.steps = a.qsteps + (a.hk + per - 1) / per;
}

constexpr int kSlots = 1024;  // workgroups of the backward pass, at most

// Waves that share a token backwards, and workgroups, each with a slot for its
// sums: a wave for each step of a token while the slots last.
int grad_parts(int64_t tokens, int steps) {
    const int64_t parts = tokens ? kSlots * (kThreads / 64) / tokens : 1;
    return (int)(parts < 1 ? 1 : parts > steps ? steps : parts);
}

int grad_blocks(int64_t tokens, int64_t parts) {
    const int64_t blocks = (tokens * parts + kThreads / 64 - 1) / (kThreads / 64);
    return (int)(blocks < 1 ? 1 : blocks < kSlots ? blocks : kSlots);
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
    a.tokens = tokens, a.table = table, a.hq = heads, a.hk = kv_heads;
    a.rotated = rotated, a.interleaved = interleaved != 0, a.eps = eps;
    count_steps(a, dim);
    // Few rows, or few to a token: a wave for each step, since what a wave does
    // takes longer than its share of the memory (8000 tokens of 16 heads of 64:
    // 9.7 us, and 11.2 with both steps to a wave).  Many: as many steps to a
    // wave as leave sixteen waves for each SIMD (eight at once: 53.6 us for 268
    // MB against 57.7 with eight in all), which read their token's cosines and
    // sines once.
    const bool few = tokens * a.steps <= 8192 || a.steps <= 2;
    const int64_t parts = few ? a.steps : (16384 + tokens - 1) / tokens;
    a.per = (int)((a.steps + parts - 1) / parts);
    if (!few) a.per = (a.per + 3) / 4 * 4;
    a.parts = (a.steps + a.per - 1) / a.per;
    const bool vec = rq.vec() && rk.vec() && oq.vec() && ok.vec() && aligned_to(q_weight, 16) &&
                     aligned_to(k_weight, 16) && aligned_to(cos_sin, 16);
    const int64_t blocks = (tokens * a.parts + kThreads / 64 - 1) / (kThreads / 64);
    if (blocks > 0x7FFFFFFF / kThreads) return AR_EINVAL;
    const int64_t bytes = 4 * tokens * (heads + kv_heads) * dim;
    return launch(pick(dim, false, vec, few, bytes > kStreamBytes), (unsigned)blocks, kThreads, a, stream);
}

int64_t ar_qk_norm_rope_bwd_workspace(int64_t tokens, int heads, int kv_heads, int dim) {
    if (!valid_shape(tokens, heads, kv_heads, dim)) return AR_EINVAL;
    NormArgs a = {};
    a.hq = heads, a.hk = kv_heads;
    count_steps(a, dim);
    // The workgroups of no call of fewer tokens or heads are more than with a
    // wave for every step (those of single calls rise and fall with the tokens,
    // as the waves that share one get fewer).
    return (int64_t)grad_blocks(tokens, a.steps) * 2 * dim * 4;
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
    a.slots = static_cast<float *>(workspace);
    a.tokens = tokens, a.table = table, a.hq = heads, a.hk = kv_heads;
    a.rotated = rotated, a.interleaved = interleaved != 0, a.eps = eps;
    count_steps(a, dim);
    const bool vec = rq.vec() && rk.vec() && gq.vec() && gk.vec() && oq.vec() && ok.vec() &&
                     aligned_to(q_weight, 16) && aligned_to(k_weight, 16) && aligned_to(cos_sin, 16);
    // no tokens: one workgroup still writes the weights' gradients, zeros
    const int parts = grad_parts(tokens, a.steps);
    a.per = (a.steps + parts - 1) / parts;
    a.parts = (a.steps + a.per - 1) / a.per;
    a.blocks = grad_blocks(tokens, parts);
    const int64_t bytes = 6 * tokens * (heads + kv_heads) * dim;
    const int rc2 = launch(pick(dim, true, vec, false, bytes > kStreamBytes), (unsigned)a.blocks, kThreads, a, stream);
    if (rc2 != AR_OK) return rc2;
    void *args[] = {&a, &dim};
    return hipLaunchKernel(reinterpret_cast<const void *>(&k_norm_rope_weights), dim3(2 * dim / 8), dim3(256), args, 0,
                           static_cast<hipStream_t>(stream)) == hipSuccess
               ? AR_OK
               : AR_ELAUNCH;
}

}  // extern "C"
