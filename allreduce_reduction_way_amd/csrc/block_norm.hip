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
// Both are bound by memory: each row is read and written once, in binary32
// between.  A row lies in one workgroup, eight channels to a lane (twice eight
// beyond 8192 channels), so that both norms' sums are exchanges within it.
#include "host.h"
#include "rows.h"
#include "wave.h"

namespace ar {
namespace {

constexpr int kMaxDim = 1 << 14;
constexpr int kMaxThreads = 1024;
// Above this many bytes, rows are read and written past the caches.
constexpr int64_t kStreamBytes = (int64_t)128 << 20;

struct BlockArgs {
    const uint16_t *part[AR_MAX_P];
    Rows x, gate, h, z;      // h, z: outputs, or what comes in for them (backwards)
    Rows dx, dy, dgate;      // backwards only
    const uint16_t *post, *pre;
    float *slots;            // backwards: sums over a workgroup's tokens, 3 dim floats each
    int64_t part_stride, tokens;
    int dim;
    int shared_gate;         // backwards: all tokens have one gate
    float scale, eps;
};

template <bool NT>
__device__ __forceinline__ void store_vec8(uint16_t *p, const float (&f)[8], int n) {
    const u32x4 v = {bf16_pair(f[0], f[1]), bf16_pair(f[2], f[3]), bf16_pair(f[4], f[5]), bf16_pair(f[6], f[7])};
    if (n >= 8) {
        u32x4_any *to = reinterpret_cast<u32x4_any *>(p);
        if (NT) __builtin_nontemporal_store(v, to);
        else *to = v;
        return;
    }
#pragma unroll
    for (int i = 0; i < 7; ++i)
        if (i < n) p[i] = (uint16_t)(v[i / 2] >> (i % 2 * 16));
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

// P parts; V times eight channels to a lane.
template <int P, int V, bool NT>
__global__ __launch_bounds__(kMaxThreads) void k_block_norm(BlockArgs a) {
    __shared__ float part1[1][kMaxThreads / 64], part2[1][kMaxThreads / 64];
    const int64_t token = blockIdx.x;
    u32x4 y[V][P], x[V], g[V], w1[V], w2[V];
    int at[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
        at[i] = (int)(threadIdx.x + i * blockDim.x) * 8;
        const int n = a.dim - at[i];
#pragma unroll
        for (int p = 0; p < P; ++p) y[i][p] = u32x4{0, 0, 0, 0};
        x[i] = g[i] = w1[i] = w2[i] = u32x4{0, 0, 0, 0};
        if (n >= 8) {
#pragma unroll
            for (int p = 0; p < P; ++p) y[i][p] = load_vec8<NT>(a.part[p] + token * a.part_stride + at[i]);
            x[i] = load_vec8<NT>(a.x.p + token * a.x.ts + at[i]);
            if (a.gate.p) g[i] = load_vec8<false>(a.gate.p + token * a.gate.ts + at[i]);
            if (a.post) w1[i] = load_vec8<false>(a.post + at[i]);
            if (a.pre) w2[i] = load_vec8<false>(a.pre + at[i]);
        } else if (n > 0) {
#pragma unroll
            for (int p = 0; p < P; ++p) y[i][p] = load_few(a.part[p] + token * a.part_stride + at[i], n);
            x[i] = load_few(a.x.p + token * a.x.ts + at[i], n);
            if (a.gate.p) g[i] = load_few(a.gate.p + token * a.gate.ts + at[i], n);
            if (a.post) w1[i] = load_few(a.post + at[i], n);
            if (a.pre) w2[i] = load_few(a.pre + at[i], n);
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
        store_vec8<NT>(const_cast<uint16_t *>(a.h.p) + token * a.h.ts + at[i], f[i], a.dim - at[i]);
    }
    if (!a.pre) return;
    block_sum(s, part2);
    const float r = rsqrtf(s[0] * by + a.eps);
#pragma unroll
    for (int i = 0; i < V; ++i) {
        float w[8];
        widen(w2[i], w);
#pragma unroll
        for (int e = 0; e < 8; ++e) f[i][e] = f[i][e] * r * w[e];
        store_vec8<NT>(const_cast<uint16_t *>(a.z.p) + token * a.z.ts + at[i], f[i], a.dim - at[i]);
    }
}

// What a lane holds of one token's rows backwards.
template <bool NT>
struct GradRow {
    u32x4 x, y, dh, dz, g;
    __device__ __forceinline__ void load(const BlockArgs &a, int64_t token, int at) {
        const int n = a.dim - at;
        x = y = dh = dz = g = u32x4{0, 0, 0, 0};
        if (n >= 8) {
            y = load_vec8<NT>(a.part[0] + token * a.part_stride + at);
            x = load_vec8<NT>(a.x.p + token * a.x.ts + at);
            if (a.h.p) dh = load_vec8<NT>(a.h.p + token * a.h.ts + at);
            if (a.pre) dz = load_vec8<NT>(a.z.p + token * a.z.ts + at);
            if (a.gate.p) g = load_vec8<false>(a.gate.p + token * a.gate.ts + at);
        } else if (n > 0) {
            y = load_few(a.part[0] + token * a.part_stride + at, n);
            x = load_few(a.x.p + token * a.x.ts + at, n);
            if (a.h.p) dh = load_few(a.h.p + token * a.h.ts + at, n);
            if (a.pre) dz = load_few(a.z.p + token * a.z.ts + at, n);
            if (a.gate.p) g = load_few(a.gate.p + token * a.gate.ts + at, n);
        }
    }
};

// Backwards.  A workgroup takes tokens in turn, and each lane keeps its
// channels' sums over them; a second launch adds the workgroups' up, in a fixed
// order.
template <int V, bool NT>
__global__ __launch_bounds__(kMaxThreads) void k_block_norm_grad(BlockArgs a) {
    __shared__ float part1[1][kMaxThreads / 64], part2[2][kMaxThreads / 64], part3[1][kMaxThreads / 64];
    const float by = 1.0f / a.dim;
    float sg[V][8] = {}, s1[V][8] = {}, s2[V][8] = {};
    u32x4 w1[V], w2[V];
    int at[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
        at[i] = (int)(threadIdx.x + i * blockDim.x) * 8;
        const int n = a.dim - at[i];
        w1[i] = w2[i] = u32x4{0, 0, 0, 0};
        if (n > 0) {
            if (a.post) w1[i] = n >= 8 ? load_vec8<false>(a.post + at[i]) : load_few(a.post + at[i], n);
            if (a.pre) w2[i] = n >= 8 ? load_vec8<false>(a.pre + at[i]) : load_few(a.pre + at[i], n);
        }
    }
    // One set of rows to a lane: the next token's are on their way while this
    // one's are worked on.  They stay packed until they are used.
    constexpr bool kAhead = V == 1;
    GradRow<NT> next[V];
    if (kAhead) {
#pragma unroll
        for (int i = 0; i < V; ++i) next[i].load(a, blockIdx.x, at[i]);
    }
    for (int64_t token = blockIdx.x; token < a.tokens; token += gridDim.x) {
        GradRow<NT> row[V];
#pragma unroll
        for (int i = 0; i < V; ++i) {
            if (kAhead) row[i] = next[i];
            else row[i].load(a, token, at[i]);
        }
        if (kAhead && token + gridDim.x < a.tokens) {
#pragma unroll
            for (int i = 0; i < V; ++i) next[i].load(a, token + gridDim.x, at[i]);
        }
        float y[V][8], h[V][8], e[V][8];
        float r1 = 1.0f;
#pragma unroll
        for (int i = 0; i < V; ++i) widen(row[i].y, y[i]);
        if (a.post) {
            float s[1] = {0};
#pragma unroll
            for (int i = 0; i < V; ++i)
#pragma unroll
                for (int c = 0; c < 8; ++c) s[0] += y[i][c] * y[i][c];
            block_sum(s, part1);
            r1 = rsqrtf(s[0] * by + a.eps);
        }
        // y becomes n1 (y itself without a norm after the block)
        float s[2] = {0, 0};
#pragma unroll
        for (int i = 0; i < V; ++i) {
            float w[8], g[8], q[8];
            widen(w1[i], w);
            widen(row[i].g, g);
            widen(row[i].x, h[i]);
            widen(row[i].dz, q);
#pragma unroll
            for (int c = 0; c < 8; ++c) {
                y[i][c] *= r1;
                const float u = a.post ? y[i][c] * w[c] : y[i][c];
                h[i][c] = a.scale * h[i][c] + (a.gate.p ? g[c] * u : u);
            }
            widen(w2[i], w);
#pragma unroll
            for (int c = 0; c < 8; ++c) {
                s[0] += h[i][c] * h[i][c];
                s[1] += q[c] * w[c] * h[i][c];
            }
            widen(row[i].dh, e[i]);
        }
        if (a.pre) {
            block_sum(s, part2);
            const float r2 = rsqrtf(s[0] * by + a.eps), along = s[1] * by * r2;
#pragma unroll
            for (int i = 0; i < V; ++i) {
                float w[8], q[8];
                widen(w2[i], w);
                widen(row[i].dz, q);
#pragma unroll
                for (int c = 0; c < 8; ++c) {
                    const float n2 = h[i][c] * r2;
                    s2[i][c] += q[c] * n2;
                    e[i][c] += r2 * (q[c] * w[c] - n2 * along);
                }
            }
        }
        float d[1] = {0};
#pragma unroll
        for (int i = 0; i < V; ++i) {
            float w[8], g[8], t[8];
            widen(w1[i], w);
            widen(row[i].g, g);
#pragma unroll
            for (int c = 0; c < 8; ++c) t[c] = a.scale * e[i][c];
            store_vec8<NT>(const_cast<uint16_t *>(a.dx.p) + token * a.dx.ts + at[i], t, a.dim - at[i]);
#pragma unroll
            for (int c = 0; c < 8; ++c) {
                t[c] = e[i][c] * (a.post ? y[i][c] * w[c] : y[i][c]);
                sg[i][c] += t[c];
                if (a.gate.p) e[i][c] *= g[c];
                s1[i][c] += e[i][c] * y[i][c];
                if (a.post) e[i][c] *= w[c];
                d[0] += e[i][c] * y[i][c];
            }
            if (a.dgate.p) store_vec8<NT>(const_cast<uint16_t *>(a.dgate.p) + token * a.dgate.ts + at[i], t, a.dim - at[i]);
        }
        if (a.post) {
            block_sum(d, part3);
            const float along = d[0] * by;
#pragma unroll
            for (int i = 0; i < V; ++i)
#pragma unroll
                for (int c = 0; c < 8; ++c) e[i][c] = r1 * (e[i][c] - y[i][c] * along);
        }
#pragma unroll
        for (int i = 0; i < V; ++i)
            store_vec8<NT>(const_cast<uint16_t *>(a.dy.p) + token * a.dy.ts + at[i], e[i], a.dim - at[i]);
        // Each sum's part is written again after the barrier of another one.
        // Where there is one sum alone, after this one.
        if (!a.post) __syncthreads();
    }
    float *slot = a.slots + (int64_t)blockIdx.x * 3 * a.dim;
#pragma unroll
    for (int i = 0; i < V; ++i)
#pragma unroll
        for (int c = 0; c < 8; ++c)
            if (at[i] + c < a.dim) {
                if (a.shared_gate) slot[at[i] + c] = sg[i][c];
                if (a.post) slot[a.dim + at[i] + c] = s1[i][c];
                if (a.pre) slot[2 * a.dim + at[i] + c] = s2[i][c];
            }
}

struct SumArgs {
    const float *slots;
    float *out[3];  // of the gate, the norm after, the norm before; null: not wanted
    int dim, blocks;
};

// Adds the workgroups' sums up: 64 columns to a workgroup, its four waves taking
// every fourth slot.
__global__ __launch_bounds__(256) void k_block_norm_sums(SumArgs a) {
    __shared__ float part[4][64];
    const int per = (a.dim + 63) / 64, which = blockIdx.x / per;
    const int c = blockIdx.x % per * 64 + threadIdx.x % 64, wave = threadIdx.x / 64;
    float *out = a.out[which];
    if (!out) return;
    float t = 0;
    if (c < a.dim) {
        const float *p = a.slots + (int64_t)which * a.dim + c;
        for (int s = wave; s < a.blocks; s += 4 * 16) {
            float v[16];  // all on their way at once
#pragma unroll
            for (int k = 0; k < 16; ++k) v[k] = p[(int64_t)min(s + 4 * k, a.blocks - 1) * 3 * a.dim];
#pragma unroll
            for (int k = 0; k < 16; ++k) t += s + 4 * k < a.blocks ? v[k] : 0.0f;
        }
    }
    part[wave][threadIdx.x % 64] = t;
    __syncthreads();
    if (wave == 0 && c < a.dim) out[c] = (part[0][threadIdx.x] + part[1][threadIdx.x]) + (part[2][threadIdx.x] + part[3][threadIdx.x]);
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

const void *pick_grad(bool wide, bool stream) {
    return wide ? (stream ? reinterpret_cast<const void *>(&k_block_norm_grad<2, true>) : reinterpret_cast<const void *>(&k_block_norm_grad<2, false>))
                : (stream ? reinterpret_cast<const void *>(&k_block_norm_grad<1, true>) : reinterpret_cast<const void *>(&k_block_norm_grad<1, false>));
}

bool is_wide(int dim) { return dim > 8 * kMaxThreads; }

unsigned threads_of(int dim) {
    const int vecs = (dim + 7) / 8, lanes = is_wide(dim) ? (vecs + 1) / 2 : vecs;
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

constexpr int kSlots = 256;  // workgroups backwards, at most: one a compute unit

int grad_blocks(int64_t tokens) { return (int)(tokens < 1 ? 1 : tokens < kSlots ? tokens : kSlots); }

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
    const int64_t bytes = 2 * tokens * dim * (P + 3);
    return launch(pick(P, is_wide(dim), bytes > kStreamBytes), (unsigned)tokens, threads_of(dim), a, stream);
}

int64_t ar_block_norm_bwd_workspace(int64_t tokens, int dim) {
    if (!valid_shape(tokens, dim)) return AR_EINVAL;
    return round_up((int64_t)grad_blocks(tokens) * 3 * dim * 4, 16);
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
    SumArgs sum = {static_cast<const float *>(workspace),
                   {static_cast<float *>(sums[0]), static_cast<float *>(sums[1]), static_cast<float *>(sums[2])},
                   dim,
                   tokens ? grad_blocks(tokens) : 0};
    if (tokens > 0) {
        BlockArgs a = {};
        a.part[0] = static_cast<const uint16_t *>(y.p), a.part_stride = ry.r.token_stride;
        a.x = rows(rx), a.dx = rows(rdx), a.dy = rows(rdy);
        if (h_grad.p) a.h = rows(rdh);
        if (pre_weight) a.z = rows(rdz);
        if (gate.p) a.gate = rows(rg);
        if (gate_rows) a.dgate = rows(rdg);
        a.post = static_cast<const uint16_t *>(post_weight), a.pre = static_cast<const uint16_t *>(pre_weight);
        a.slots = static_cast<float *>(workspace);
        a.shared_gate = shared;
        a.tokens = tokens, a.dim = dim, a.scale = residual_scale, a.eps = eps;
        const int64_t bytes = 2 * tokens * dim * 6;
        const int rc = launch(pick_grad(is_wide(dim), bytes > kStreamBytes), (unsigned)grad_blocks(tokens), threads_of(dim), a, stream);
        if (rc != AR_OK) return rc;
    }
    if (!wanted) return AR_OK;
    return launch(reinterpret_cast<const void *>(&k_block_norm_sums), (unsigned)(3 * ((dim + 63) / 64)), 256, sum, stream);
}

}  // extern "C"
