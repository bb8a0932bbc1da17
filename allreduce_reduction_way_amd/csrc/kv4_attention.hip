// kv4_attention.hip -- attention over a paged cache held in 4 bits: steps of
// single tokens, drafted tokens, and chunks of prompts.
//
// For query i of a sequence of n cached tokens whose last m are its own, at
// position p = n - m + i, over tokens j <= p (and j > p - window):
//     s_j = scale q . k_j,   out = sum_j exp(s_j) v_j / sum_j exp(s_j).
// One pass over the tokens with a running maximum and sum.
//
// Rows of the matrix products are the (query, head) pairs that share a key
// head, sixteen to a row tile, and one wave holds R row tiles.  All products
// are done by the matrix unit in tiles of 16 rows x 32 tokens:
//
// Scores, transposed: S^T = K Q^T.  K goes in as it is stored, E2M1 codes with
// their scales, without any conversion.  Q is split into two e4m3 parts,
// q = h 2^x + l 2^(x-5) with one x for the row: h is q rounded to four bits
// and l what is left, which for a bf16 of eight bits is exact until l falls
// below the smallest e4m3 number, 2^-21 of the row's largest element.  So the
// scores are as good as a product in binary32, for two products of the fast
// kind.
//
// Output, transposed: O^T = V^T P^T with P rounded to bf16 (half a step, 2^-8,
// of each weight; the sum of weights is kept unrounded) and V's codes turned
// into bf16 exactly.  The lane that the score product leaves a weight in is
// the lane that this product takes it from, because the order of K's scales in
// the cache gives token rows 4 a + i of the first sixteen and the second
// sixteen to tokens 8 a + i and 8 a + 4 + i: P never moves between lanes.  The
// statistics of a row are in the lanes that hold its output, too.
//
// A step of one sequence reads its cache once for few rows: bound by memory.
// The waves of a workgroup then take the tiles of a range of tokens in turn
// and join their results through LDS, several workgroups share a sequence, and
// the last of them to arrive joins theirs.
#include "host.h"
#include "join.h"
#include "kv4.h"
#include "rows.h"

namespace ar {
namespace {

typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

constexpr int kWaves = kThreads / 64;
constexpr float kNegInf = -__builtin_inff();
constexpr float kLn2 = 0.693147180559945309f, kLog2e = 1.44269504088896341f;

struct AttnArgs {
    Rows q, out;
    const uint8_t *cache;
    const int32_t *table, *q_start, *kv_len;
    float *lse;
    uint32_t *counters;
    float *part;
    int64_t table_stride;
    int tokens, batch, heads, kv_heads, group;
    int pages, per_seq, shift;  // pages of the cache, entries of a table row, log2 of tiles a page
    int window, max_q;
    int blocks;  // row blocks of a sequence's key head
    int splits;  // workgroups that share a row block
    int vec;
    float c;  // scale log2(e)
};

// The codes and scales that a lane takes of one tile.
template <int D>
struct Tile {
    static constexpr int kBlocks = D > 128 ? D / 128 : 1;  // K = 128 products along D
    u32x4 k[2][kBlocks];
    uint32_t ks[kBlocks];
    uint32_t v[D / 16];
    uint32_t vs[2];
    int index;   // tile of the sequence
    bool known;  // its page is one of the cache's
};

template <int D>
__device__ __forceinline__ void load_tile(Tile<D> &t, const AttnArgs &a, const int32_t *pages, int h,
                                          int index, int lane) {
    using L = Kv4<D>;
    const int r = lane % 16, q = lane / 16;
    const int page = pages[index >> a.shift];
    t.index = index;
    t.known = page >= 0 && page < a.pages;
    const int64_t at = (((int64_t)(t.known ? page : 0) * a.kv_heads + h) << a.shift) + (index & ((1 << a.shift) - 1));
    const uint8_t *p = a.cache + at * L::kBytes;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int tok = r / 4 * 8 + i * 4 + r % 4;
#pragma unroll
        for (int b = 0; b < Tile<D>::kBlocks; ++b)
            t.k[i][b] = *reinterpret_cast<const u32x4 *>(p + L::k_code(tok, D == 64 ? q % 2 * 32 : b * 128 + q * 32));
    }
#pragma unroll
    for (int b = 0; b < Tile<D>::kBlocks; ++b)
        t.ks[b] = *reinterpret_cast<const uint16_t *>(p + L::kKScale + ((D == 64 ? q % 2 : b * 4 + q) * 16 + r) * 2);
    const u32x4 *v = reinterpret_cast<const u32x4 *>(p + L::kV + lane % 16 * (4 * L::W) + q * (64 * L::W));
#pragma unroll
    for (int i = 0; i < D / 64; ++i) {
        const u32x4 w = v[i];
#pragma unroll
        for (int j = 0; j < 4; ++j) t.v[i * 4 + j] = w[j];
    }
    const uint2 s = *reinterpret_cast<const uint2 *>(p + L::kVScale + (q * L::G + r * L::W / kGroup) * 8);
    t.vs[0] = s.x, t.vs[1] = s.y;
}

// Sixteen rows of queries as the score product takes them: D/4 channels of row
// lane % 16 in each lane, in two e4m3 parts.
template <int D>
struct Query {
    static constexpr int kWords = D / 16;  // words of each part
    uint32_t hi[kWords], lo[kWords];
    uint32_t scale;  // the parts' scale bytes: hi in byte 0, lo in byte 1

    __device__ __forceinline__ void load(const uint16_t *row, int lane, bool vec) {
        const int q = lane / 16;
        float x[D / 4];
        uint32_t most = 0;
#pragma unroll
        for (int i = 0; i < D / 64; ++i) {  // runs of sixteen channels
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const uint16_t *p = row + i * 64 + q * 16 + j * 8;
                const u32x4 w = vec ? load8<true>(p) : load8<false>(p);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    most = max(most, max((w[e] << 16) & 0x7FFFFFFFu, w[e] & 0x7FFF0000u));
                    x[i * 16 + j * 8 + 2 * e] = lo_f32(w[e]);
                    x[i * 16 + j * 8 + 2 * e + 1] = hi_f32(w[e]);
                }
            }
        }
        most = max(most, (uint32_t)__shfl_xor((int)most, 16));
        most = max(most, (uint32_t)__shfl_xor((int)most, 32));
        // the largest lands in [128, 256) of 448; tiny rows keep a scale that
        // the lower part's can follow
        const uint32_t e = max(most >> 23, 12u);
        const float up = __uint_as_float((254u + 7u - min(e, 254u)) << 23);
#pragma unroll
        for (int i = 0; i < kWords; ++i) {
            float y[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) y[j] = x[4 * i + j] * up;
            int w = __builtin_amdgcn_cvt_pk_fp8_f32(y[0], y[1], 0, false);
            w = __builtin_amdgcn_cvt_pk_fp8_f32(y[2], y[3], w, true);
            hi[i] = (uint32_t)w;
            y[0] = (y[0] - __builtin_amdgcn_cvt_f32_fp8(w, 0)) * 32.0f;
            y[1] = (y[1] - __builtin_amdgcn_cvt_f32_fp8(w, 1)) * 32.0f;
            y[2] = (y[2] - __builtin_amdgcn_cvt_f32_fp8(w, 2)) * 32.0f;
            y[3] = (y[3] - __builtin_amdgcn_cvt_f32_fp8(w, 3)) * 32.0f;
            w = __builtin_amdgcn_cvt_pk_fp8_f32(y[0], y[1], 0, false);
            w = __builtin_amdgcn_cvt_pk_fp8_f32(y[2], y[3], w, true);
            lo[i] = (uint32_t)w;
        }
        // a row that is not finite has no scores: NaN
        scale = most >= 0x7F800000u ? 0xFFFFu : (e - 7u) | (e - 12u) << 8;
        // at 64 channels one product takes both parts, a K of 64 each: its
        // scales are the lanes' halves
        if (D == 64) scale = q < 2 ? scale & 0xFFu : scale >> 8;
    }
};

__device__ __forceinline__ i32x8 codes8(u32x4 v) {
    return i32x8{(int)v[0], (int)v[1], (int)v[2], (int)v[3], 0, 0, 0, 0};
}

__device__ __forceinline__ i32x8 words8(const uint32_t *a, const uint32_t *b) {
    return i32x8{(int)a[0], (int)a[1], (int)a[2], (int)a[3], (int)b[0], (int)b[1], (int)b[2], (int)b[3]};
}

constexpr int kFp4 = 4, kFp8 = 0;  // operand formats of the scaled product

template <int H, int PART>
__device__ __forceinline__ f32x4 score_step(i32x8 k, i32x8 q, f32x4 s, uint32_t ks, uint32_t qs) {
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(k, q, s, kFp4, kFp8, H, (int)ks, PART, (int)qs);
}

// Scores of a row tile against tokens 8 a + 4 H + i of a tile, i = 0..3.
template <int D, int H>
__device__ __forceinline__ f32x4 scores(const Tile<D> &t, const Query<D> &q) {
    f32x4 s = {0, 0, 0, 0};
    if (D == 64) return score_step<H, 0>(codes8(t.k[H][0]), words8(q.hi, q.lo), s, t.ks[0], q.scale);
#pragma unroll
    for (int b = 0; b < Tile<D>::kBlocks; ++b) {
        s = score_step<H, 0>(codes8(t.k[H][b]), words8(q.hi + 8 * b, q.hi + 8 * b + 4), s, t.ks[b], q.scale);
        s = score_step<H, 1>(codes8(t.k[H][b]), words8(q.lo + 8 * b, q.lo + 8 * b + 4), s, t.ks[b], q.scale);
    }
    return s;
}

// V of a tile as the output product takes it: block j holds channel r W + j of
// tokens 8 a .. 8 a + 7.
template <int D>
struct Values {
    uint32_t w[Kv4<D>::W][4];

    __device__ __forceinline__ void load(const Tile<D> &t) {
        constexpr int W = Kv4<D>::W;
#pragma unroll
        for (int n = 0; n < 4; ++n) {  // tokens 2 n and 2 n + 1
            const float s0 = kv4_scale((t.vs[n / 2] >> (n % 2 * 16)) & 255u);
            const float s1 = kv4_scale((t.vs[n / 2] >> (n % 2 * 16 + 8)) & 255u);
#pragma unroll
            for (int j = 0; j < W; j += 2) {
                const int b0 = (2 * n * W + j) / 2, b1 = b0 + W / 2;
                const uint32_t x = kv4_pair(t.v[b0 / 4], s0, b0 % 4), y = kv4_pair(t.v[b1 / 4], s1, b1 % 4);
                w[j][n] = __builtin_amdgcn_perm(y, x, 0x05040100u);
                w[j + 1][n] = __builtin_amdgcn_perm(y, x, 0x07060302u);
            }
        }
    }
};

__device__ __forceinline__ bf16x8 as_bf16(const uint32_t (&w)[4]) {
    return __builtin_bit_cast(bf16x8, u32x4{w[0], w[1], w[2], w[3]});
}

__device__ __forceinline__ uint32_t bf16_pair(float lo, float hi) {
    bf16x2 r;
    r[0] = (__bf16)lo;
    r[1] = (__bf16)hi;
    return __builtin_bit_cast(uint32_t, r);
}

// A byte of 255 among four.
__device__ __forceinline__ bool any_nan_scale(uint32_t w) {
    const uint32_t z = ~w;
    return ((z - 0x01010101u) & ~z & 0x80808080u) != 0;
}

// A row tile's running result: the maximum (in units of log2) and the sum of
// weights of row lane % 16, and its output: acc[j][i] is channel
// (4 a + i) W + j.
template <int D>
struct RowTile {
    static constexpr int W = Kv4<D>::W;
    float m, l;
    f32x4 acc[W];

    __device__ __forceinline__ void clear() {
        m = kNegInf, l = 0;
#pragma unroll
        for (int j = 0; j < W; ++j) acc[j] = f32x4{0, 0, 0, 0};
    }
    __device__ __forceinline__ void rescale(float by) {
        l *= by;
#pragma unroll
        for (int j = 0; j < W; ++j) acc[j] *= by;
    }
    // The weight of a result with maximum `mine` where the joint one is `all`.
    static __device__ __forceinline__ float weight(float mine, float all) {
        return __builtin_amdgcn_exp2f(mine - (all == kNegInf ? 0.0f : all));
    }
};

template <int D, int R>
struct State {
    RowTile<D> row[R];
    Query<D> q[R];
    int pos[R];  // position of this lane's row
};

// One tile.  MASKED: some of its tokens are unseen by some rows.
template <int D, int R, bool MASKED>
__device__ __forceinline__ void step(State<D, R> &st, Tile<D> &t, const AttnArgs &a, int lane) {
    constexpr int W = Kv4<D>::W;
    bool nan_values = false;
    uint32_t flag[4] = {0, 0, 0, 0};  // 1 for each token whose V scale stands for NaN
    if (MASKED) {
        // a token that a row does not see adds nothing to it, whatever V holds:
        // NaNs are taken out here and given to the rows that see them
        nan_values = __any(any_nan_scale(t.vs[0]) || any_nan_scale(t.vs[1]));
        if (nan_values) {
#pragma unroll
            for (int n = 0; n < 8; ++n)
                if (((t.vs[n / 4] >> (n % 4 * 8)) & 255u) == 255u) {
                    flag[n / 2] |= 0x3F80u << (n % 2 * 16);
                    t.vs[n / 4] &= ~(255u << (n % 4 * 8));
                }
        }
    }
    Values<D> v;
    v.load(t);
#pragma unroll
    for (int r = 0; r < R; ++r) {
        RowTile<D> &o = st.row[r];
        f32x4 s[2] = {scores<D, 0>(t, st.q[r]), scores<D, 1>(t, st.q[r])};
        uint32_t seen[4] = {0, 0, 0, 0};
        if (MASKED) {
            const int first = t.index * kTile + lane / 16 * 8;
#pragma unroll
            for (int n = 0; n < 8; ++n) {
                const int j = first + n;
                const bool see = j <= st.pos[r] && (a.window == 0 || st.pos[r] - j < a.window);
                if (!see) s[n / 4][n % 4] = kNegInf;
                if (see) seen[n / 2] |= 0x3F80u << (n % 2 * 16);
            }
        }
        float top = s[0][0];
#pragma unroll
        for (int n = 1; n < 8; ++n) top = fmaxf(top, s[n / 4][n % 4]);
        top = fmaxf(top, __shfl_xor(top, 16));
        top = fmaxf(top, __shfl_xor(top, 32));
        const float m = fmaxf(o.m, top * a.c);
        const float base = m == kNegInf ? 0.0f : m;
        o.rescale(__builtin_amdgcn_exp2f(o.m - base));
        o.m = m;
        float p[8];
#pragma unroll
        for (int n = 0; n < 8; ++n) {
            p[n] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[n / 4][n % 4], a.c, -base));
            o.l += p[n];
        }
        const uint32_t w[4] = {bf16_pair(p[0], p[1]), bf16_pair(p[2], p[3]), bf16_pair(p[4], p[5]), bf16_pair(p[6], p[7])};
        const bf16x8 pb = as_bf16(w);
#pragma unroll
        for (int j = 0; j < W; ++j)
            o.acc[j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(as_bf16(v.w[j]), pb, o.acc[j], 0, 0, 0);
        if (MASKED && nan_values) {
            const f32x4 z = {0, 0, 0, 0};
            const f32x4 n = __builtin_amdgcn_mfma_f32_16x16x32_bf16(as_bf16(flag), as_bf16(seen), z, 0, 0, 0);
#pragma unroll
            for (int j = 0; j < W; ++j)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (n[i] > 0) o.acc[j][i] = __uint_as_float(0x7FC00000u);
        }
    }
}

// The rows of a block, where they lie, and the tiles that they see.
struct Block {
    int seq, head, first, rows;  // rows: of the sequence's key head, first: of this block
    int q0, n, len;              // first query token; cached tokens; queries
    int lo, hi;                  // tiles [lo, hi)
    int seen_lo, seen_hi;        // tokens that every row sees: [seen_lo, seen_hi)
};

__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }

__device__ __forceinline__ bool locate(Block &b, const AttnArgs &a, int seq, int head, int block, int size) {
    const int q0 = min(max(a.q_start[seq], 0), a.tokens), q1 = min(max(a.q_start[seq + 1], q0), a.tokens);
    b.seq = seq, b.head = head;
    b.q0 = q0, b.len = q1 - q0;
    // 31 bits hold the tokens of a table row: checked on the host
    b.n = min(max(a.kv_len[seq], 0), a.per_seq << (a.shift + 5));
    b.rows = min(b.len, a.max_q) * a.group;
    b.first = block * size;
    if (b.first >= b.rows) return false;
    const int lowest = b.n - b.len + b.first / a.group;
    const int highest = b.n - b.len + (min(b.rows, b.first + size) - 1) / a.group;
    const int from = a.window ? (int)max((int64_t)0, (int64_t)lowest - a.window + 1) : 0;
    b.lo = from / kTile;
    b.hi = highest >= from ? highest / kTile + 1 : b.lo;
    b.seen_lo = a.window ? (int)max((int64_t)0, (int64_t)highest - a.window + 1) : 0;
    b.seen_hi = lowest + 1;
    return true;
}

template <int D, int R>
__device__ __forceinline__ void begin(State<D, R> &st, const AttnArgs &a, const Block &b, int lane) {
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const int row = min(b.first + r * 16 + lane % 16, b.rows - 1);  // rows past the last repeat it
        const int i = row / a.group, h = b.head * a.group + row % a.group;
        st.q[r].load(a.q.p + (int64_t)(b.q0 + i) * a.q.ts + (int64_t)h * a.q.hs, lane, a.vec);
        st.pos[r] = b.n - b.len + i;
        st.row[r].clear();
    }
}

// Tiles lo, lo + by, ... below hi.
template <int D, int R>
__device__ __forceinline__ void sweep(State<D, R> &st, const AttnArgs &a, const Block &b, int lo, int hi, int by, int lane) {
    if (lo >= hi) return;
    const int32_t *pages = a.table + (int64_t)b.seq * a.table_stride;
    Tile<D> now, next;
    load_tile(now, a, pages, b.head, lo, lane);
    for (int t = lo; t < hi; t += by) {
        load_tile(next, a, pages, b.head, t + by < hi ? t + by : t, lane);
        if (now.known) {
            if (t * kTile >= b.seen_lo && (t + 1) * kTile <= b.seen_hi)
                step<D, R, false>(st, now, a, lane);
            else
                step<D, R, true>(st, now, a, lane);
        }
        now = next;
    }
#pragma unroll
    for (int r = 0; r < R; ++r) {  // each lane has added its own tokens
        st.row[r].l += __shfl_xor(st.row[r].l, 16);
        st.row[r].l += __shfl_xor(st.row[r].l, 32);
    }
}

__device__ __forceinline__ float log_sum(float m, float l) {
    return l == 0 ? kNegInf : (m + log2f(l)) * kLn2;
}

// Writes a row tile's rows: an unseen row gives zeros.
template <int D>
__device__ __forceinline__ void finish(const RowTile<D> &o, const AttnArgs &a, const Block &b, int r, int lane) {
    constexpr int W = Kv4<D>::W;
    const int row = b.first + r * 16 + lane % 16;
    if (row >= b.rows) return;
    const int i = row / a.group, h = b.head * a.group + row % a.group;
    const int64_t token = b.q0 + i;
    const float inv = o.l == 0 ? 0.0f : 1.0f / o.l;
    uint16_t *p = const_cast<uint16_t *>(a.out.p) + token * a.out.ts + (int64_t)h * a.out.hs + lane / 16 * (4 * W);
#pragma unroll
    for (int k = 0; k < W / 2; ++k) {  // eight channels each
        u32x4 w;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int c = k * 8 + e * 2;
            w[e] = pack_bf16x2(o.acc[c % W][c / W] * inv, o.acc[c % W + 1][c / W] * inv);
        }
        if (a.vec) store8<true>(p + k * 8, w);
        else store8<false>(p + k * 8, w);
    }
    if (lane < 16) a.lse[token * a.heads + h] = log_sum(o.m, o.l);
}

// Many rows: every wave has a row block of its own and sweeps all its tiles.
template <int D, int R>
__global__ __launch_bounds__(kThreads) void k_kv4_attention_wide(AttnArgs a) {
    const int lane = threadIdx.x % 64, wave = uniform(threadIdx.x / 64);
    const int per = (a.blocks + kWaves - 1) / kWaves;
    const int id = blockIdx.x;
    const int unit = id / per, block = id % per * kWaves + wave;
    Block b;
    if (block >= a.blocks || !locate(b, a, unit % a.batch, unit / a.batch, block, 16 * R)) return;
    State<D, R> st;
    begin(st, a, b, lane);
    sweep(st, a, b, b.lo, b.hi, 1, lane);
#pragma unroll
    for (int r = 0; r < R; ++r) finish(st.row[r], a, b, r, lane);
}

// Few rows: the waves of a workgroup share a row block.
template <int D, int R>
__global__ __launch_bounds__(kThreads) void k_kv4_attention(AttnArgs a) {
    constexpr int W = Kv4<D>::W;
    __shared__ f32x4 acc[kWaves / 2][R][W][64];
    __shared__ float ml[kWaves / 2][R][2][16];
    __shared__ uint32_t order;
    const int lane = threadIdx.x % 64, wave = uniform(threadIdx.x / 64);
    const int split = blockIdx.x % a.splits, unit = blockIdx.x / a.splits;
    const int pair = unit / a.blocks;
    Block b;
    if (!locate(b, a, pair / a.kv_heads, pair % a.kv_heads, unit % a.blocks, 16 * R)) return;
    // the tiles in equal ranges, none shorter than a tile for each wave
    const int tiles = b.hi - b.lo;
    const int chunk = max(kWaves, (tiles + a.splits - 1) / a.splits);
    const int count = max(1, (tiles + chunk - 1) / chunk);
    if (split >= count) return;
    State<D, R> st;
    begin(st, a, b, lane);
    const int lo = b.lo + split * chunk;
    sweep(st, a, b, lo + wave, min(b.hi, lo + chunk), kWaves, lane);

    // the upper half of the waves hands its results to the lower half
#pragma unroll
    for (int half = kWaves / 2; half > 0; half /= 2) {
        if (wave >= half && wave < 2 * half) {
#pragma unroll
            for (int r = 0; r < R; ++r) {
#pragma unroll
                for (int j = 0; j < W; ++j) acc[wave - half][r][j][lane] = st.row[r].acc[j];
                if (lane < 16) ml[wave - half][r][0][lane] = st.row[r].m, ml[wave - half][r][1][lane] = st.row[r].l;
            }
        }
        __syncthreads();
        if (wave < half) {
#pragma unroll
            for (int r = 0; r < R; ++r) {
                RowTile<D> &o = st.row[r];
                const float m2 = ml[wave][r][0][lane % 16], l2 = ml[wave][r][1][lane % 16];
                const float m = fmaxf(o.m, m2), w1 = o.weight(o.m, m), w2 = o.weight(m2, m);
                o.m = m;
                o.l = o.l * w1 + l2 * w2;
#pragma unroll
                for (int j = 0; j < W; ++j) o.acc[j] = o.acc[j] * w1 + acc[wave][r][j][lane] * w2;
            }
        }
        __syncthreads();
    }
    if (count == 1) {
        if (wave == 0) {
#pragma unroll
            for (int r = 0; r < R; ++r) finish(st.row[r], a, b, r, lane);
        }
        return;
    }

    // results of a split: R W 64 vectors as the lanes hold them, then the
    // maxima and sums
    constexpr int kPart = R * W * 256 + R * 32;
    float *base = a.part + (int64_t)unit * a.splits * kPart;
    if (wave == 0) {
        float *p = base + (int64_t)split * kPart;
#pragma unroll
        for (int r = 0; r < R; ++r) {
            if (b.first + r * 16 + lane % 16 < b.rows) {
#pragma unroll
                for (int j = 0; j < W; ++j) reinterpret_cast<f32x4 *>(p)[(r * W + j) * 64 + lane] = st.row[r].acc[j];
                if (lane < 16) {
                    p[R * W * 256 + r * 32 + lane] = st.row[r].m;
                    p[R * W * 256 + r * 32 + 16 + lane] = st.row[r].l;
                }
            }
        }
    }
    if (!arrive_last(a.counters + unit, count, &order)) return;
    for (int r = wave; r < R; r += kWaves) {
        if (b.first + r * 16 + lane % 16 >= b.rows) continue;
        RowTile<D> o;
        o.clear();
        for (int s = 0; s < count; ++s) {
            const float *p = base + (int64_t)s * kPart;
            const float m2 = p[R * W * 256 + r * 32 + lane % 16], l2 = p[R * W * 256 + r * 32 + 16 + lane % 16];
            const float m = fmaxf(o.m, m2), w1 = o.weight(o.m, m), w2 = o.weight(m2, m);
            o.m = m;
            o.l = o.l * w1 + l2 * w2;
#pragma unroll
            for (int j = 0; j < W; ++j)
                o.acc[j] = o.acc[j] * w1 + reinterpret_cast<const f32x4 *>(p)[(r * W + j) * 64 + lane] * w2;
        }
        finish(o, a, b, r, lane);
    }
}

constexpr int kCounters = 16384;  // counters at the start of the workspace
constexpr int kSplits = 32;       // workgroups that share a row block, at most
constexpr int kFill = 1024;       // workgroups that fill the device: four on each compute unit

// How a call is laid out, by its sizes alone.
struct Plan {
    bool wide;
    int tiles;  // row tiles of a wave
    int blocks, splits;
    int64_t units;
};

Plan plan(int batch, int max_q, int64_t max_kv, int group, int kv_heads, int dim) {
    Plan p = {};
    const int64_t rows = (int64_t)max_q * group, tiles = (rows + 15) / 16;
    const int most = dim > 128 ? 1 : 4;
    p.tiles = (int)(tiles < most ? tiles : most);
    p.blocks = (int)((tiles + p.tiles - 1) / p.tiles);
    p.units = (int64_t)batch * kv_heads * p.blocks;
    p.wide = p.blocks >= kWaves && p.units >= kFill;
    p.splits = 1;
    if (p.wide || p.units >= kFill) return p;
    const int64_t steps = (max_kv + kTile - 1) / kTile;
    int64_t s = (kFill + p.units - 1) / p.units;
    if (s > steps / (2 * kWaves)) s = steps / (2 * kWaves);
    if (s > kSplits) s = kSplits;
    p.splits = s < 1 ? 1 : (int)s;
    return p;
}

int64_t part_floats(const Plan &p, int dim) { return (int64_t)p.tiles * (dim / 16 * 256 + 32); }

bool valid_sizes(int64_t batch, int64_t tokens, int64_t max_q, int64_t max_kv, int heads, int kv_heads, int dim) {
    return batch >= 0 && batch <= 1 << 20 && tokens >= 0 && tokens <= 1 << 28 && max_q >= 0 &&
           max_q <= 1 << 24 && max_kv >= 0 && max_kv <= 0x7FFFFFFF && kv_heads >= 1 &&
           kv_heads <= 1 << 12 && heads >= 1 && heads <= 1 << 14 && heads % kv_heads == 0 &&
           max_q * heads <= 1 << 30 &&
           (dim == 64 || dim == 128 || dim == 256);
}

#define AR_NARROW(D_, R_) \
    case R_: return reinterpret_cast<const void *>(&k_kv4_attention<D_, R_>);

const void *pick(const Plan &p, int dim) {
    if (p.wide) {
        switch (dim) {
            case 64: return reinterpret_cast<const void *>(&k_kv4_attention_wide<64, 4>);
            case 128: return reinterpret_cast<const void *>(&k_kv4_attention_wide<128, 4>);
            default: return reinterpret_cast<const void *>(&k_kv4_attention_wide<256, 1>);
        }
    }
    switch (dim) {
        case 64:
            switch (p.tiles) { AR_NARROW(64, 1) AR_NARROW(64, 2) AR_NARROW(64, 3) AR_NARROW(64, 4) }
            break;
        case 128:
            switch (p.tiles) { AR_NARROW(128, 1) AR_NARROW(128, 2) AR_NARROW(128, 3) AR_NARROW(128, 4) }
            break;
        default:
            switch (p.tiles) { AR_NARROW(256, 1) }
    }
    return nullptr;
}

}  // namespace
}  // namespace ar

using namespace ar;

extern "C" {

int64_t ar_kv4_attention_workspace(int64_t batch, int64_t tokens, int64_t max_q, int64_t max_kv,
                                   int heads, int kv_heads, int dim) {
    if (!valid_sizes(batch, tokens, max_q, max_kv, heads, kv_heads, dim)) return AR_EINVAL;
    if (batch == 0 || max_q == 0) return 4 * kCounters;
    const Plan p = plan((int)batch, (int)max_q, max_kv, heads / kv_heads, kv_heads, dim);
    return 4 * kCounters + (p.splits > 1 ? p.units * p.splits * part_floats(p, dim) * 4 : 0);
}

int ar_kv4_attention(ar_rows q, const void *cache, const void *page_table, int64_t table_stride,
                     const void *q_start, const void *kv_len, ar_rows out, void *lse, void *workspace,
                     int64_t tokens, int64_t batch, int heads, int kv_heads, int dim, int64_t pages,
                     int page_size, int64_t pages_per_seq, int64_t max_q, int64_t max_kv, int64_t window,
                     float scale, void *stream) {
    int shift = 0;
    if (!valid_sizes(batch, tokens, max_q, max_kv, heads, kv_heads, dim) ||
        !kv4_shape(kv_heads, dim, pages, page_size, &shift) || pages_per_seq < 0 ||
        pages_per_seq > 0x7FFFFFFF / page_size || table_stride < 0 || window < 0 ||
        window > 0x7FFFFFFF || !(scale > 0) || !(scale <= 3.0e38f) ||
        table_stride > ((int64_t)1 << 40) / (batch + 1))
        return AR_EINVAL;
    if (tokens == 0 || batch == 0) return AR_OK;
    const RowsArg rq{q, tokens, heads, dim}, ro{out, tokens, heads, dim};
    if (!rq.valid() || !ro.valid() || ro.self_overlap() || !q_start || !aligned_to(q_start, 4) ||
        !kv_len || !aligned_to(kv_len, 4) || !lse || !aligned_to(lse, 4) || !workspace ||
        !aligned_to(workspace, 16) || (pages > 0 && (!cache || !aligned_to(cache, 16))) ||
        (pages_per_seq > 0 && (!page_table || !aligned_to(page_table, 4))) || max_q < 1)
        return AR_EINVAL;
    const Span reads[] = {rq.span(),
                          {addr(cache), (uintptr_t)kv4_bytes(kv_heads, dim, pages, page_size)},
                          {addr(page_table), (uintptr_t)(pages_per_seq ? 4 * ((batch - 1) * table_stride + pages_per_seq) : 0)},
                          {addr(q_start), (uintptr_t)(4 * (batch + 1))},
                          {addr(kv_len), (uintptr_t)(4 * batch)}};
    const Span writes[] = {ro.span(),
                           {addr(lse), (uintptr_t)(4 * tokens * heads)},
                           {addr(workspace), (uintptr_t)ar_kv4_attention_workspace(batch, tokens, max_q, max_kv, heads, kv_heads, dim)}};
    for (int i = 0; i < 3; ++i) {
        for (const Span &r : reads)
            if (overlap(writes[i], r)) return AR_EALIAS;
        for (int j = i + 1; j < 3; ++j)
            if (overlap(writes[i], writes[j])) return AR_EALIAS;
    }
    const Plan p = plan((int)batch, (int)max_q, max_kv, heads / kv_heads, kv_heads, dim);
    AttnArgs a = {};
    a.q = rows(rq), a.out = rows(ro);
    a.cache = static_cast<const uint8_t *>(cache);
    a.table = static_cast<const int32_t *>(page_table);
    a.q_start = static_cast<const int32_t *>(q_start), a.kv_len = static_cast<const int32_t *>(kv_len);
    a.lse = static_cast<float *>(lse);
    a.counters = static_cast<uint32_t *>(workspace);
    a.part = reinterpret_cast<float *>(a.counters + kCounters);
    a.table_stride = table_stride;
    a.tokens = (int)tokens, a.batch = (int)batch, a.heads = heads, a.kv_heads = kv_heads, a.group = heads / kv_heads;
    a.pages = (int)pages, a.per_seq = pages ? (int)pages_per_seq : 0, a.shift = shift - 5;
    a.window = (int)window, a.max_q = (int)max_q;
    a.blocks = p.blocks, a.splits = p.splits;
    a.vec = rq.vec() && ro.vec();
    a.c = scale * kLog2e;
    const int64_t pairs = batch * kv_heads;
    const int64_t grid = p.wide ? pairs * ((p.blocks + kWaves - 1) / kWaves) : pairs * p.blocks * p.splits;
    if (grid > 0x7FFFFFFF / kThreads) return AR_EINVAL;
    return launch(pick(p, dim), (unsigned)grid, kThreads, a, stream);
}

}  // extern "C"
