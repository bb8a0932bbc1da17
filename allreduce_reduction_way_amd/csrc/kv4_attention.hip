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
// Scores, transposed: S^T = K Q^T, with K's codes turned into bf16, which is
// exact.  (The scaled instructions take codes as they are, against a query in
// two e4m3 parts, for the same time in the matrix unit.  But they align the
// terms of a product to its largest and drop what lies 2^-20 below: scores
// were off by 4e-6 where these are by 3e-8.)
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

// The codes and scales that a lane takes of one tile.  With r = lane % 16 and
// a = lane / 16, of K: D/4 channels of tokens r / 4 * 8 + r % 4 and four on,
// which lie in one group of channels (in two blocks of 128 at D = 256, half a
// group at 64); of V: channels r W .. r W + W - 1 of tokens 8 a .. 8 a + 7.
template <int D>
struct Tile {
    static constexpr int kBlocks = D > 128 ? D / 128 : 1;
    static constexpr int kWords = D / 32 / kBlocks;  // words of K codes in a block
    uint32_t k[2][kBlocks][kWords];
    uint32_t ks[kBlocks];  // scale bytes of the two tokens
    uint32_t v[D / 16];
    uint32_t vs[2];
};

template <int N>
__device__ __forceinline__ void load_words(uint32_t (&w)[N], const uint8_t *p) {
    if (N == 2) {
        const uint2 t = *reinterpret_cast<const uint2 *>(p);
        w[0] = t.x, w[1] = t.y;
        return;
    }
#pragma unroll
    for (int i = 0; i < N / 4; ++i) {
        const u32x4 t = reinterpret_cast<const u32x4 *>(p)[i];
#pragma unroll
        for (int j = 0; j < 4; ++j) w[i * 4 + j] = t[j];
    }
}

template <int D>
__device__ __forceinline__ void load_tile(Tile<D> &t, const uint8_t *p, int lane) {
    using L = Kv4<D>;
    const int r = lane % 16, q = lane / 16;
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int b = 0; b < Tile<D>::kBlocks; ++b)
            load_words(t.k[i][b], p + L::k_code(r / 4 * 8 + i * 4 + r % 4, D == 64 ? q * 16 : b * 128 + q * 32));
#pragma unroll
    for (int b = 0; b < Tile<D>::kBlocks; ++b)
        t.ks[b] = *reinterpret_cast<const uint16_t *>(p + L::kKScale + ((D == 64 ? q / 2 : b * 4 + q) * 16 + r) * 2);
    load_words(t.v, p + L::kV + lane * (4 * L::W));
    load_words(t.vs, p + L::kVScale + (q * L::G + r * L::W / kGroup) * 8);
}

// Byte n of the scales as a scale.  The conversions take the exponent's bits
// alone, so what else a shift leaves in the word does no harm.
template <int N>
__device__ __forceinline__ float scale_at(const uint32_t (&w)[N], int n) {
    return n % 4 == 3 ? __uint_as_float(w[n / 4] >> 1) : __uint_as_float(w[n / 4] << (23 - n % 4 * 8));
}

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
    uint32_t q[R][D / 32][4];  // D/4 channels of row lane % 16, in K's order
    int pos[R];                // position of this lane's row
};

// How far the weights may outgrow 1 (in units of log2) before a new maximum is
// taken: bf16 and binary32 lose nothing up to there, and most tiles move the
// maximum by less, so that rescaling the output is rare.
constexpr float kSlack = 8.0f;

__device__ __forceinline__ bool sees(int pos, int token, int window) {
    return token <= pos && (window == 0 || pos - token < window);
}

// One tile.  `masked` (the same in all lanes): some of its tokens are unseen by
// some rows.
template <int D, int R>
__device__ __forceinline__ void step(State<D, R> &st, Tile<D> &t, int index, bool masked, const AttnArgs &a, int lane) {
    constexpr int W = Kv4<D>::W;
    using T = Tile<D>;
    bool nan_values = false;
    uint32_t flag[4] = {0, 0, 0, 0};  // 1 for each token whose V scale stands for NaN
    if (masked) {
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
    f32x4 s[R][2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
#pragma unroll
        for (int r = 0; r < R; ++r) s[r][h] = f32x4{0, 0, 0, 0};
#pragma unroll
        for (int n = 0; n < D / 32; ++n) {
            const uint32_t ks[1] = {t.ks[n / T::kWords]};
            const float scale = scale_at(ks, h);
            uint32_t k[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) k[e] = kv4_pair(t.k[h][n / T::kWords][n % T::kWords], scale, e);
#pragma unroll
            for (int r = 0; r < R; ++r)
                s[r][h] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(as_bf16(k), as_bf16(st.q[r][n]), s[r][h], 0, 0, 0);
        }
    }
    uint32_t p[R][4];
    const int first = index * kTile + lane / 16 * 8;  // this lane's first token
#pragma unroll
    for (int r = 0; r < R; ++r) {
        RowTile<D> &o = st.row[r];
        if (masked) {
#pragma unroll
            for (int n = 0; n < 8; ++n)
                if (!sees(st.pos[r], first + n, a.window)) s[r][n / 4][n % 4] = kNegInf;
        }
        float top = s[r][0][0];
#pragma unroll
        for (int n = 1; n < 8; ++n) top = fmaxf(top, s[r][n / 4][n % 4]);
        if (__any(top * a.c > o.m + kSlack)) {
            top = fmaxf(top, __shfl_xor(top, 16));
            top = fmaxf(top, __shfl_xor(top, 32));
            const float m = fmaxf(o.m, top * a.c);
            o.rescale(o.weight(o.m, m));
            o.m = m;
        }
        const float base = o.m == kNegInf ? 0.0f : o.m;
        float w[8];
#pragma unroll
        for (int n = 0; n < 8; ++n) {
            w[n] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[r][n / 4][n % 4], a.c, -base));
            o.l += w[n];
        }
#pragma unroll
        for (int n = 0; n < 4; ++n) p[r][n] = bf16_pair(w[2 * n], w[2 * n + 1]);
    }
#pragma unroll
    for (int j = 0; j < W; j += 2) {
        uint32_t v[2][4];  // channels j and j + 1 of eight tokens
#pragma unroll
        for (int n = 0; n < 4; ++n) {
            const int b0 = (2 * n * W + j) / 2, b1 = b0 + W / 2;
            const uint32_t x = kv4_pair(t.v[b0 / 4], scale_at(t.vs, 2 * n), b0 % 4);
            const uint32_t y = kv4_pair(t.v[b1 / 4], scale_at(t.vs, 2 * n + 1), b1 % 4);
            v[0][n] = __builtin_amdgcn_perm(y, x, 0x05040100u);
            v[1][n] = __builtin_amdgcn_perm(y, x, 0x07060302u);
        }
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
            for (int i = 0; i < 2; ++i)
                st.row[r].acc[j + i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(as_bf16(v[i]), as_bf16(p[r]), st.row[r].acc[j + i], 0, 0, 0);
    }
    if (nan_values) {
#pragma unroll
        for (int r = 0; r < R; ++r) {
            uint32_t seen[4] = {0, 0, 0, 0};
#pragma unroll
            for (int n = 0; n < 8; ++n)
                if (sees(st.pos[r], first + n, a.window)) seen[n / 2] |= 0x3F80u << (n % 2 * 16);
            const f32x4 z = {0, 0, 0, 0};
            const f32x4 n = __builtin_amdgcn_mfma_f32_16x16x32_bf16(as_bf16(flag), as_bf16(seen), z, 0, 0, 0);
#pragma unroll
            for (int j = 0; j < W; ++j)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (n[i] > 0) st.row[r].acc[j][i] = __uint_as_float(0x7FC00000u);
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
    constexpr int kRun = D == 64 ? 16 : 32;  // channels of a lane that lie side by side
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const int row = min(b.first + r * 16 + lane % 16, b.rows - 1);  // rows past the last repeat it
        const int i = row / a.group, h = b.head * a.group + row % a.group;
        const uint16_t *p = a.q.p + (int64_t)(b.q0 + i) * a.q.ts + (int64_t)h * a.q.hs + lane / 16 * kRun;
#pragma unroll
        for (int n = 0; n < D / 32; ++n) {
            const uint16_t *at = p + n / (kRun / 8) * 128 + n % (kRun / 8) * 8;
            const u32x4 w = a.vec ? load8<true>(at) : load8<false>(at);
#pragma unroll
            for (int e = 0; e < 4; ++e) st.q[r][n][e] = w[e];
        }
        st.pos[r] = b.n - b.len + i;
        st.row[r].clear();
    }
}

// Tiles lo, lo + by, ... below hi.  While a tile is worked on, the next one is
// on its way; the pages of 64 tiles are looked up at once, one in each lane.
template <int D, int R>
__device__ __forceinline__ void sweep(State<D, R> &st, const AttnArgs &a, const Block &b, int lo, int hi, int by, int lane) {
    const int32_t *pages = a.table + (int64_t)b.seq * a.table_stride;
    for (int t = lo; t < hi; t += 64 * by) {
        const int count = min(64, (hi - t + by - 1) / by);
        const int page = pages[(t + min(lane, count - 1) * by) >> a.shift];
        Tile<D> now, next;
        const auto at = [&](int i, bool &known) {
            const int pg = __builtin_amdgcn_readlane(page, i);
            known = pg >= 0 && pg < a.pages;
            const int64_t tile = (((int64_t)(known ? pg : 0) * a.kv_heads + b.head) << a.shift) + ((t + i * by) & ((1 << a.shift) - 1));
            return a.cache + tile * Kv4<D>::kBytes;
        };
        bool known, known_next;
        load_tile(now, at(0, known), lane);
        for (int i = 0; i < count; ++i) {
            load_tile(next, at(min(i + 1, count - 1), known_next), lane);
            const int index = t + i * by;
            if (known) {
                const bool masked = index * kTile < b.seen_lo || (index + 1) * kTile > b.seen_hi;
                step<D, R>(st, now, index, masked, a, lane);
            }
            now = next;
            known = known_next;
        }
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

constexpr int kJoinSplits = 16;  // results that one workgroup joins

// Joins `count` results that lie `stride` floats apart: into the output (LAST),
// or into the first of them.  A wave takes pairs of channels of all rows.
template <int D, int R, bool LAST>
__device__ __forceinline__ void join(float *base, int64_t stride, int count, const AttnArgs &a, const Block &b, float *lds, int lane, int wave) {
    constexpr int W = Kv4<D>::W, kStats = R * W * 256;
    float *ms = lds, *ls = lds + kJoinSplits * 16;
    static_assert(kJoinSplits * 32 <= kWaves / 2 * W * 256, "the maxima and sums fit the exchange memory");
    for (int r = 0; r < R; ++r) {
        if (b.first + r * 16 >= b.rows) break;
        __syncthreads();
        for (int i = threadIdx.x; i < count * 16; i += kThreads) {
            const float *p = base + i / 16 * stride + kStats + r * 32 + i % 16;
            const bool used = b.first + r * 16 + i % 16 < b.rows;
            ms[i] = used ? load_shared(p) : kNegInf;
            ls[i] = used ? load_shared(p + 16) : 0.0f;
        }
        __syncthreads();
        const int row = b.first + r * 16 + lane % 16;
        float m = kNegInf, l = 0;
        for (int s = 0; s < count; ++s) m = fmaxf(m, ms[s * 16 + lane % 16]);
        for (int s = 0; s < count; ++s) l += ls[s * 16 + lane % 16] * RowTile<D>::weight(ms[s * 16 + lane % 16], m);
        if (row >= b.rows) continue;
        for (int j = wave * 2; j < W; j += kWaves * 2) {
            float *p = base + ((r * W + j) * 64 + lane) * 4;
            f32x4 sum[2] = {{0, 0, 0, 0}, {0, 0, 0, 0}};
#pragma unroll 8
            for (int s = 0; s < count; ++s) {
                const float w = RowTile<D>::weight(ms[s * 16 + lane % 16], m);
                sum[0] += load_shared4(p + s * stride) * w;
                sum[1] += load_shared4(p + s * stride + 256) * w;
            }
            if (LAST) {
                const int i = row / a.group, h = b.head * a.group + row % a.group;
                const float inv = l == 0 ? 0.0f : 1.0f / l;
                uint16_t *o = const_cast<uint16_t *>(a.out.p) + (int64_t)(b.q0 + i) * a.out.ts + (int64_t)h * a.out.hs + lane / 16 * (4 * W) + j;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const uint32_t w = pack_bf16x2(sum[0][e] * inv, sum[1][e] * inv);
                    if (a.vec) {
                        *reinterpret_cast<uint32_t *>(o + e * W) = w;
                    } else {
                        o[e * W] = (uint16_t)w;
                        o[e * W + 1] = (uint16_t)(w >> 16);
                    }
                }
                if (wave == 0 && j == 0 && lane < 16) a.lse[(int64_t)(b.q0 + i) * a.heads + h] = log_sum(m, l);
            } else {
                store_shared(p, sum[0]);
                store_shared(p + 256, sum[1]);
                if (wave == 0 && j == 0 && lane < 16) {
                    store_shared(base + kStats + r * 32 + lane, m);
                    store_shared(base + kStats + r * 32 + 16 + lane, l);
                }
            }
        }
    }
}

// Many rows: every wave has a row block of its own and sweeps all its tiles.
template <int D, int R>
__global__ __launch_bounds__(kThreads, 2) void k_kv4_attention_wide(AttnArgs a) {
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
__global__ __launch_bounds__(kThreads, 2) void k_kv4_attention(AttnArgs a) {
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

    // A split's result: R W vectors as the lanes hold them, then maxima and
    // sums.  Up to kJoinSplits of them are joined at once; more, in two levels.
    constexpr int kPart = R * W * 256 + R * 32;
    float *base = a.part + (int64_t)unit * a.splits * kPart;
    uint32_t *counter = a.counters + unit * (1 + kJoinSplits);
    if (wave == 0) {
        float *p = base + (int64_t)split * kPart;
#pragma unroll
        for (int r = 0; r < R; ++r) {
            if (b.first + r * 16 + lane % 16 < b.rows) {
#pragma unroll
                for (int j = 0; j < W; ++j) store_shared(p + ((r * W + j) * 64 + lane) * 4, st.row[r].acc[j]);
                if (lane < 16) {
                    store_shared(p + R * W * 256 + r * 32 + lane, st.row[r].m);
                    store_shared(p + R * W * 256 + r * 32 + 16 + lane, st.row[r].l);
                }
            }
        }
    }
    const int groups = (count + kJoinSplits - 1) / kJoinSplits;
    float *scratch = reinterpret_cast<float *>(&acc[0][0][0][0]);
    if (groups > 1) {
        const int g = split / kJoinSplits;
        const int size = min(kJoinSplits, count - g * kJoinSplits);
        if (!arrive_last(counter + 1 + g, size, &order)) return;
        float *p = base + (int64_t)g * kJoinSplits * kPart;
        join<D, R, false>(p, kPart, size, a, b, scratch, lane, wave);
        if (!arrive_last(counter, groups, &order)) return;
        join<D, R, true>(base, (int64_t)kJoinSplits * kPart, groups, a, b, scratch, lane, wave);
    } else {
        if (!arrive_last(counter, count, &order)) return;
        join<D, R, true>(base, kPart, count, a, b, scratch, lane, wave);
    }
}

constexpr int kCounters = 16384;  // counters at the start of the workspace
constexpr int kSplits = kJoinSplits * kJoinSplits;  // workgroups that share a row block, at most
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
    const int most = dim == 64 ? 3 : dim == 128 ? 2 : 1;
    p.tiles = (int)(tiles < most ? tiles : most);
    p.blocks = (int)((tiles + p.tiles - 1) / p.tiles);
    p.units = (int64_t)batch * kv_heads * p.blocks;
    p.wide = p.blocks >= kWaves && p.units >= kFill;
    p.splits = 1;
    if (p.wide || p.units >= kFill || p.units * (1 + kJoinSplits) > kCounters) return p;
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
            case 64: return reinterpret_cast<const void *>(&k_kv4_attention_wide<64, 3>);
            case 128: return reinterpret_cast<const void *>(&k_kv4_attention_wide<128, 2>);
            default: return reinterpret_cast<const void *>(&k_kv4_attention_wide<256, 1>);
        }
    }
    switch (dim) {
        case 64:
            switch (p.tiles) { AR_NARROW(64, 1) AR_NARROW(64, 2) AR_NARROW(64, 3) }
            break;
        case 128:
            switch (p.tiles) { AR_NARROW(128, 1) AR_NARROW(128, 2) }
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
