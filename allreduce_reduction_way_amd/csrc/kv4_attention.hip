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
// Three kernels, by the number of rows alone (plan() below):
//
// k_kv4_attention, few rows: bound by the cache's bytes, or by latency where
// there are few of those.  The waves of a workgroup take the tiles of a range of
// tokens in turn and join their results through LDS, and several workgroups
// share a sequence.  128 sequences of 2048 to 8192 tokens, 8 key heads of 128:
// 731 MB in 146 us, 5.0 TB/s (a copy of 1 GiB runs at 5.1); one sequence of
// 200003 tokens, one key head: 27 MB in 14 us with the join.
//
// k_kv4_join joins the ranges of a row block.
//
// k_kv4_attention_wide, many rows: bound by the issue of vector and matrix
// instructions.  Two chunks of 2048 queries over 8192 and fewer tokens, 32
// heads: 468 GFLOP in 460 us, 1.02 PFLOP/s (a library product of 8192^3 reaches
// 1.16); the matrix unit is busy for 43% of the time.
#include "host.h"
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
    float *part;
    int64_t table_stride;
    int tokens, batch, heads, kv_heads, group;
    int pages, per_seq, shift;  // pages of the cache, entries of a table row, log2 of tiles a page
    int window, max_q;  // window: 2^31 - 1 where there is none
    int blocks;  // row blocks of a sequence's key head
    int splits;  // workgroups that share a row block, at most
    int chunk;   // tiles of such a workgroup, at least
    int waves;   // of such a workgroup
    int vec;
    float c;  // scale log2(e)
};

// The kernel's arguments, read again: what is needed after a sweep is not kept
// in scalar registers during it.  (They did not all fit: those of the drafted
// tokens' kernel were moved to and from vector registers some thirty times a
// tile.)
__device__ __forceinline__ const AttnArgs &again() {
    typedef const __attribute__((address_space(4))) AttnArgs *Args;
    Args p = (Args)__builtin_amdgcn_kernarg_segment_ptr();
    asm volatile("" : "+s"(p));
    return *(const AttnArgs *)p;
}

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

// A tile is addressed by a buffer resource, the same in all lanes, and an
// offset of 32 bits: no addresses of 64 bits are added up in the lanes.
typedef __amdgpu_buffer_rsrc_t TileAddr;

template <int D>
__device__ __forceinline__ TileAddr tile_addr(const uint8_t *p) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t *>(p), (short)0, Kv4<D>::kBytes, 0x00020000);
}

template <int N>
__device__ __forceinline__ void load_words(uint32_t (&w)[N], TileAddr p, uint32_t at) {
    if constexpr (N == 1) {
        w[0] = __builtin_amdgcn_raw_buffer_load_b32(p, at, 0, 0);
    } else if constexpr (N == 2) {
        typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
        const u32x2 t = __builtin_amdgcn_raw_buffer_load_b64(p, at, 0, 0);
        w[0] = t[0], w[1] = t[1];
    } else {
#pragma unroll
        for (int i = 0; i < N / 4; ++i) {
            const u32x4 t = __builtin_amdgcn_raw_buffer_load_b128(p, at + 16 * i, 0, 0);
#pragma unroll
            for (int j = 0; j < 4; ++j) w[i * 4 + j] = t[j];
        }
    }
}

// Where a lane's parts lie in every tile: offsets to the tile's address, which
// is the same in all lanes.
template <int D>
struct Places {
    using L = Kv4<D>;
    uint32_t k, ks, v, vs;
    explicit __device__ __forceinline__ Places(int lane) {
        const int r = lane % 16, q = lane / 16;
        k = L::k_code(r / 4 * 8 + r % 4, D == 64 ? q * 16 : q * 32);
        ks = L::kKScale + ((D == 64 ? q / 2 : q) * 16 + r) * 2;
        v = L::kV + lane * (4 * L::W);
        vs = L::kVScale + (q * L::G + r * L::W / kGroup) * 8;
    }
};

template <int D>
__device__ __forceinline__ void load_tile(Tile<D> &t, const uint8_t *tile, const Places<D> &at) {
    using L = Kv4<D>;
    const TileAddr p = tile_addr<D>(tile);
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int b = 0; b < Tile<D>::kBlocks; ++b) load_words(t.k[i][b], p, at.k + (uint32_t)L::k_code(i * 4, b * 128));
#pragma unroll
    for (int b = 0; b < Tile<D>::kBlocks; ++b) t.ks[b] = (uint16_t)__builtin_amdgcn_raw_buffer_load_b16(p, at.ks + 128u * b, 0, 0);
    load_words(t.v, p, at.v);
    load_words(t.vs, p, at.vs);
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

// A byte from kWildScale on among four: one of their complements below 3.
__device__ __forceinline__ bool any_wild_scale(uint32_t w) {
    static_assert(kWildScale == 253, "the complement's bound");
    return ((~w - 0x03030303u) & w & 0x80808080u) != 0;
}

// A row tile's running result: the maximum (in units of log2) and the sum of
// weights of row lane % 16 (each lane's own tokens until the end of a sweep),
// and its output: acc[j][i] is channel (4 a + i) W + j.
template <int D>
struct RowTile {
    static constexpr int W = Kv4<D>::W;
    float m, l;
    float base, limit;  // m, 0 before there is one; the score from which m has to move (see settle)
    f32x4 d;  // four times the same: the sum of the weights as they were rounded
    f32x4 acc[W];

    __device__ __forceinline__ void clear() {
        m = limit = kNegInf, l = base = 0;
        d = f32x4{0, 0, 0, 0};
#pragma unroll
        for (int j = 0; j < W; ++j) acc[j] = f32x4{0, 0, 0, 0};
    }
    // m is the largest score itself, and limit lies below every score.
    __device__ __forceinline__ bool far() const { return limit == kNegInf && m != kNegInf; }
    // The end of a sweep: each lane has added its own tokens.
    __device__ __forceinline__ void end(float c) {
        if (far()) m *= c;
        l += __shfl_xor(l, 16);
        l += __shfl_xor(l, 32);
    }
    __device__ __forceinline__ void rescale(float by) {
        l *= by;
        d *= by;
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

// A maximum (in units of log2) whose own rounding is a power of two or more.
// From 2^31 on it would be 2^128: weights of finite scores became infinite, or
// all of them 0.
__device__ __forceinline__ bool is_far(float m) { return fabsf(m) > 0x1p24f && m != kNegInf; }

// Tiles that a wave of the split kernel has in its registers: the one that it
// works on and the next.  A third gained nothing: drafted tokens took 19.0 us
// with it and 18.5 without, the long sequence 10.3 and 9.4.
constexpr int kRing = 2;

// The value, which the compiler takes for another one: what is computed from it
// stays in the branch where it is needed.  (Comparisons of masks were done for
// every tile otherwise, a quarter of the instructions of an unmasked one.)
__device__ __forceinline__ int here(int v) {
    asm volatile("" : "+v"(v));
    return v;
}

__device__ __forceinline__ bool sees(int pos, int token, int window) {
    return (uint32_t)(pos - token) < (uint32_t)window;  // a token past pos: 2^31 or more; window 0: none
}

// The token that a lane's score n = 4 h + i belongs to, of its eight from
// `first` on: pairs of them begin at pair -turn, which is 0 for the split
// kernel and lane / 16 for the one of many rows (see Quarter).
__device__ __forceinline__ int place(int first, int n, int turn) { return first + ((n / 2 - turn) & 3) * 2 + n % 2; }

// Scores of a tile, s[r][h][i] of row tile r's row lane % 16 against token
// place(first, 4 h + i, turn), made ready for weights(): tokens that a row does not see are
// taken out, and its maximum moves if they outgrow it.  Of a row whose maximum is
// far the scores are made relative to the largest one here, in every tile (base
// is 0 then).  That adds nothing to other rows' tiles, and 4 us to the 455 of the
// chunked prompts: the scores may change where the maximum moves.
template <int D, int R>
__device__ __forceinline__ void settle(State<D, R> &st, f32x4 (&s)[R][2], int first, int turn, bool masked, int window, const AttnArgs &a) {
    if (masked) {
        const int token = here(first);
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
            for (int n = 0; n < 8; ++n)
                if (!sees(st.pos[r], place(token, n, turn), window)) s[r][n / 4][n % 4] = kNegInf;
    }
    float top[R];
    bool more = false;
#pragma unroll
    for (int r = 0; r < R; ++r) {
        top[r] = s[r][0][0];
#pragma unroll
        for (int n = 1; n < 8; ++n) top[r] = fmaxf(top[r], s[r][n / 4][n % 4]);
        more |= top[r] > st.row[r].limit;
    }
    if (__any(more)) {
#pragma unroll
        for (int r = 0; r < R; ++r) {
            RowTile<D> &o = st.row[r];
            float t = fmaxf(top[r], __shfl_xor(top[r], 16));
            t = fmaxf(t, __shfl_xor(t, 32));
            const bool was = o.far();
            if (was) t = fmaxf(t, o.m);
            const float before = was ? o.m * a.c : o.m, m = fmaxf(before, t * a.c);
            o.rescale(o.weight(before, m));
            const bool far = is_far(m);
            o.m = far ? t : m;
            o.base = far || m == kNegInf ? 0.0f : m;
            o.limit = far ? kNegInf : (m + kSlack) / a.c;
            if (far) {
#pragma unroll
                for (int n = 0; n < 8; ++n) s[r][n / 4][n % 4] -= t;
            }
        }
    }
}

// The weights of the lane's eight tokens, two in a word, as bf16.
template <int D, int R>
__device__ __forceinline__ void weights(State<D, R> &st, const f32x4 (&s)[R][2], bf16x8 (&p)[R], const AttnArgs &a) {
#pragma unroll
    for (int r = 0; r < R; ++r) {
        RowTile<D> &o = st.row[r];
        float w[8];
#pragma unroll
        for (int n = 0; n < 8; ++n) {
            w[n] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[r][n / 4][n % 4], a.c, -o.base));
            o.l += w[n];
        }
        asm volatile("" : "+v"(o.l));  // here, and not where the compiler would put it: after the products
        const uint32_t v[4] = {bf16_pair(w[0], w[1]), bf16_pair(w[2], w[3]), bf16_pair(w[4], w[5]), bf16_pair(w[6], w[7])};
        p[r] = as_bf16(v);
    }
}

// What else a tile adds to the running results.
template <int D, int R>
__device__ __forceinline__ void finish_step(State<D, R> &st, const bf16x8 (&p)[R], const uint32_t (&flag)[4], bool nan_values, int first, int turn, int window) {
    constexpr int W = Kv4<D>::W;
    // The output is divided by the sum of the rounded weights, so that a row
    // that few tokens dominate keeps no error of their rounding; the matrix
    // unit adds it up beside the output.  lse has the unrounded sum.
    const uint32_t ones[4] = {0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u};
#pragma unroll
    for (int r = 0; r < R; ++r)
        st.row[r].d = __builtin_amdgcn_mfma_f32_16x16x32_bf16(as_bf16(ones), p[r], st.row[r].d, 0, 0, 0);
    if (nan_values) {
#pragma unroll
        for (int r = 0; r < R; ++r) {
            uint32_t seen[4] = {0, 0, 0, 0};
            const int token = here(first);
#pragma unroll
            for (int n = 0; n < 8; ++n)
                if (sees(st.pos[r], place(token, n, turn), window)) seen[n / 2] |= 0x3F80u << (n % 2 * 16);
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

// One tile.  `masked` (the same in all lanes): some of its tokens are unseen by
// some rows.
template <int D, int R>
__device__ __forceinline__ void step(State<D, R> &st, Tile<D> &t, int index, bool masked, const AttnArgs &a, int lane) {
    constexpr int W = Kv4<D>::W;
    using T = Tile<D>;
    bool nan_values = false;
    uint32_t flag[4] = {0, 0, 0, 0};  // 1 for each token whose V scale is wild
    if (masked) {
        // a token that a row does not see adds nothing to it, whatever V holds:
        // what could be infinite or NaN (0 times it is NaN) is taken out here,
        // and the rows that see it get NaN
        nan_values = __any(any_wild_scale(t.vs[0]) || any_wild_scale(t.vs[1]));
        if (nan_values) {
#pragma unroll
            for (int n = 0; n < 8; ++n)
                if (((t.vs[n / 4] >> (n % 4 * 8)) & 255u) >= kWildScale) {
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
    const int first = index * kTile + lane / 16 * 8;  // this lane's first token
    settle<D, R>(st, s, first, 0, masked, a.window, a);
    bf16x8 p[R];
    weights<D, R>(st, s, p, a);
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
                st.row[r].acc[j + i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(as_bf16(v[i]), p[r], st.row[r].acc[j + i], 0, 0, 0);
    }
    finish_step<D, R>(st, p, flag, nan_values, first, 0, a.window);
}

// The rows of a block, where they lie, and the tiles that they see.
struct Block {
    int seq, head, first, rows;  // rows: of the sequence's key head, first: of this block
    int q0, n, len;              // first query token; cached tokens, the table's or more; queries
    int lo, hi;                  // tiles [lo, hi)
    int seen_lo, seen_hi;        // tokens that every row sees: [seen_lo, seen_hi)
};

__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }

__device__ __forceinline__ bool locate(Block &b, const AttnArgs &a, int seq, int head, int block, int size) {
    const int q0 = min(max(a.q_start[seq], 0), a.tokens), q1 = min(max(a.q_start[seq + 1], q0), a.tokens);
    b.seq = seq, b.head = head;
    b.q0 = q0, b.len = q1 - q0;
    b.n = max(a.kv_len[seq], 0);
    b.rows = min(b.len, a.max_q) * a.group;
    b.first = block * size;
    if (b.first >= b.rows) return false;
    const int lowest = b.n - b.len + b.first / a.group;
    const int highest = b.n - b.len + (min(b.rows, b.first + size) - 1) / a.group;
    const int from = (int)max((int64_t)0, (int64_t)lowest - a.window + 1);
    const int tiles = a.per_seq << a.shift;  // that the table has: 25 bits, checked on the host
    b.lo = min(from / kTile, tiles);
    b.hi = highest >= from ? min(highest / kTile + 1, tiles) : b.lo;
    b.seen_lo = (int)max((int64_t)0, (int64_t)highest - a.window + 1);
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
        st.pos[r] = max(b.n - b.len + i, -1);  // before all tokens
        st.row[r].clear();
    }
}

// The pages of up to 64 tiles of a sequence, t, t + by, ..., one in each lane.
struct Pages {
    int page;        // of this lane's tile; the first where it is lost
    uint64_t known;  // tiles whose page is one of the cache's
    int t, by, count;

    __device__ __forceinline__ Pages(const AttnArgs &a, const int32_t *row, int t_, int by_, int hi, int lane)
        : t(t_), by(by_), count(min(64, (hi - t_ + by_ - 1) / by_)) {
        page = row[(t + min(lane, count - 1) * by) >> a.shift];
        known = __ballot((uint32_t)page < (uint32_t)a.pages);
        if ((uint32_t)page >= (uint32_t)a.pages) page = 0;
    }
    // Tile i, or the last one past it.
    __device__ __forceinline__ bool has(int i) const { return known >> min(i, count - 1) & 1; }
    template <int D>
    __device__ __forceinline__ const uint8_t *tile(const AttnArgs &a, int head, int i) const {
        i = min(i, count - 1);
        const int64_t at = (((int64_t)__builtin_amdgcn_readlane(page, i) * a.kv_heads + head) << a.shift) + ((t + i * by) & ((1 << a.shift) - 1));
        return a.cache + at * Kv4<D>::kBytes;
    }
};

// Tiles lo, lo + by, ... below hi.  While a tile is worked on, the next N - 1
// are on their way; the pages of 64 tiles are looked up at once, one in each
// lane.
template <int D, int R, int N>
__device__ __forceinline__ void sweep(State<D, R> &st, const AttnArgs &a, const Block &b, int lo, int hi, int by, int lane) {
    const int32_t *row = a.table + (int64_t)b.seq * a.table_stride;
    const Places<D> places(lane);
    for (int t = lo; t < hi; t += 64 * by) {
        const Pages pages(a, row, t, by, hi, lane);
        Tile<D> ring[N];
#pragma unroll
        for (int k = 0; k < N - 1; ++k) load_tile(ring[k], pages.tile<D>(a, b.head, k), places);
        for (int i = 0; i < pages.count; i += N) {
#pragma unroll
            for (int k = 0; k < N; ++k) {
                if (i + k >= pages.count) break;
                load_tile(ring[(k + N - 1) % N], pages.tile<D>(a, b.head, i + k + N - 1), places);
                if (!pages.has(i + k)) continue;
                const int index = t + (i + k) * by;
                const bool masked = index * kTile < b.seen_lo || (index + 1) * kTile > b.seen_hi;
                step<D, R>(st, ring[k], index, masked, a, lane);
            }
        }
    }
#pragma unroll
    for (int r = 0; r < R; ++r) st.row[r].end(a.c);
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
    const float inv = o.d[0] == 0 ? 0.0f : 1.0f / o.d[0];
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

// Where a row's output goes: channels j and j + 1 of each of the lane's four
// runs of W, and the row's lse.
template <int D>
__device__ __forceinline__ void put_pair(const AttnArgs &a, const Block &b, int r, int j, const f32x4 (&sum)[2], float m, float l, float d, int lane) {
    constexpr int W = Kv4<D>::W;
    const int row = b.first + r * 16 + lane % 16;
    if (row >= b.rows) return;
    const int i = row / a.group, h = b.head * a.group + row % a.group;
    const float inv = d == 0 ? 0.0f : 1.0f / d;
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
    if (j == 0 && lane < 16) a.lse[(int64_t)(b.q0 + i) * a.heads + h] = log_sum(m, l);
}

// Results that the waves of a workgroup leave in LDS, and joins there: a wave
// takes pairs of channels of a row tile.
template <int D, int R, int NW>
struct Exchange {
    static constexpr int W = Kv4<D>::W;
    f32x4 acc[NW][R][W][64];
    float m[NW][R][16], l[NW][R][16], d[NW][R][16];

    __device__ __forceinline__ void leave(const RowTile<D> (&row)[R], int lane, int wave) {
#pragma unroll
        for (int r = 0; r < R; ++r) {
#pragma unroll
            for (int j = 0; j < W; ++j) acc[wave][r][j][lane] = row[r].acc[j];
            if (lane < 16) m[wave][r][lane] = row[r].m, l[wave][r][lane] = row[r].l, d[wave][r][lane] = row[r].d[0];
        }
        __syncthreads();
    }
    template <typename Put>
    __device__ __forceinline__ void join(int rows, int lane, int wave, Put put) const {
        for (int item = wave; item < R * W / 2; item += NW) {
            const int r = item / (W / 2), j = item % (W / 2) * 2, row = lane % 16;
            if (r * 16 + row >= rows) continue;
            float all = kNegInf, ls = 0, ds = 0;
#pragma unroll
            for (int s = 0; s < NW; ++s) all = fmaxf(all, m[s][r][row]);
            f32x4 sum[2] = {{0, 0, 0, 0}, {0, 0, 0, 0}};
#pragma unroll
            for (int s = 0; s < NW; ++s) {
                const float w = RowTile<D>::weight(m[s][r][row], all);
                ls += l[s][r][row] * w;
                ds += d[s][r][row] * w;
                sum[0] += acc[s][r][j][lane] * w;
                sum[1] += acc[s][r][j + 1][lane] * w;
            }
            put(r, j, sum, all, ls, ds);
        }
    }
};

// Many rows: the four waves of a workgroup have R row tiles each, and share
// the work of turning codes into bf16: each turns a quarter of a tile, two words
// of K and two of each lane's eight tokens of V at D = 128, and leaves it in LDS
// as the products take it.
//
// While a tile's scores become weights, the products of the next tile's scores
// run, and the next tiles are turned beside the products of the output: in one
// stream of instructions, because one wave alone issues to its vector unit only
// every eighth cycle, and two waves to a SIMD are what the registers allow.
template <int D>
struct SharedK {
    u32x4 k[2][D / 32][64];
};

template <int D>
struct SharedV {
    static constexpr int W = Kv4<D>::W;
    uint32_t v[W][64][4];
    uint32_t flag[64][4];  // of a masked tile: tokens whose V scale is wild
};

// A wave's quarter of a tile's keys, or values, as it lies in the cache.
//
// The lanes' pairs of tokens are turned by lane / 16 places in LDS, so that the
// sixty-four words that a wave writes of a pair fall on as many banks (they
// fell on sixteen, and conflicts were a third of LDS's time: the chunked prompts
// took 567 us traced, and 547 without them).  K's tokens are taken in that
// order, too, which leaves the weights in it.
template <int D>
struct Quarter {
    static constexpr int kWords = D / 64;
    uint32_t w[kWords];
    uint32_t scale;

    // The places of a lane's parts, as in Places.
    static __device__ __forceinline__ Places<D> places(int lane, int wave) {
        using L = Kv4<D>;
        const int r = lane % 16, q = lane / 16, h = wave % 2, part = wave / 2;
        Places<D> at(lane);
        const int token = place(r / 4 * 8, h * 4 + r % 4, r / 4);
        at.k = L::k_code(token, D == 64 ? q * 16 + part * 8 : D == 128 ? q * 32 + part * 16 : part * 128 + q * 32);
        at.ks = L::k_scale(token, D == 64 ? q / 2 : D == 128 ? q : part * 4 + q);
        at.v += wave * L::W;
        at.vs += wave * 2;
        return at;
    }
    __device__ __forceinline__ void load_k(const uint8_t *tile, const Places<D> &at) {
        const TileAddr p = tile_addr<D>(tile);
        load_words(w, p, at.k);
        scale = (uint8_t)__builtin_amdgcn_raw_buffer_load_b8(p, at.ks, 0, 0);
    }
    __device__ __forceinline__ void load_v(const uint8_t *tile, const Places<D> &at) {
        const TileAddr p = tile_addr<D>(tile);
        load_words(w, p, at.v);
        scale = (uint16_t)__builtin_amdgcn_raw_buffer_load_b16(p, at.vs, 0, 0);
    }
    __device__ __forceinline__ void turn_k(SharedK<D> &to, int lane, int wave) const {
        const float by = kv4_scale(scale);
#pragma unroll
        for (int n = 0; n < kWords; ++n) {
            u32x4 t;
#pragma unroll
            for (int e = 0; e < 4; ++e) t[e] = kv4_pair(w[n], by, e);
            to.k[wave % 2][wave / 2 * kWords + n][lane] = t;
        }
    }
    // Values that could be infinite or NaN are taken out of a masked tile, and
    // flagged.
    __device__ __forceinline__ void hide(SharedV<D> &to, int lane, int wave) {
        uint32_t f = 0;
        if ((scale & 255u) >= kWildScale) f |= 0x3F80u, scale &= 0xFF00u;
        if (scale >> 8 >= kWildScale) f |= 0x3F800000u, scale &= 0xFFu;
        to.flag[lane][(wave + lane / 16) % 4] = f;
    }
    __device__ __forceinline__ void turn_v(SharedV<D> &to, int lane, int wave) const {
        constexpr int W = Kv4<D>::W;
        const uint32_t one[1] = {scale};
        const float s0 = scale_at(one, 0), s1 = scale_at(one, 1);
#pragma unroll
        for (int j = 0; j < W; j += 2) {
            const int b0 = j / 2, b1 = b0 + W / 2;
            const uint32_t x = kv4_pair(w[b0 / 4], s0, b0 % 4), y = kv4_pair(w[b1 / 4], s1, b1 % 4);
            to.v[j][lane][(wave + lane / 16) % 4] = __builtin_amdgcn_perm(y, x, 0x05040100u);
            to.v[j + 1][lane][(wave + lane / 16) % 4] = __builtin_amdgcn_perm(y, x, 0x07060302u);
        }
    }
};

template <int D, int R>
__device__ __forceinline__ void scores(f32x4 (&s)[R][2], const State<D, R> &st, const bf16x8 (&k)[2][D / 32]) {
#pragma unroll
    for (int n = 0; n < D / 32; ++n) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
#pragma unroll
            for (int r = 0; r < R; ++r) {
                const f32x4 z = {0, 0, 0, 0};
                s[r][h] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(k[h][n], as_bf16(st.q[r][n]), n ? s[r][h] : z, 0, 0, 0);
            }
        }
    }
}

template <int D, int R>
__global__ __launch_bounds__(kThreads, 2) void k_kv4_attention_wide(AttnArgs a) {
    constexpr int W = Kv4<D>::W;
    __shared__ __attribute__((aligned(16))) SharedK<D> ks[2];
    __shared__ __attribute__((aligned(16))) SharedV<D> vs[2];
    const int lane = threadIdx.x % 64, wave = uniform(threadIdx.x / 64);
    // Each XCD takes a run of workgroups, so that the row blocks that read one
    // key head find it in one L2; later rows see more tokens and begin first.
    const int runs = gridDim.x / 8, id = blockIdx.x % 8 * runs + blockIdx.x / 8;
    const int unit = id / a.blocks, block = a.blocks - 1 - id % a.blocks;
    if (unit >= a.batch * a.kv_heads) return;
    Block b, w;  // of the workgroup, of this wave
    constexpr int kRows = 16 * R;
    if (!locate(b, a, unit % a.batch, unit / a.batch, block, kWaves * kRows)) return;
    // a wave past the last row repeats that one, and writes nothing
    const bool works = locate(w, a, b.seq, b.head, block * kWaves + wave, kRows);
    State<D, R> st;
    begin(st, a, w, lane);
    const Places<D> places = Quarter<D>::places(lane, wave);
    // A tile's page is looked up an iteration before its address is needed, by
    // a scalar load.  Tiles past the last are that one again, and not used.
    typedef const __attribute__((address_space(4))) int32_t *Table;
    const Table row = (Table)(uintptr_t)(a.table + (int64_t)b.seq * a.table_stride);
    const auto page = [&](int t) { return row[min(t, b.hi - 1) >> a.shift]; };
    const auto lost = [&](int pg) { return (uint32_t)pg >= (uint32_t)a.pages; };
    const auto tile = [&](int t, int pg) {
        const int64_t at = (((int64_t)(lost(pg) ? 0 : pg) * a.kv_heads + b.head) << a.shift) + (min(t, b.hi - 1) & ((1 << a.shift) - 1));
        return a.cache + at * Kv4<D>::kBytes;
    };
    // whether tile t, on that page, has tokens that a row does not see
    const auto masked = [&](int t, int pg) { return lost(pg) | (t * kTile < b.seen_lo) | ((t + 1) * kTile > b.seen_hi); };
    if (b.lo < b.hi) {
        int pg[5];  // of tiles t .. t + 4
#pragma unroll
        for (int i = 0; i < 5; ++i) pg[i] = page(b.lo + i);
        Quarter<D> k, v, ahead_k;
        f32x4 s[R][2];
        const uint8_t *next = tile(b.lo + 2, pg[2]);  // of the values that are loaded next
        k.load_k(tile(b.lo, pg[0]), places);
        v.load_v(tile(b.lo, pg[0]), places);
        ahead_k.load_k(tile(b.lo + 1, pg[1]), places);
        k.turn_k(ks[0], lane, wave);
        if (masked(b.lo, pg[0])) v.hide(vs[0], lane, wave);
        v.turn_v(vs[0], lane, wave);
        v.load_v(tile(b.lo + 1, pg[1]), places);
        k.load_k(next, places);
        ahead_k.turn_k(ks[1], lane, wave);
        __syncthreads();
        {
            bf16x8 kf[2][D / 32];
#pragma unroll
            for (int n = 0; n < D / 32; ++n)
#pragma unroll
                for (int h = 0; h < 2; ++h) kf[h][n] = __builtin_bit_cast(bf16x8, ks[0].k[h][n][lane]);
            scores<D, R>(s, st, kf);
        }
        __syncthreads();
        for (int t = b.lo, now = 0; t < b.hi; ++t, now ^= 1) {
            const bool hidden = masked(t, pg[0]);
            const int window = lost(pg[0]) ? 0 : a.window;
            const int first = t * kTile + lane / 16 * 8;
            if (masked(t + 1, pg[1])) v.hide(vs[1 - now], lane, wave);
            settle<D, R>(st, s, first, lane / 16, hidden, window, a);
            // weights beside the products of the next scores, whose operands
            // are on their way from LDS already
            bf16x8 p[R], kf[2][D / 32], vf[W];
            f32x4 ahead[R][2];
#pragma unroll
            for (int n = 0; n < D / 32; ++n)
#pragma unroll
                for (int h = 0; h < 2; ++h) kf[h][n] = __builtin_bit_cast(bf16x8, ks[1 - now].k[h][n][lane]);
            __builtin_amdgcn_sched_barrier(0);
            __builtin_amdgcn_s_setprio(1);  // before the wave that waits or looks pages up
            weights<D, R>(st, s, p, a);
            scores<D, R>(ahead, st, kf);
#pragma unroll
            for (int j = 0; j < W; ++j) vf[j] = __builtin_bit_cast(bf16x8, *reinterpret_cast<const u32x4 *>(vs[now].v[j][lane]));
            // the tiles after beside the output's products
            k.turn_k(ks[now], lane, wave);
            v.turn_v(vs[1 - now], lane, wave);
#pragma unroll
            for (int j = 0; j < W; ++j)
#pragma unroll
                for (int r = 0; r < R; ++r)
                    st.row[r].acc[j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(vf[j], p[r], st.row[r].acc[j], 0, 0, 0);
            __builtin_amdgcn_s_setprio(0);
            v.load_v(next, places);
            next = tile(t + 3, pg[3]);
            k.load_k(next, places);
#pragma unroll
            for (int i = 0; i < 4; ++i) pg[i] = pg[i + 1];
            pg[4] = page(t + 5);
            uint32_t flag[4] = {0, 0, 0, 0};
            bool nan_values = false;
            if (hidden) {
                const u32x4 f = *reinterpret_cast<const u32x4 *>(vs[now].flag[lane]);
#pragma unroll
                for (int n = 0; n < 4; ++n) flag[n] = f[n];
                nan_values = __any((f[0] | f[1] | f[2] | f[3]) != 0);
            }
            finish_step<D, R>(st, p, flag, nan_values, first, lane / 16, window);
#pragma unroll
            for (int r = 0; r < R; ++r) s[r][0] = ahead[r][0], s[r][1] = ahead[r][1];
            __syncthreads();
        }
    }
    if (!works) return;
#pragma unroll
    for (int r = 0; r < R; ++r) {
        st.row[r].end(again().c);
        finish(st.row[r], again(), w, r, lane);
    }
}

// How the tiles of a block are shared by workgroups: equal ranges, none shorter
// than a tile for each wave.  At most a.splits ranges, and at least one.
__device__ __forceinline__ int ranges(const AttnArgs &a, const Block &b, int waves, int &chunk) {
    const int tiles = b.hi - b.lo;
    chunk = max(max(waves, a.chunk), (tiles + a.splits - 1) / a.splits);
    return max(1, (tiles + chunk - 1) / chunk);
}

// A range's result in the workspace: R W vectors as the lanes hold them, then
// the statistics.
template <int D, int R>
struct Part {
    static constexpr int W = Kv4<D>::W, kStats = R * W * 256, kFloats = kStats + R * 48;
};

// Few rows: the NW waves of a workgroup share a row block, and several
// workgroups do.
template <int D, int R, int NW>
__global__ __launch_bounds__(64 * NW, 2) void k_kv4_attention(AttnArgs a) {
    using P = Part<D, R>;
    __shared__ Exchange<D, R, NW> ex;
    const int lane = threadIdx.x % 64, wave = uniform(threadIdx.x / 64);
    const int split = blockIdx.x % a.splits, unit = blockIdx.x / a.splits;
    const int pair = unit / a.blocks;
    Block b;
    if (!locate(b, a, pair / a.kv_heads, pair % a.kv_heads, unit % a.blocks, 16 * R)) return;
    int chunk;
    const int count = ranges(a, b, NW, chunk);
    if (split >= count) return;
    {
        State<D, R> st;
        begin(st, a, b, lane);
        const int lo = b.lo + split * chunk;
        sweep<D, R, kRing>(st, a, b, lo + wave, min(b.hi, lo + chunk), NW, lane);
        ex.leave(st.row, lane, wave);
    }
    const AttnArgs &z = again();
    const int rows = min(b.rows - b.first, 16 * R);
    if (count == 1) {
        ex.join(rows, lane, wave, [&](int r, int j, const f32x4(&sum)[2], float m, float l, float d) {
            put_pair<D>(z, b, r, j, sum, m, l, d, lane);
        });
        return;
    }
    float *to = z.part + ((int64_t)unit * z.splits + split) * P::kFloats;
    ex.join(rows, lane, wave, [&](int r, int j, const f32x4(&sum)[2], float m, float l, float d) {
        f32x4 *v = reinterpret_cast<f32x4 *>(to) + (r * P::W + j) * 64 + lane;
        v[0] = sum[0];
        v[64] = sum[1];
        float *p = to + P::kStats + r * 48 + lane;
        if (j == 0 && lane < 16) p[0] = m, p[16] = l, p[32] = d;
    });
}

// Joins the ranges of a row block: four channels of sixteen rows are an item of
// one wave, or of the four of a workgroup.  Each sixteen lanes take a range of
// their own, and a wave has 4 kBatch ranges in flight.  A launch of its own:
// with the last workgroup to arrive joining them, stores that have to reach the
// coherence point, an atomic and loads from there followed one another, twice
// for 256 ranges, and took 10 us where this takes 4.6.
template <int D, int R, int kBatch, int NW>
__global__ __launch_bounds__(256) void k_kv4_join(AttnArgs a) {
    using P = Part<D, R>;
    constexpr int kItems = R * P::W * 4;  // of a row block
    __shared__ f32x4 acc[NW][16];
    __shared__ float stats[NW][3][16];
    const int lane = threadIdx.x % 64, wave = NW > 1 ? uniform(threadIdx.x / 64) : 0, row = lane % 16;
    const int id = NW > 1 ? blockIdx.x : blockIdx.x * 4 + uniform(threadIdx.x / 64);
    const int item = id % kItems, unit = id / kItems;  // kItems is a multiple of 4
    const int pair = unit / a.blocks, block = unit % a.blocks, r = item / (P::W * 4), j = item / 4 % P::W, q = item % 4;
    const float *base = a.part + (int64_t)unit * a.splits * P::kFloats;
    const int s0 = wave * 4 + lane / 16;
    f32x4 v[kBatch];
    float m[kBatch], l[kBatch], d[kBatch];
    // on their way while the block is looked up; ranges past the last that
    // there may be repeat it, and rows that no sequence has are left out
    if ((block * R + r) * 16 + row < a.max_q * a.group) {
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
            const float *p = base + (int64_t)min(s0 + k * (NW * 4), a.splits - 1) * P::kFloats;
            v[k] = reinterpret_cast<const f32x4 *>(p)[(r * P::W + j) * 64 + q * 16 + row];
            const float *t = p + P::kStats + r * 48 + row;
            m[k] = t[0], l[k] = t[16], d[k] = t[32];
        }
    }
    Block b;
    if (!locate(b, a, pair / a.kv_heads, pair % a.kv_heads, block, 16 * R)) return;
    int chunk;
    const int count = ranges(a, b, a.waves, chunk);
    if (count == 1) return;
    const bool used = b.first + r * 16 + row < b.rows;
    float top = kNegInf, ls = 0, ds = 0;
    f32x4 sum = {0, 0, 0, 0};
    if (used) {
#pragma unroll
        for (int k = 0; k < kBatch; ++k)
            if (s0 + k * (NW * 4) < count) top = fmaxf(top, m[k]);
    }
    top = fmaxf(top, __shfl_xor(top, 16));
    top = fmaxf(top, __shfl_xor(top, 32));
    if (used) {
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
            if (s0 + k * (NW * 4) < count) {  // the rest is memory that nothing was written to
                const float w = RowTile<D>::weight(m[k], top);
                ls += l[k] * w;
                ds += d[k] * w;
                sum += v[k] * w;
            }
        }
    }
#pragma unroll
    for (int x = 16; x < 64; x *= 2) {
        ls += __shfl_xor(ls, x);
        ds += __shfl_xor(ds, x);
#pragma unroll
        for (int e = 0; e < 4; ++e) sum[e] += __shfl_xor(sum[e], x);
    }
    if (NW > 1) {
        if (lane < 16) acc[wave][row] = sum, stats[wave][0][row] = top, stats[wave][1][row] = ls, stats[wave][2][row] = ds;
        __syncthreads();
        top = kNegInf, ls = ds = 0;
        sum = f32x4{0, 0, 0, 0};
#pragma unroll
        for (int s = 0; s < NW; ++s) top = fmaxf(top, stats[s][0][row]);
#pragma unroll
        for (int s = 0; s < NW; ++s) {
            const float w = RowTile<D>::weight(stats[s][0][row], top);
            ls += stats[s][1][row] * w;
            ds += stats[s][2][row] * w;
            sum += acc[s][row] * w;
        }
    }
    if (wave > 0 || lane >= 16 || !used) return;
    const int at = b.first + r * 16 + row, i = at / a.group, h = b.head * a.group + at % a.group;
    const float inv = ds == 0 ? 0.0f : 1.0f / ds;
    uint16_t *o = const_cast<uint16_t *>(a.out.p) + (int64_t)(b.q0 + i) * a.out.ts + (int64_t)h * a.out.hs + q * (4 * P::W) + j;
#pragma unroll
    for (int e = 0; e < 4; ++e) o[e * P::W] = (uint16_t)bf16_rne(sum[e] * inv);
    if (j == 0 && q == 0) a.lse[(int64_t)(b.q0 + i) * a.heads + h] = log_sum(top, ls);
}

constexpr int kCus = 256;
constexpr int kLong = 8;
constexpr int kSplits = 256;  // workgroups that share a row block, at most
// How a call is laid out, by its sizes alone.
struct Plan {
    bool wide;
    int tiles;  // row tiles of a wave
    int waves;  // of a workgroup
    int blocks, splits, chunk;
    int64_t units;
};

constexpr int wide_tiles(int dim) { return dim == 64 ? 3 : dim == 128 ? 2 : 1; }

Plan plan(int batch, int max_q, int64_t max_kv, int64_t window, int group, int kv_heads, int dim) {
    Plan p = {};
    const int64_t rows = (int64_t)max_q * group, tiles = (rows + 15) / 16;
    const int most = wide_tiles(dim);  // the registers' limit in both kernels
    p.tiles = (int)(tiles < most ? tiles : most);
    p.splits = p.chunk = 1;
    p.waves = kWaves;
    // Rows enough for two workgroups on each compute unit.  Where there are
    // fewer, a wave of this kernel waits for each tile's conversion, and the
    // split kernel is faster: one sequence of 4096 tokens, 8 key heads of 128,
    // four queries to each: 1024 queries take 115 us here and 91 there, 2048
    // 130 and 152.
    const int wide = kWaves * wide_tiles(dim);
    p.blocks = (int)((tiles + wide - 1) / wide);
    p.units = (int64_t)batch * kv_heads * p.blocks;
    p.wide = tiles >= wide && p.units >= 2 * kCus;
    if (p.wide) return p;
    p.blocks = (int)((tiles + p.tiles - 1) / p.tiles);
    p.units = (int64_t)batch * kv_heads * p.blocks;
    // Row blocks enough that two of their workgroups are on each compute unit:
    // none is split, and a third fits beside them.  64 sequences of 4096 tokens,
    // 8 key heads of 128, take 46 us, and 64 as two ranges of eight waves.  The
    // batch that loses is one of a long sequence among short ones: 131072
    // tokens and 63 times 1024 take 561 us, 220 as two ranges (42 for their
    // bytes).
    if (p.units >= 2 * kCus) return p;
    p.waves = 2 * kWaves;
    if (window && max_kv > window + max_q) max_kv = window + max_q;
    const int64_t steps = (max_kv + kTile - 1) / kTile;
    // One round of workgroups while there is a tile for each wave, and up to
    // four, which even out ragged lengths, while each wave has kLong tiles and
    // a sequence's rows are one block (with more, its results outweigh that).
    // Fifteen sequences of up to 108125 tokens, four key heads of 64: 42 us in four
    // rounds, 77 in one; other ragged batches take 10% longer to 30% less.
    int64_t s = kCus / p.units;
    if (s > steps / p.waves) s = steps / p.waves;
    int64_t more = p.blocks > 1 ? 1 : (4 * kCus + p.units - 1) / p.units;
    if (more > steps / (p.waves * kLong)) more = steps / (p.waves * kLong);
    if (s < more) s = more;
    if (s > kSplits) s = kSplits;
    p.splits = s < 1 ? 1 : (int)s;
    p.chunk = (int)((steps + p.splits - 1) / p.splits);
    return p;
}

// Floats of the ranges' results, at most, of all calls whose batch, max_q and
// max_kv are these or smaller.  plan() itself takes fewer ranges where there are
// more row blocks, so the sizes of single calls rise and fall with the batch.
// By its rule, with u < 2 kCus units that are split: u kCus / u is at most kCus,
// u ceil(4 kCus / u) at most 4 kCus + u - 1, neither above u times the steps' limit
// or u kSplits, and one range leaves nothing.
int64_t most_floats(int64_t batch, int64_t max_q, int64_t max_kv, int group, int kv_heads, int dim) {
    const auto least = [](int64_t x, int64_t y) { return x < y ? x : y; };
    const int64_t steps = (max_kv + kTile - 1) / kTile, few = steps / (2 * kWaves), more = steps / (2 * kWaves * kLong);
    if (few < 2) return 0;
    const int64_t tiles = (max_q * group + 15) / 16, most = wide_tiles(dim);
    const int64_t pairs = least(batch * kv_heads, 2 * kCus - 1);
    const int64_t units = least(batch * kv_heads * ((tiles + most - 1) / most), 2 * kCus - 1);
    const int64_t one_round = least(kCus, units * few);
    const int64_t rounds = least(4 * kCus + pairs - 1, pairs * least(kSplits, more));
    return (one_round > rounds ? one_round : rounds) * least(tiles, most) * (dim / 16 * 256 + 48);
}

bool valid_sizes(int64_t batch, int64_t tokens, int64_t max_q, int64_t max_kv, int heads, int kv_heads, int dim) {
    return batch >= 0 && batch <= 1 << 20 && tokens >= 0 && tokens <= 1 << 28 && max_q >= 0 &&
           max_q <= 1 << 24 && max_kv >= 0 && max_kv <= 0x7FFFFFFF && kv_heads >= 1 &&
           kv_heads <= 1 << 12 && heads >= 1 && heads <= 1 << 14 && heads % kv_heads == 0 &&
           max_q * heads <= 1 << 30 &&
           (dim == 64 || dim == 128 || dim == 256);
}

// The kernel of a call, and the one that joins its ranges.
struct Kernels {
    const void *main, *join;
    int items;  // workgroups of the second for each row block
};

template <int D, int R>
Kernels pick_rows(const Plan &p) {
    const int items = p.splits <= 64 ? R * Kv4<D>::W : R * Kv4<D>::W * 4;
    const void *join = p.splits <= 4    ? reinterpret_cast<const void *>(&k_kv4_join<D, R, 1, 1>)
                       : p.splits <= 16 ? reinterpret_cast<const void *>(&k_kv4_join<D, R, 4, 1>)
                       : p.splits <= 64 ? reinterpret_cast<const void *>(&k_kv4_join<D, R, 16, 1>)
                                        : reinterpret_cast<const void *>(&k_kv4_join<D, R, 16, 4>);
    if (p.wide) return {reinterpret_cast<const void *>(&k_kv4_attention_wide<D, wide_tiles(D)>), join, items};
    if (p.waves == kWaves) return {reinterpret_cast<const void *>(&k_kv4_attention<D, R, kWaves>), join, items};
    return {reinterpret_cast<const void *>(&k_kv4_attention<D, R, 2 * kWaves>), join, items};
}

Kernels pick(const Plan &p, int dim) {
    switch (dim * 4 + p.tiles) {
        case 64 * 4 + 1: return pick_rows<64, 1>(p);
        case 64 * 4 + 2: return pick_rows<64, 2>(p);
        case 64 * 4 + 3: return pick_rows<64, 3>(p);
        case 128 * 4 + 1: return pick_rows<128, 1>(p);
        case 128 * 4 + 2: return pick_rows<128, 2>(p);
        default: return pick_rows<256, 1>(p);
    }
}

}  // namespace
}  // namespace ar

using namespace ar;

extern "C" {

int64_t ar_kv4_attention_workspace(int64_t batch, int64_t tokens, int64_t max_q, int64_t max_kv,
                                   int heads, int kv_heads, int dim) {
    if (!valid_sizes(batch, tokens, max_q, max_kv, heads, kv_heads, dim)) return AR_EINVAL;
    const int64_t floats = most_floats(batch, max_q, max_kv, heads / kv_heads, kv_heads, dim);
    return floats > 4 ? 4 * floats : 16;
}

int ar_kv4_attention(ar_rows q, const void *cache, const void *page_table, int64_t table_stride,
                     const void *q_start, const void *kv_len, ar_rows out, void *lse, void *workspace,
                     int64_t tokens, int64_t batch, int heads, int kv_heads, int dim, int64_t pages,
                     int page_size, int64_t pages_per_seq, int64_t max_q, int64_t max_kv, int64_t window,
                     float scale, void *stream) {
    int shift = 0;
    if (!valid_sizes(batch, tokens, max_q, max_kv, heads, kv_heads, dim) ||
        !kv4_shape(kv_heads, dim, pages, page_size, &shift) || pages_per_seq < 0 ||
        pages_per_seq > 0x3FFFFFFF / page_size || table_stride < 0 || window < 0 ||
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
    const Plan p = plan((int)batch, (int)max_q, max_kv, window, heads / kv_heads, kv_heads, dim);
    AttnArgs a = {};
    a.q = rows(rq), a.out = rows(ro);
    a.cache = static_cast<const uint8_t *>(cache);
    a.table = static_cast<const int32_t *>(page_table);
    a.q_start = static_cast<const int32_t *>(q_start), a.kv_len = static_cast<const int32_t *>(kv_len);
    a.lse = static_cast<float *>(lse);
    a.part = static_cast<float *>(workspace);
    a.table_stride = table_stride;
    a.tokens = (int)tokens, a.batch = (int)batch, a.heads = heads, a.kv_heads = kv_heads, a.group = heads / kv_heads;
    a.pages = (int)pages, a.per_seq = pages ? (int)pages_per_seq : 0, a.shift = shift - 5;
    a.window = window ? (int)window : 0x7FFFFFFF, a.max_q = (int)max_q;
    a.blocks = p.blocks, a.splits = p.splits, a.chunk = p.chunk, a.waves = p.waves;
    a.vec = rq.vec() && ro.vec();
    a.c = scale * kLog2e;
    const int64_t pairs = batch * kv_heads;
    const int64_t grid = p.wide ? (pairs * p.blocks + 7) / 8 * 8 : pairs * p.blocks * p.splits;
    if (grid > 0x7FFFFFFF / (64 * p.waves)) return AR_EINVAL;
    const Kernels k = pick(p, dim);
    const int rc = launch(k.main, (unsigned)grid, 64 * p.waves, a, stream);
    if (rc != AR_OK || p.splits == 1) return rc;
    return launch(k.join, (unsigned)(p.units * k.items), 256, a, stream);
}

}  // extern "C"
