// kv4_attn.hip -- attention over the paged 4-bit cache (gfx950).
//
// Per query row and head: s_t = sm_scale * q.k_t over the tokens t that the row
// sees, o = sum_t exp(s_t - m) v_t / sum_t exp(s_t - m) with m the running
// maximum; k and v are level * scale.
#include "kv4.h"

namespace rad {
namespace {

constexpr float kLog2e = 1.44269504088896340736f;

// Tokens [lo, hi) that a row at position pos of a sequence of len tokens sees.
struct TokenRange {
    int lo, hi;
};
__device__ __forceinline__ TokenRange seen(int pos, int len, int causal, int window) {
    TokenRange r{window > 0 ? max(0, pos - window + 1) : 0, causal ? min(pos + 1, len) : len};
    if (pos < 0) r.hi = 0;
    return r;
}

// The (row, head) pairs of a sequence that share a KV head are the columns of transposed
// matrix products, 16 a product, NT of them a wave, so that nothing crosses lanes between
// the two products of a step of 32 tokens:
//
//   S^T [32 tokens][16 cols] = K Q^T    two 16x16x32 tiles; A: a lane holds D/4 dims of
//                                       one token, one dword (8 dims) per product
//   O^T [D][16 cols]        += V^T P^T  D/16 tiles; A: a lane holds one dim of eight
//                                       tokens, one dword
//
// Row r of score tile u is token 8 (r / 4) + 4 u + r % 4 of the step, so lane (g, c)
// (g = lane / 16, c = lane % 16) comes out of S^T with the scores of tokens 8 g ..
// 8 g + 7 of column c: the B operand that O^T needs against the value octets.
// Codes go from memory to registers to the products; a workgroup's four waves take
// WC groups of columns and 4 / WC groups of steps (joined through LDS at the end).
//
// e2m1 levels are exact in f16; the f16 scales meet the scores (keys) and the
// probabilities (values) in f32.  A query row is taken times a power of two that puts
// its largest value in [2^9, 2^10), where f16 holds bf16 and f16 queries exactly (what
// lies 2^-24 below the largest aside).  f32 queries and their weights are split in two
// f16 parts, 22 bits: with at most 8 columns the low parts ride in columns 8 .. 15 of
// the same products (HL 1), otherwise in products of their own (HL 2).  For bf16 and f16
// queries a weight is one f16 (HL 0).
//
// The reference exponent m of a column keeps its weights p * scale, p = 2^(score - m),
// inside f16: it is set so that the largest weight met comes to 2^kRoom, and raised only
// when one passes 2^kMost (one vote a step); then scores and scale exponents are looked at
// one by one.  A weight is thus held to 2^-24 of a scale on which the column's largest is at
// least 2^(kRoom - 1).
typedef unsigned int u4 __attribute__((ext_vector_type(4)));
typedef unsigned int u2 __attribute__((ext_vector_type(2)));
typedef float f4 __attribute__((ext_vector_type(4)));
typedef _Float16 h8 __attribute__((ext_vector_type(8)));

constexpr float kRoom = 4.0f;                       // log2
constexpr float kMost = 0x1p14f;                    // twice this is below 65504
constexpr float kMostP = 0x1p60f;                   // values of scale 0 weigh nothing, but count
constexpr float kLowest = -3.4028234663852886e38f;

// Eight e2m1 codes -> eight f16 levels.
__device__ __forceinline__ u4 levels8(uint32_t w) {
    return u4{__builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.0f, 0)),
              __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.0f, 1)),
              __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.0f, 2)),
              __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.0f, 3))};
}
__device__ __forceinline__ f4 mma16(u4 a, u4 b, f4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(h8, a), __builtin_bit_cast(h8, b), c, 0, 0, 0);
}

typedef _Float16 h2 __attribute__((ext_vector_type(2)));
// two values to f16: to the nearest, and cut (the rest a - cut is exact in f32)
__device__ __forceinline__ uint32_t f16_pack2(float a, float b) {
    return __builtin_bit_cast(uint32_t, h2{static_cast<_Float16>(a), static_cast<_Float16>(b)});
}
__device__ __forceinline__ uint32_t f16_cut2(float a, float b) {
    return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_pkrtz(a, b));
}
__device__ __forceinline__ u4 f16_pack8(const float (&w)[8]) {
    return u4{f16_pack2(w[0], w[1]), f16_pack2(w[2], w[3]), f16_pack2(w[4], w[5]), f16_pack2(w[6], w[7])};
}
// high and low f16 parts of eight values
__device__ __forceinline__ void f16_split8(const float (&w)[8], u4 &hi, u4 &low) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t cut = f16_cut2(w[2 * i], w[2 * i + 1]);
        const h2 h = __builtin_bit_cast(h2, cut);
        hi[i] = cut;
        low[i] = f16_pack2(fmaf(static_cast<float>(h[0]), -1.0f, w[2 * i]), fmaf(static_cast<float>(h[1]), -1.0f, w[2 * i + 1]));
    }
}

__device__ __forceinline__ float max8(const float (&s)[8]) {
    return fmaxf(fmaxf(fmaxf(s[0], s[1]), fmaxf(s[2], s[3])), fmaxf(fmaxf(s[4], s[5]), fmaxf(s[6], s[7])));
}
// Maximum (sum) over the four lanes that hold one column.
__device__ __forceinline__ float col_max(float v) {
    v = fmaxf(v, __shfl_xor(v, 16));
    return fmaxf(v, __shfl_xor(v, 32));
}
__device__ __forceinline__ float col_sum(float v) {
    v += __shfl_xor(v, 16);
    return v + __shfl_xor(v, 32);
}

// ---- how a call's work is shared out --------------------------------------
//
// A sequence's (row, head of the group) pairs of one KV head form tiles of TM; a tile's
// context, in steps of 32 tokens, is cut into equal parts, one workgroup each.  Lengths
// are known on the device alone, so every workgroup works out the same cut: `chunk`
// steps a part such that about `target` workgroups result over all sequences and KV
// heads (as many as the chip holds at once), the same number of parts for each tile of
// a sequence.  With the sum over sequences of tiles * steps at most target / heads *
// chunk, there are at most target / heads + tiles pieces a head, and at most target /
// heads tiles in several parts, of 2 * target / heads parts together.  Each lane looks
// at one sequence, 64 at a time; beyond kMostScanned sequences nothing is split.
constexpr int kMostScanned = 512;
struct Plan {
    int tm, target, min_chunk, split;     // rows a tile; workgroups wanted; least steps a part; 0: one part a tile
    int pieces, items, slots;             // bounds a KV head: workgroups, tiles in several parts, parts of those
};
struct Piece {
    int seq, tile, part, parts, slot;     // parts 0: none.  slot: place among the parts kept apart
};

// Rows of a sequence that a call handles, and what they see together.
struct SeqWork {
    RowRange rr;
    int n, len, pos0, lo, hi;             // rows handled, tokens, first row's position, tokens [lo, hi)
};
__device__ __forceinline__ SeqWork seq_work(const KvBatch &b, const Kv4Attn &a, int seq) {
    SeqWork s;
    s.rr = kv_rows(b, seq);
    s.n = min(s.rr.n, b.max_q);
    s.len = kv_len(b, seq);
    s.pos0 = s.len - s.rr.n;
    s.lo = seen(max(s.pos0, 0), s.len, a.causal, a.window).lo;
    s.hi = a.causal ? s.pos0 + s.n : (s.pos0 + s.n > 0 ? s.len : 0);
    if (s.hi < s.lo) s.hi = s.lo;
    return s;
}
__device__ __forceinline__ int steps_of(int lo, int hi) { return hi > lo ? ((hi + 31) >> 5) - (lo >> 5) : 0; }

// Inclusive sum over the lanes of a wave: inside rows of 16, then row 0 into 1 and 2 into
// 3, then rows 0 .. 1 into 2 .. 3.
__device__ __forceinline__ int wave_scan(int v) {
    v += __builtin_amdgcn_update_dpp(0, v, 0x111, 0xF, 0xF, true);     // row_shr 1, 2, 4, 8
    v += __builtin_amdgcn_update_dpp(0, v, 0x112, 0xF, 0xF, true);
    v += __builtin_amdgcn_update_dpp(0, v, 0x114, 0xF, 0xF, true);
    v += __builtin_amdgcn_update_dpp(0, v, 0x118, 0xF, 0xF, true);
    v += __builtin_amdgcn_update_dpp(0, v, 0x142, 0xA, 0xF, false);    // row_bcast 15
    v += __builtin_amdgcn_update_dpp(0, v, 0x143, 0xC, 0xF, false);    // row_bcast 31
    return v;
}

// Steps a part: about `target` parts over all sequences and KV heads, rounded up.
__device__ __forceinline__ int chunk_of(uint64_t total, const Plan &pl, int heads) {
    const uint64_t all = total * static_cast<uint32_t>(heads) + static_cast<uint32_t>(pl.target - 1);
    const int even = all >> 32 ? static_cast<int>(all / static_cast<uint32_t>(pl.target))
                               : static_cast<int>(static_cast<uint32_t>(all) / static_cast<uint32_t>(pl.target));
    return max(even, pl.min_chunk);
}

// The x-th piece of a KV head (ITEMS false), or the x-th tile in several parts (true).
// Every lane of the wave calls it and gets the same answer.
template <bool ITEMS>
__device__ __forceinline__ Piece find_piece(const KvBatch &b, const Kv4Attn &a, const Plan &pl, int heads, int G, int x) {
    const int lane = threadIdx.x & 63;
    if (b.B == 1 && !ITEMS) {
        const SeqWork s = seq_work(b, a, 0);
        const int tiles = (s.n * G + pl.tm - 1) / pl.tm, steps = steps_of(s.lo, s.hi);
        const int chunk = chunk_of(static_cast<uint64_t>(tiles) * static_cast<uint32_t>(steps), pl, heads);
        const int parts = pl.split ? max(1, (steps + chunk - 1) / chunk) : 1;
        const int tile = x / parts;
        if (tile >= tiles || (parts > 1 && x >= pl.slots)) return Piece{0, 0, 0, 0, 0};
        return Piece{0, tiles - 1 - tile, x % parts, parts, x};
    }
    uint64_t total = 0;
    if (pl.split) {
        for (int b0 = 0; b0 < b.B; b0 += 64) {
            uint64_t t = 0;
            if (b0 + lane < b.B) {
                const SeqWork s = seq_work(b, a, b0 + lane);
                t = static_cast<uint64_t>((s.n * G + pl.tm - 1) / pl.tm) * static_cast<uint32_t>(steps_of(s.lo, s.hi));
            }
            // in two parts, so that 64 of each fit 32 bits
            const int low = wave_scan(static_cast<int>(t & 0xFFFFFFu)), high = wave_scan(static_cast<int>(t >> 24));
            total += static_cast<uint32_t>(__builtin_amdgcn_readlane(low, 63)) +
                     (static_cast<uint64_t>(static_cast<uint32_t>(__builtin_amdgcn_readlane(high, 63))) << 24);
        }
    }
    const int chunk = chunk_of(total, pl, heads);
    int before = 0, kept = 0;
    for (int b0 = 0; b0 < b.B; b0 += 64) {
        int tiles = 0, parts = 0;
        if (b0 + lane < b.B) {
            const SeqWork s = seq_work(b, a, b0 + lane);
            tiles = (s.n * G + pl.tm - 1) / pl.tm;
            parts = pl.split ? max(1, (steps_of(s.lo, s.hi) + chunk - 1) / chunk) : 1;
        }
        const int many = parts > 1 ? tiles : 0, mine = ITEMS ? many : tiles * parts, keep = many * parts;
        const int sum = wave_scan(mine), sum_keep = wave_scan(keep);
        const uint64_t hit = __ballot(mine > 0 && x >= before + sum - mine && x < before + sum);
        if (hit) {
            const int src = __builtin_ctzll(hit);
            Piece p;
            p.seq = b0 + src;
            p.parts = __builtin_amdgcn_readlane(parts, src);
            const int local = x - (before + __builtin_amdgcn_readlane(sum - mine, src));
            const int slot0 = kept + __builtin_amdgcn_readlane(sum_keep - keep, src);
            const int tile = ITEMS ? local : local / p.parts;
            p.part = ITEMS ? 0 : local % p.parts;
            p.slot = slot0 + tile * p.parts + p.part;
            // holds for every ascending q_start; another must not leave the workspace
            if (p.parts > 1 && (p.slot < 0 || p.slot + (ITEMS ? p.parts : 1) > pl.slots)) break;
            // the last rows of a causal prompt see most: they go first
            p.tile = __builtin_amdgcn_readlane(tiles, src) - 1 - tile;
            return p;
        }
        before += __builtin_amdgcn_readlane(sum, 63);
        kept += __builtin_amdgcn_readlane(sum_keep, 63);
    }
    return Piece{0, 0, 0, 0, 0};
}

// A step's codes and scales, one lane's share.
template <int D>
struct Step {
    uint32_t k[2][D / 32];      // D / 4 dims of a token of each tile
    u4 v[D / 64];               // one octet of tokens, dims 64 j + 4 r ..
    u4 ks, vs;                  // f16 scales of the octet
};

// NT: nontemporal, for codes that only one workgroup reads
template <bool NT>
__device__ __forceinline__ u4 load16(const u4 *p) {
    if constexpr (NT) return __builtin_nontemporal_load(p);
    else return *p;
}
template <int D, bool NT>
__device__ __forceinline__ void load_step(Step<D> &s, const Kv4Cache &c, int64_t tok, int g, int r) {
    // tok: index of the step's first token in the cache's [pages][heads][page] order
#pragma unroll
    for (int u = 0; u < 2; ++u) {
        const uint8_t *p = c.k_codes + (tok + 8 * (r >> 2) + 4 * u + (r & 3)) * (D / 2) + g * (D / 8);
        if constexpr (D == 64) {
            const u2 x = *reinterpret_cast<const u2 *>(p);
            s.k[u][0] = x.x;
            s.k[u][1] = x.y;
        } else {
#pragma unroll
            for (int j = 0; j < D / 128; ++j) {
                const u4 x = load16<NT>(reinterpret_cast<const u4 *>(p) + j);
                s.k[u][4 * j] = x.x;
                s.k[u][4 * j + 1] = x.y;
                s.k[u][4 * j + 2] = x.z;
                s.k[u][4 * j + 3] = x.w;
            }
        }
    }
    const u4 *vp = reinterpret_cast<const u4 *>(c.v_codes) + (((tok >> 3) + g) * D + 4 * r) / 4;
#pragma unroll
    for (int j = 0; j < D / 64; ++j) s.v[j] = load16<NT>(vp + 16 * j);
    s.ks = *reinterpret_cast<const u4 *>(c.k_scale + tok + 8 * g);
    s.vs = *reinterpret_cast<const u4 *>(c.v_scale + tok + 8 * g);
}

// f times the i-th of eight f16 values, as one mixed-precision multiply-add
__device__ __forceinline__ float times_half(float f, const u4 &x, int i) {
    const h2 h = __builtin_bit_cast(h2, static_cast<uint32_t>(x[i >> 1]));
    return fmaf(f, static_cast<float>(h[i & 1]), 0.0f);
}

// blockIdx: x piece, y KV head.  A tile has TM = 16 * NT * WC columns, `cols` of them in
// use at most.  Parts of a tile in several leave their sums in part_o [heads][slots][cols][D]
// and part_ml [..][cols][2]; the others write the outputs.
template <int DT, int D, int HL, int NT, int WC>
__global__ __launch_bounds__(256, 2) void attn_kernel(Kv4Cache c, KvBatch b, Kv4Attn a, Plan pl, int cols,
                                                      float *part_o, float *part_ml) {
    constexpr int TG = 4 / WC, TC = 16 * NT, TM = TC * WC;
    static_assert(HL != 1 || (NT == 1 && WC == 1), "low parts ride along in one product of columns");
    __shared__ float lds_o[TG > 1 ? TG : 1][TG > 1 ? TM : 1][D + 4], lds_ml[TG > 1 ? TG : 1][TM][2];
    const int lane = threadIdx.x & 63, wid = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int g = lane >> 4, col = lane & 15, tg = wid / WC, wc = wid % WC;
    const int h = blockIdx.y, G = a.q_heads / c.heads;
    const Piece pc = find_piece<false>(b, a, pl, c.heads, G, blockIdx.x);
    if (pc.parts == 0) return;
    const int seq = __builtin_amdgcn_readfirstlane(pc.seq);
    const SeqWork sw = seq_work(b, a, seq);
    const RowRange rr = sw.rr;
    const int len = sw.len, pos0 = sw.pos0, pairs = sw.n * G, tile0 = pc.tile * TM;   // first pair of the tile

    // the tile's and this wave's share of the context
    const int tile_last = min(tile0 + TM, pairs) - 1, wave0 = tile0 + wc * TC, wave_last = min(wave0 + TC, pairs) - 1;
    const bool idle = wave0 >= pairs;
    auto range = [&](int first, int last) {
        const int p0 = pos0 + first / G, p1 = pos0 + last / G;
        TokenRange r{seen(max(p0, 0), len, a.causal, a.window).lo, seen(p1, len, a.causal, a.window).hi};
        if (r.hi < r.lo) r.hi = r.lo;
        return r;
    };
    const TokenRange tile_r = range(tile0, tile_last), wave_r = range(idle ? tile0 : wave0, idle ? tile_last : wave_last);
    const int steps = steps_of(tile_r.lo, tile_r.hi), share = (steps + pc.parts - 1) / pc.parts;
    const int from = (tile_r.lo >> 5) + pc.part * share, to = (tile_r.lo >> 5) + min((pc.part + 1) * share, steps);
    const int begin = __builtin_amdgcn_readfirstlane(max(from, wave_r.lo >> 5) + tg);
    const int end = __builtin_amdgcn_readfirstlane(idle ? 0 : min(to, (wave_r.hi + 31) >> 5));

    // steps [open_lo, open_hi) that all of the wave's rows see whole: rows see ever later tokens
    const TokenRange first_r = range(idle ? tile0 : wave0, idle ? tile0 : wave0);
    const int open_lo = __builtin_amdgcn_readfirstlane((seen(max(pos0 + (idle ? tile_last : wave_last) / G, 0), len, a.causal, a.window).lo + 31) >> 5);
    const int open_hi = __builtin_amdgcn_readfirstlane(first_r.hi >> 5);

    // this lane's columns: pair cp is row cp / G of the sequence, head h * G + cp % G
    bool used[NT];
    TokenRange tr[NT];
    int64_t qrow[NT];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
        const int cp = wave0 + 16 * t + (HL == 1 ? col & 7 : col);
        used[t] = cp < pairs;
        const int ci = used[t] ? cp / G : 0, cg = used[t] ? cp % G : 0;
        tr[t] = used[t] ? seen(pos0 + ci, len, a.causal, a.window) : wave_r;
        qrow[t] = (static_cast<int64_t>(rr.first + ci) * a.q_heads + h * G + cg) * D;
    }
    // the queries' values are asked for first, then the first steps
    constexpr int NK = D / 32;
    float qv[NT][NK][8];
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int j = 0; j < NK; ++j) {
            const int64_t at = qrow[t] + g * (D / 4) + 8 * j;
            const float4 x = load4<DT>(a.q, at), y = load4<DT>(a.q, at + 4);
            qv[t][j][0] = x.x; qv[t][j][1] = x.y; qv[t][j][2] = x.z; qv[t][j][3] = x.w;
            qv[t][j][4] = y.x; qv[t][j][5] = y.y; qv[t][j][6] = y.z; qv[t][j][7] = y.w;
        }

    const int per_page = b.page_shift - 5;                    // log2 of steps a page
    // Page ids come through the scalar cache (no kernel writes them while this one runs): a
    // vector load here would wait for every code on its way.
    typedef const __attribute__((address_space(4))) int32_t *scalar_ids;
    const scalar_ids table = (scalar_ids)(b.block_table + static_cast<int64_t>(seq) * b.max_pages);
    auto page_of = [&](int step) { return step < end ? table[step >> per_page] : -1; };
    auto token_of = [&](int page, int step) {
        const int64_t p = page >= 0 && page < c.pages ? page : 0;
        return ((p * c.heads + h) << c.page_shift) + (step < end ? (step << 5) & ((1 << c.page_shift) - 1) : 0);
    };

    // A wave's steps go through a ring: two (one, where the columns' sums fill the
    // registers) on their way while one is worked on.  Past the end the loads go on, to the
    // start of page 0 (cached, unused): were they conditional, the wait for a step's codes
    // would have to be a wait for the later ones too.
    constexpr int NB = D == 256 || NT > 1 ? 2 : 3;
    constexpr bool ONCE = WC == 1;                            // no other wave reads these codes
    Step<D> ring[NB];
    int page[NB];
#pragma unroll
    for (int k = 0; k < NB; ++k) page[k] = page_of(begin + k * TG);
#pragma unroll
    for (int k = 0; k < NB - 1; ++k) load_step<D, ONCE>(ring[k], c, token_of(page[k], begin + k * TG), g, col);

    u4 qf[NT][NK], ql[HL == 2 ? NT : 1][HL == 2 ? NK : 1];
    float scale[NT];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
        float big = 0.0f;
#pragma unroll
        for (int j = 0; j < NK; ++j)
#pragma unroll
            for (int i = 0; i < 8; ++i) big = fmaxf(big, fabsf(qv[t][j][i]));
        big = col_max(big);
        // largest value to [2^9, 2^10), undone in the scores' factor (both exact)
        const int e = big > 0.0f ? 10 - __builtin_amdgcn_frexp_expf(big) : 0;
#pragma unroll
        for (int j = 0; j < NK; ++j) {
#pragma unroll
            for (int i = 0; i < 8; ++i) qv[t][j][i] = used[t] ? __builtin_amdgcn_ldexpf(qv[t][j][i], e) : 0.0f;
            if constexpr (HL == 0) {
                qf[t][j] = f16_pack8(qv[t][j]);
            } else {
                u4 hi, low;
                f16_split8(qv[t][j], hi, low);
                if constexpr (HL == 2) ql[t][j] = low;
                qf[t][j] = HL == 1 && col >= 8 ? low : hi;
            }
        }
        scale[t] = fmaxf(__builtin_amdgcn_ldexpf(a.sm_scale * kLog2e, -e), 1e-30f);   // never 0: a masked score is -inf
    }

    float m[NT], l[NT];
    f4 acc[NT][D / 16];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
        m[t] = kLowest;
        l[t] = 0.0f;
#pragma unroll
        for (int j = 0; j < D / 16; ++j) acc[t][j] = f4{0.f, 0.f, 0.f, 0.f};
    }

    auto work = [&](Step<D> &cur, int step) {
        float s[NT][8];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            f4 x[NT];
#pragma unroll
            for (int t = 0; t < NT; ++t) x[t] = f4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int j = 0; j < NK; ++j) {
                const u4 kf = levels8(cur.k[u][j]);
#pragma unroll
                for (int t = 0; t < NT; ++t) {
                    if constexpr (HL == 2) x[t] = mma16(kf, ql[t][j], x[t]);
                    x[t] = mma16(kf, qf[t][j], x[t]);
                }
            }
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    float y = x[t][i];
                    if constexpr (HL == 1) y += lane_xor<8>(y);          // high and low part of the query
                    s[t][4 * u + i] = times_half(y, cur.ks, 4 * u + i);
                }
        }
        if (step < open_lo || step >= open_hi) {
            const int t0 = (step << 5) + 8 * g;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                bool any = false;
#pragma unroll
                for (int t = 0; t < NT; ++t) {
                    const bool on = t0 + i >= tr[t].lo && t0 + i < tr[t].hi;
                    s[t][i] = on ? s[t][i] : -INFINITY;
                    any = any || on;
                }
                // a scale past the sequence's end may be anything
                cur.vs[i >> 1] &= any ? 0xFFFFFFFFu : (i & 1 ? 0x0000FFFFu : 0xFFFF0000u);
            }
        }
        float w[NT][8], sum[NT];
        bool pass = false;
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            sum[t] = 0.0f;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float p = __builtin_amdgcn_exp2f(fmaf(s[t][i], scale[t], -m[t]));
                sum[t] += p;
                w[t][i] = times_half(p, cur.vs, i);
            }
            pass = pass || !(max8(w[t]) <= kMost && sum[t] <= kMostP);
        }
        if (__any(pass)) {                                 // also the first step: m is the lowest
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                float most = -INFINITY;
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float vs = times_half(1.0f, cur.vs, i);
                    most = fmaxf(most, fmaf(s[t][i], scale[t], vs > 0.0f ? static_cast<float>(__builtin_amdgcn_frexp_expf(vs)) : -24.0f));
                }
                const float mn = fmaxf(m[t], col_max(most) - kRoom), shrink = __builtin_amdgcn_exp2f(m[t] - mn);
                m[t] = mn;
                l[t] *= shrink;
#pragma unroll
                for (int j = 0; j < D / 16; ++j) acc[t][j] *= shrink;
                sum[t] = 0.0f;
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float p = __builtin_amdgcn_exp2f(fmaf(s[t][i], scale[t], -m[t]));
                    sum[t] += p;
                    w[t][i] = times_half(p, cur.vs, i);
                }
            }
        }
        u4 wf[NT], wl[NT];
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            l[t] += sum[t];
            if constexpr (HL == 0) {
                wf[t] = f16_pack8(w[t]);
            } else {
                u4 hi;
                f16_split8(w[t], hi, wl[t]);
                wf[t] = HL == 1 && col >= 8 ? wl[t] : hi;
            }
        }
#pragma unroll
        for (int j = 0; j < D / 64; ++j) {
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                const u4 vf = levels8(cur.v[j][x]);
#pragma unroll
                for (int t = 0; t < NT; ++t) {
                    if constexpr (HL == 2) acc[t][4 * j + x] = mma16(vf, wl[t], acc[t][4 * j + x]);
                    acc[t][4 * j + x] = mma16(vf, wf[t], acc[t][4 * j + x]);
                }
            }
        }
    };
    for (int step = begin; step < end;) {
#pragma unroll
        for (int k = 0; k < NB; ++k) {
            constexpr int ahead = NB - 1;
            const int in = (k + ahead) % NB;
            load_step<D, ONCE>(ring[in], c, token_of(page[in], step + ahead * TG), g, col);
            const int now = page[k];
            page[k] = page_of(step + NB * TG);
            if (now >= 0 && now < c.pages) work(ring[k], step);
            step += TG;
            if (step >= end) break;
        }
    }

    // lane (g, c) holds dims 64 j + 16 g .. + 15 of column c: acc[4 j + x][i] is 4 i + x of them
    auto dims4 = [&](int t, int j, int i) { return f4{acc[t][4 * j][i], acc[t][4 * j + 1][i], acc[t][4 * j + 2][i], acc[t][4 * j + 3][i]}; };
    auto put = [&](int cc, int d, f4 o, float mt, float lt) {
        // sums of the tile's column cc
        if (pc.parts == 1) {
            const float inv = lt > 0.0f ? 1.0f / lt : 0.0f;
            const int cp = tile0 + cc;
            const int64_t at = (static_cast<int64_t>(rr.first + cp / G) * a.q_heads + h * G + cp % G) * D + d;
            store4<DT>(a.o, at, make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv));
        } else {
            const int64_t slot = (static_cast<int64_t>(h) * pl.slots + pc.slot) * cols + cc;
            *reinterpret_cast<f4 *>(part_o + slot * D + d) = o;
            if (d == 0) *reinterpret_cast<float2 *>(part_ml + 2 * slot) = make_float2(mt, lt);
        }
    };
#pragma unroll
    for (int t = 0; t < NT; ++t) l[t] = col_sum(l[t]);
    if constexpr (TG == 1) {
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            if (!used[t]) continue;
#pragma unroll
            for (int j = 0; j < D / 64; ++j)
#pragma unroll
                for (int i = 0; i < 4; ++i) put(wc * TC + 16 * t + col, 64 * j + 16 * g + 4 * i, dims4(t, j, i), m[t], l[t]);
        }
    } else {
        // the step groups' sums of a column become one
        const int lc = wc * TC + col;
#pragma unroll
        for (int t = 0; t < NT; ++t)
            if (g == 0) {
                lds_ml[tg][lc + 16 * t][0] = m[t];
                lds_ml[tg][lc + 16 * t][1] = l[t];
            }
        __syncthreads();
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            float top = kLowest;
#pragma unroll
            for (int k = 0; k < TG; ++k) top = fmaxf(top, lds_ml[k][lc + 16 * t][0]);
            const float mine = __builtin_amdgcn_exp2f(m[t] - top);
#pragma unroll
            for (int j = 0; j < D / 64; ++j)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    f4 o = dims4(t, j, i);
                    if constexpr (HL == 1) o = f4{o.x + lane_xor<8>(o.x), o.y + lane_xor<8>(o.y), o.z + lane_xor<8>(o.z), o.w + lane_xor<8>(o.w)};
                    *reinterpret_cast<f4 *>(&lds_o[tg][lc + 16 * t][64 * j + 16 * g + 4 * i]) = o * mine;
                }
        }
        __syncthreads();
        const int n = min(TM, pairs - tile0);
        for (int e = threadIdx.x; e < n * (D / 4); e += 256) {
            const int cc = e / (D / 4), d = 4 * (e % (D / 4));
            f4 o{0.f, 0.f, 0.f, 0.f};
            float mt = kLowest, lt = 0.0f;
#pragma unroll
            for (int k = 0; k < TG; ++k) mt = fmaxf(mt, lds_ml[k][cc][0]);
#pragma unroll
            for (int k = 0; k < TG; ++k) {
                o += *reinterpret_cast<const f4 *>(&lds_o[k][cc][d]);
                lt += lds_ml[k][cc][1] * __builtin_amdgcn_exp2f(lds_ml[k][cc][0] - mt);
            }
            put(cc, d, o, mt, lt);
        }
    }
}

// The parts' sums of a tile and KV head become its outputs, `wide` columns (of `cols`) a
// workgroup: D / 4 threads take a part of a column, the rest of the 512 other columns and
// parts, each with a running maximum of its own; LDS joins the parts.
template <int DT, int D>
__global__ __launch_bounds__(512) void attn_join_kernel(Kv4Cache c, KvBatch b, Kv4Attn a, Plan pl, int cols, int wide,
                                                        const float *__restrict__ part_o,
                                                        const float *__restrict__ part_ml) {
    constexpr int L = D / 4, N = 512 / L;
    __shared__ f4 lds_o[N][L];
    __shared__ float lds_ml[N][2];
    const int h = blockIdx.y, G = a.q_heads / c.heads;
    const Piece pc = find_piece<true>(b, a, pl, c.heads, G, blockIdx.x);
    if (pc.parts == 0) return;
    const SeqWork sw = seq_work(b, a, pc.seq);
    const int64_t first = (static_cast<int64_t>(h) * pl.slots + pc.slot) * cols;
    const int idx = threadIdx.x / L, ln = threadIdx.x % L, d = 4 * ln;
    const int at_col = idx % wide, gr = idx / wide, groups = N / wide, cc = blockIdx.z * wide + at_col;
    const bool on = gr < groups && cc < cols && pc.tile * pl.tm + cc < sw.n * G;
    f4 o{0.f, 0.f, 0.f, 0.f};
    float m = kLowest, l = 0.0f;
    if (on) {
#pragma unroll 4
        for (int p = gr; p < pc.parts; p += groups) {
            const int64_t slot = first + static_cast<int64_t>(p) * cols + cc;
            const float2 ml = *reinterpret_cast<const float2 *>(part_ml + 2 * slot);
            const f4 x = *reinterpret_cast<const f4 *>(part_o + slot * D + d);
            const float mn = fmaxf(m, ml.x), f = __builtin_amdgcn_exp2f(m - mn), e = __builtin_amdgcn_exp2f(ml.x - mn);
            l = l * f + ml.y * e;
            o = o * f + x * e;
            m = mn;
        }
    }
    lds_o[idx][ln] = o;
    if (ln == 0) {
        lds_ml[idx][0] = m;
        lds_ml[idx][1] = l;
    }
    __syncthreads();
    if (on && gr == 0) {
        float top = m;
        for (int k = 1; k < groups; ++k) top = fmaxf(top, lds_ml[k * wide + at_col][0]);
        const float f = __builtin_amdgcn_exp2f(m - top);
        o = o * f;
        l = l * f;
        for (int k = 1; k < groups; ++k) {
            const float e = __builtin_amdgcn_exp2f(lds_ml[k * wide + at_col][0] - top);
            l += lds_ml[k * wide + at_col][1] * e;
            o += lds_o[k * wide + at_col][ln] * e;
        }
        const float inv = l > 0.0f ? 1.0f / l : 0.0f;
        const int cp = pc.tile * pl.tm + cc;
        const int64_t at = (static_cast<int64_t>(sw.rr.first + cp / G) * a.q_heads + h * G + cp % G) * D + d;
        store4<DT>(a.o, at, make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv));
    }
}

// The bounds of a plan (see above) for tiles of tm rows of `per` (row, head) pairs a row.
Plan make_plan(const KvBatch &b, int heads, int G, int tm, int target, int min_chunk) {
    const int64_t steps = ((static_cast<int64_t>(b.max_pages) << b.page_shift) + 31) >> 5;
    const int64_t rows = static_cast<int64_t>(b.max_q) * G <= tm ? b.B : static_cast<int64_t>(b.rows) * G / tm + b.B;
    // Each tile may add a part to the even share: where tiles are few, the parts still fit one
    // round of workgroups; where they are many, twice as many parts even the rounds out.
    const int64_t tiles = rows * heads;
    target = 2 * tiles <= target ? target - static_cast<int>(tiles) : 2 * target;
    Plan p{tm, target, min_chunk, 0, 0, 0, 0};
    p.split = b.B <= kMostScanned && steps > min_chunk;
    const int64_t even = (target + heads - 1) / heads, cuts = (steps + min_chunk - 1) / min_chunk;
    const int64_t extra = p.split ? (even < rows * cuts ? even : rows * cuts) : 0;
    p.pieces = static_cast<int>(rows + extra);
    p.items = static_cast<int>(extra < rows ? extra : rows);
    p.slots = static_cast<int>(2 * extra < rows + extra ? 2 * extra : rows + extra);
    return p;
}

// The kernel's shape for a call: by the pairs of one sequence and KV head, the most columns
// a workgroup is offered, so that no wave multiplies mostly padding and short prompts keep
// their waves busy on the context.  Heads of 256 fill the registers with one product of
// columns a wave.
struct Shape {
    int nt, wc;             // products of 16 columns a wave, groups of columns
    Plan plan;
    int cols;               // columns kept for a part
    int64_t sums, stats;    // bytes of the parts' sums and of their statistics
};
Shape attn_shape(const KvBatch &b, const Kv4Cache &c, int q_heads) {
    Shape s;
    const int G = q_heads / c.heads;
    const int64_t pairs = static_cast<int64_t>(b.max_q) * G;
    s.nt = c.D == 256 || pairs <= 16 ? 1 : 2;
    s.wc = pairs <= 16 * s.nt ? 1 : pairs <= 32 * s.nt ? 2 : 4;
    const int tm = 16 * s.nt * s.wc;
    // workgroups that the chip's 256 CUs hold at once
    const int held = c.D == 64 && s.nt == 1 ? 5 : c.D == 128 && s.nt == 1 ? 3 : 2;
    s.plan = make_plan(b, c.heads, G, tm, 256 * held, s.wc == 1 ? 4 : 8);
    s.cols = static_cast<int>(pairs < tm ? pairs : tm);
    s.sums = static_cast<int64_t>(c.heads) * s.plan.slots * s.cols * c.D * 4;
    s.stats = static_cast<int64_t>(c.heads) * s.plan.slots * s.cols * 8;
    return s;
}

template <int DT, int D, int NT, int WC>
void launch_shape(const Shape &s, const Kv4Cache &c, const KvBatch &b, const Kv4Attn &a, float *part_o, float *part_ml,
                  hipStream_t st) {
    const dim3 grid(s.plan.pieces, c.heads), block(256);
    if constexpr (DT != kDtF32) {
        hipLaunchKernelGGL((attn_kernel<DT, D, 0, NT, WC>), grid, block, 0, st, c, b, a, s.plan, s.cols, part_o, part_ml);
    } else {
        if constexpr (NT == 1 && WC == 1) {
            if (s.cols <= 8) {
                hipLaunchKernelGGL((attn_kernel<DT, D, 1, NT, WC>), grid, block, 0, st, c, b, a, s.plan, s.cols, part_o, part_ml);
                return;
            }
        }
        hipLaunchKernelGGL((attn_kernel<DT, D, 2, NT, WC>), grid, block, 0, st, c, b, a, s.plan, s.cols, part_o, part_ml);
    }
}

template <int DT, int D>
hipError_t launch_d(const Kv4Cache &c, const KvBatch &b, const Kv4Attn &a, hipStream_t st) {
    const Shape s = attn_shape(b, c, a.q_heads);
    float *part_o = static_cast<float *>(a.workspace), *part_ml = part_o + s.sums / 4;
    if constexpr (D == 256) {
        if (s.wc == 1) launch_shape<DT, D, 1, 1>(s, c, b, a, part_o, part_ml, st);
        else if (s.wc == 2) launch_shape<DT, D, 1, 2>(s, c, b, a, part_o, part_ml, st);
        else launch_shape<DT, D, 1, 4>(s, c, b, a, part_o, part_ml, st);
    } else {
        if (s.nt == 1) launch_shape<DT, D, 1, 1>(s, c, b, a, part_o, part_ml, st);
        else if (s.wc == 1) launch_shape<DT, D, 2, 1>(s, c, b, a, part_o, part_ml, st);
        else if (s.wc == 2) launch_shape<DT, D, 2, 2>(s, c, b, a, part_o, part_ml, st);
        else launch_shape<DT, D, 2, 4>(s, c, b, a, part_o, part_ml, st);
    }
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || s.plan.items == 0) return e;
    // columns a workgroup: few where there are few tiles, so that many parts are read side
    // by side, up to what its threads hold
    const int64_t most = s.cols < 2048 / D ? s.cols : 2048 / D, even = static_cast<int64_t>(s.plan.items) * c.heads * s.cols / 512;
    const int wide = static_cast<int>(even < 1 ? 1 : even < most ? even : most);
    hipLaunchKernelGGL((attn_join_kernel<DT, D>), dim3(s.plan.items, c.heads, (s.cols + wide - 1) / wide), dim3(512), 0, st,
                       c, b, a, s.plan, s.cols, wide, part_o, part_ml);
    return hipGetLastError();
}

template <int DT>
hipError_t launch_t(const Kv4Cache &c, const KvBatch &b, const Kv4Attn &a, hipStream_t st) {
    if (c.D == 64) return launch_d<DT, 64>(c, b, a, st);
    if (c.D == 128) return launch_d<DT, 128>(c, b, a, st);
    return launch_d<DT, 256>(c, b, a, st);
}

}  // namespace

int64_t kv4_attn_workspace(const Kv4Cache &c, const KvBatch &b, int q_heads, int) {
    const Shape s = attn_shape(b, c, q_heads);
    return s.sums + s.stats;
}

hipError_t launch_kv4_attn(const Kv4Cache &c, const KvBatch &b, const Kv4Attn &a, int dtype, hipStream_t st) {
    if (dtype == kDtF32) return launch_t<kDtF32>(c, b, a, st);
    if (dtype == kDtBf16) return launch_t<kDtBf16>(c, b, a, st);
    return launch_t<kDtF16>(c, b, a, st);
}

}  // namespace rad
