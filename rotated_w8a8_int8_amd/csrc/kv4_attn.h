// kv4_attn.h -- attention over the paged 4-bit cache (gfx950): the kernels of
// kv4_attn.hip (masks by position) and kv4_attn_tree.hip (drafted trees).
//
// Per query row and head: s_t = sm_scale * q.k_t over the tokens t that the row
// sees, o = sum_t exp(s_t - m) v_t / sum_t exp(s_t - m) with m the running
// maximum; k and v are level * scale.
//
// Few query rows leave it to the memory: the cache is read once, as it lies.  199999
// tokens (one f32 row, 40 query and 8 KV heads of 128; 211 MB) take 39 us and 4.6 us for
// the join, 4.9 TB/s in all; 64 bf16 sequences of up to 16000 tokens (506 MB) 89 + 5 us,
// 5.4 TB/s, where a read-only stream reaches 5.8.  Many rows are bound by a SIMD's issue
// of vector and matrix instructions, which overlap little: an 8192-token prompt (687
// GFLOP, bf16) takes 0.81 to 0.84 ms, 0.82 to 0.85 PFLOP/s, where a library product of
// this size reaches 1.2; 77% of a SIMD's cycles issue vector instructions (codes to f16 and
// exponents first) and 37% keep the matrix cores busy.  8 x 16 draft rows over 8192
// tokens take 29 + 6 us.
#pragma once

#include "kv4.h"

namespace rad {
namespace {

constexpr int kWaves = 4;                            // of a workgroup
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

// ---- trees ------------------------------------------------------------------
//
// Bound as the causal form is: 64 nodes over 199936 tokens (262 GFLOP, bf16) take 300 us and 5.9 us for
// the join, 0.87 PFLOP/s; 8 trees of up to 60 nodes over up to 16000 tokens 82 + 9.2 us; 8 nodes over 500 tokens
// 11.7 us, latency.
//
// A sequence's n rows are nodes 0 .. n - 1, at tokens base .. base + n - 1.  Every row sees the tokens
// before base (from `lo` on, where there is a window); among the nodes its mask decides, a bit
// a node.  Only the steps that hold nodes look at masks: two bytes for eight tokens.

// Bits of nodes j .. j + 7 of the mask of `bytes` bytes from mask[first] on (bits outside it are 0).
__device__ __forceinline__ uint32_t mask_bits8(const uint8_t *mask, uint32_t first, int bytes, int j) {
    const int at = j >> 3;                                    // floor, for negative j too
    const uint32_t lo = at >= 0 && at < bytes ? mask[first + at] : 0u, hi = at >= -1 && at + 1 < bytes ? mask[first + at + 1] : 0u;
    return ((lo | hi << 8) >> (j & 7)) & 0xFFu;
}
// Nodes from `from` to n - 1 that a row sees.
__device__ __forceinline__ int mask_count(const uint64_t *mask, int words, int from, int n) {
    int c = 0;
    for (int w = from >> 6; w < words && 64 * w < n; ++w) {
        uint64_t m = mask[w];
        if (from > 64 * w) m &= ~uint64_t(0) << (from - 64 * w);
        if (n < 64 * w + 64) m &= ~uint64_t(0) >> (64 * w + 64 - n);
        c += __popcll(m);
    }
    return c;
}

// The (row, head) pairs of a sequence that share a KV head are the columns of transposed
// matrix products, 16 a wave (32 where there are more), so that nothing crosses lanes
// between the two products of a step of 32 tokens:
//
//   S^T [32 tokens][16 cols] = K Q^T    two 16x16x32 tiles; A: a lane holds D/4 dims of
//                                       one token, one dword (8 dims) per product
//   O^T [D][16 cols]        += V^T P^T  D/16 tiles; A: a lane holds one dim of eight
//                                       tokens, one dword
//
// Row r of score tile u is token 8 (r / 4) + 4 u + r % 4 of the step, so lane (g, c)
// (g = lane / 16, c = lane % 16) comes out of S^T with the scores of tokens 8 g ..
// 8 g + 7 of column c: the B operand that O^T needs against the value octets.
// Codes go from memory to registers to the products; a workgroup's four waves take every
// fourth step of its tile of columns each and are joined through LDS at the end.
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
// inside f16: it is set so that the largest weight met comes to 2^room, and raised only
// when one passes kMost (one vote a step); then scores and scale exponents are looked at
// one by one.  A weight is off by up to 2^-25, half of f16's smallest step, where the
// column's largest is at least 2^(room - 1): by 2^(-24 - room) of it, however small it is
// itself (see kRoom).
typedef unsigned int u4 __attribute__((ext_vector_type(4)));
typedef unsigned int u2 __attribute__((ext_vector_type(2)));
typedef float f4 __attribute__((ext_vector_type(4)));
typedef _Float16 h8 __attribute__((ext_vector_type(8)));

// log2 of the largest weight after a rise.  What a wave's n tokens lose beside a largest weight is
// at most n 2^(-24 - kRoom) of it: for 50000 a tenth of half a step of a bf16 or f16 output, and
// 6e-6 in f32 (1.9e-4 with 4).  The rest of f16's range is what weights may grow by before the next
// rise, and rises cost: an 8192-token bf16 prompt takes 834 us with 4, 846 with 8, 855 with 9, 911
// with 12; an f32 block of 16 rows 67, 69, 70 and 73 us.
template <int DT>
constexpr float kRoom = DT == kDtF32 ? 9.0f : DT == kDtF16 ? 7.0f : 4.0f;
constexpr float kMost = 63488.0f;                   // f16, below its largest, 65504
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
// sm_scale log2(e) 2^-e, never 0: a masked score stays -inf.  At most 2^90: products and key scales come to
// less than 2^37, so no score is infinite, and at more than that any difference is far past exp's range.
__device__ __forceinline__ float score_factor(float sm_scale, int e) {
    return fminf(fmaxf(__builtin_amdgcn_ldexpf(sm_scale * kLog2e, -e), 1e-30f), 0x1p90f);
}
// log2 of a power of two above a value's scale; scales of 0 weigh nothing, but count
__device__ __forceinline__ float scale_log2(float vs) {
    return vs > 0.0f ? static_cast<float>(__builtin_amdgcn_frexp_expf(vs)) : -24.0f;
}
// The reference exponent for a largest log2 weight `most`: never above most - room by rounding.
template <int DT>
__device__ __forceinline__ float reference(float m, float most) {
    return fmaxf(m, fmaf(fabsf(most), -0x1p-22f, most - kRoom<DT>));
}
// Beyond kNear (the lowest, the mark of nothing seen, aside) f32 holds a reference to half a unit or worse, and with
// it what the room leaves: there 2^(score - m) is held to 1, every step.  The vote's third compare and the minimum
// cost 1% of a prompt (816 -> 824 us) and of short calls (9.69 -> 9.81 us).
constexpr float kNear = 0x1p22f;
__device__ __forceinline__ float most_power(float m) { return fabsf(m) > kNear && m > -0x1.8p127f ? 0.0f : INFINITY; }

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
// at one sequence, 64 at a time; beyond kMostScanned sequences nothing is split, and a
// workgroup finds its tile without the others' lengths (find_uncut): every workgroup
// looking at every sequence grew with their square (8 KV heads, 30 tokens: 4096 single rows
// 616 us, 184 us this way; 4096 blocks of 8 rows 3.0 and 0.9 ms).
constexpr int kMostScanned = 512;
struct Plan {
    int tm, target, min_chunk, split;     // rows a tile; workgroups wanted; least steps a part; 0: one part a tile
    int pieces, items, slots;             // bounds a KV head: workgroups, tiles in several parts, parts of those
    int per;                              // pieces of a KV head that one of its XCDs takes; 0: no matter which
};
struct Piece {
    int seq, tile, part, parts, slot;     // parts 0: none.  slot: place among the parts kept apart
};

// Arguments of a kernel below: these, a count of columns and two addresses (see Kv4Attn).
static_assert(sizeof(Kv4Cache) + sizeof(KvBatch) + sizeof(Kv4Attn) + sizeof(Plan) + 24 <= 192, "three lines");

// Workgroups go to the eight XCDs in turn, each with an L2 of its own.  Where tiles share codes, a KV head's
// pieces stay on one XCD (on 8 / heads of them in turn, where there are fewer heads), the tiles of a part
// side by side (8 trees of up to 60 nodes over 16000 tokens 87 -> 82 us, an 8192-token prompt 850 -> 844 us).
struct Place {
    int x, h;
};
// log2 of the largest power of two up to 8 that divides heads.
__host__ __device__ __forceinline__ int common8(int heads) { return heads & 1 ? 0 : heads & 2 ? 1 : heads & 4 ? 2 : 3; }
__device__ __forceinline__ Place piece_place(const Plan &pl, int heads) {
    if (pl.per == 0) return Place{static_cast<int>(blockIdx.x), static_cast<int>(blockIdx.y)};
    const int g = common8(heads), xcd = blockIdx.x & 7, j = blockIdx.x >> 3;
    return Place{(j << (3 - g)) + (xcd >> g), (static_cast<int>(blockIdx.y) << g) + (xcd & ((1 << g) - 1))};
}

// Rows of a sequence that a call handles, and what they see together.
struct SeqWork {
    RowRange rr;
    int n, len, pos0, lo, hi;             // rows handled, tokens, first row's position, tokens [lo, hi)
};
template <bool TREE>
__device__ __forceinline__ SeqWork seq_work(const KvBatch &b, const Kv4Attn &a, int seq) {
    SeqWork s;
    s.rr = kv_rows(b, seq);
    s.n = min(s.rr.n, b.max_q);
    s.len = kv_len(b, seq);
    s.pos0 = s.len - s.rr.n;
    if constexpr (TREE) {
        s.lo = a.window > 0 ? max(0, s.pos0 - a.window) : 0;
        s.hi = s.pos0 + s.n > 0 ? max(s.len, s.lo) : s.lo;
        return s;
    }
    s.lo = seen(max(s.pos0, 0), s.len, a.causal, a.window).lo;
    s.hi = a.causal ? s.pos0 + s.n : (s.pos0 + s.n > 0 ? s.len : 0);
    if (s.hi < s.lo) s.hi = s.lo;
    return s;
}
__device__ __forceinline__ int steps_of(int lo, int hi) { return hi > lo ? ((hi + 31) >> 5) - (lo >> 5) : 0; }

// Steps a part: about `target` parts over all sequences and KV heads, rounded up.
__device__ __forceinline__ int chunk_of(uint64_t total, const Plan &pl, int heads) {
    const uint64_t all = total * static_cast<uint32_t>(heads) + static_cast<uint32_t>(pl.target - 1);
    const int even = all >> 32 ? static_cast<int>(min(all / static_cast<uint32_t>(pl.target), uint64_t(1) << 30))
                               : static_cast<int>(static_cast<uint32_t>(all) / static_cast<uint32_t>(pl.target));
    return max(even, pl.min_chunk);
}

// The x-th piece of a KV head where no tile is cut, without a look at every sequence.  One tile
// a sequence: piece b is its tile.  More: sequence b's tiles are among the pieces from floor(q_start[b] G /
// tm) + b on, which rises by at least ceil(n G / tm) to the next sequence's, and ends below rows G / tm + B;
// 64 sequences are looked at a trip.  Every lane of the wave calls it and gets the same answer.
template <bool TREE>
__device__ __forceinline__ Piece find_uncut(const KvBatch &b, const Kv4Attn &a, const Plan &pl, int G, int x) {
    int seq = x, first = x;
    if (static_cast<int64_t>(b.max_q) * G > pl.tm) {
        const int lane = threadIdx.x & 63, log_tm = __builtin_ctz(static_cast<uint32_t>(pl.tm));       // 16 or 32
        auto first_of = [&](int i) { return (static_cast<int64_t>(b.q_start ? b.q_start[i] : i) * G >> log_tm) + i; };
        seq = 0;
        for (int n = b.B; n > 1;) {                           // the sequence lies in [seq, seq + n)
            const int each = (n + 63) >> 6, i = lane * each;
            const int at = max(__popcll(__ballot(i < n && first_of(seq + min(i, n - 1)) <= x)) - 1, 0) * each;
            seq += at;
            n = min(each, n - at);
        }
        first = static_cast<int>(first_of(seq));
    }
    if (seq >= b.B) return Piece{0, 0, 0, 0, 0};
    const int tiles = (seq_work<TREE>(b, a, seq).n * G + pl.tm - 1) / pl.tm, tile = x - first;
    return tile >= 0 && tile < tiles ? Piece{seq, tiles - 1 - tile, 0, 1, 0} : Piece{0, 0, 0, 0, 0};
}

// The x-th piece of a KV head (ITEMS false), or the x-th tile in several parts (true).
// Every lane of the wave calls it and gets the same answer.  ONCE: a sequence is one tile, so that no order
// of tiles matters, and the count of tiles, held early, would be the one register too many (64 decoding
// sequences of up to 16000 tokens, bf16: 94 us, 96 us with it in scratch).
template <bool ITEMS, bool ONCE, bool TREE>
__device__ __forceinline__ Piece find_piece(const KvBatch &b, const Kv4Attn &a, const Plan &pl, int heads, int G, int x) {
    const int lane = threadIdx.x & 63;
    if (b.B == 1) {
        const SeqWork s = seq_work<TREE>(b, a, 0);
        const int tiles = (s.n * G + pl.tm - 1) / pl.tm, steps = steps_of(s.lo, s.hi);
        const int chunk = chunk_of(static_cast<uint64_t>(tiles) * static_cast<uint32_t>(steps), pl, heads);
        const int parts = pl.split ? max(1, (steps + chunk - 1) / chunk) : 1;
        int part, tile, slot;
        if constexpr (ITEMS || ONCE) {
            part = ITEMS ? 0 : x % parts, tile = ITEMS ? x : x / parts, slot = ITEMS ? x * parts : x;
            if (tile >= tiles || (ITEMS && parts == 1)) return Piece{0, 0, 0, 0, 0};
        } else if (!pl.split) {                               // short calls: no division
            if (x >= tiles) return Piece{0, 0, 0, 0, 0};
            part = 0, tile = x, slot = x;
        } else {
            if (tiles == 0 || x / tiles >= parts) return Piece{0, 0, 0, 0, 0};
            part = x / tiles, tile = x % tiles, slot = tile * parts + part;
        }
        if (parts > 1 && slot + (ITEMS ? parts : 1) > pl.slots) return Piece{0, 0, 0, 0, 0};
        return Piece{0, tiles - 1 - tile, part, parts, slot};
    }
    if (b.B > kMostScanned) return ITEMS ? Piece{0, 0, 0, 0, 0} : find_uncut<TREE>(b, a, pl, G, x);
    uint64_t total = 0;
    if (pl.split) {
        for (int b0 = 0; b0 < b.B; b0 += 64) {
            uint64_t t = 0;
            if (b0 + lane < b.B) {
                const SeqWork s = seq_work<TREE>(b, a, b0 + lane);
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
            const SeqWork s = seq_work<TREE>(b, a, b0 + lane);
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
            int tile;
            if constexpr (ITEMS || ONCE) {
                tile = ITEMS ? local : local / p.parts;
                p.part = ITEMS ? 0 : local % p.parts;
            } else if (!pl.split) {                           // short calls: no division
                tile = local;
                p.part = 0;
            } else {
                const int n = __builtin_amdgcn_readlane(tiles, src);
                tile = local % n;
                p.part = local / n;
            }
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

// A wave's share of a piece.
struct Share {
    int first_row, len, pos0, pairs;      // the sequence: first row, tokens, first row's position, (row, head) pairs
    int tile0;                            // first pair of the tile
    int begin, end;                       // steps: begin, begin + kWaves, .. below end
    int open_lo, open_hi;                 // steps [open_lo, open_hi) that all the tile's rows see whole
    TokenRange tile_r;                    // what the tile's rows see together
};
template <int TM, bool TREE>
__device__ __forceinline__ Share wave_share(const KvBatch &b, const Kv4Attn &a, const Piece &pc, int seq, int G, int tg) {
    const SeqWork sw = seq_work<TREE>(b, a, seq);
    Share s;
    s.first_row = sw.rr.first;
    s.len = sw.len;
    s.pos0 = sw.pos0;
    s.pairs = sw.n * G;
    s.tile0 = pc.tile * TM;
    const int first = s.tile0 / G, last = (min(s.tile0 + TM, s.pairs) - 1) / G;
    // rows see ever later tokens: the first row's beginning and the last row's end
    s.tile_r = TokenRange{seen(max(s.pos0 + first, 0), s.len, a.causal, a.window).lo,
                          seen(s.pos0 + last, s.len, a.causal, a.window).hi};
    if constexpr (TREE) s.tile_r = TokenRange{sw.lo, s.pos0 + last >= 0 ? s.len : 0};
    if (s.tile_r.hi < s.tile_r.lo) s.tile_r.hi = s.tile_r.lo;
    const int step0 = s.tile_r.lo >> 5, steps = steps_of(s.tile_r.lo, s.tile_r.hi);
    const int each = (steps + pc.parts - 1) / pc.parts;
    s.begin = __builtin_amdgcn_readfirstlane(step0 + pc.part * each + tg);
    s.end = __builtin_amdgcn_readfirstlane(step0 + min((pc.part + 1) * each, steps));
    s.open_lo = __builtin_amdgcn_readfirstlane((seen(max(s.pos0 + last, 0), s.len, a.causal, a.window).lo + 31) >> 5);
    s.open_hi = __builtin_amdgcn_readfirstlane(seen(s.pos0 + first, s.len, a.causal, a.window).hi >> 5);
    if constexpr (TREE) {                                     // with a window a row's begins n tokens late at most
        s.open_lo = __builtin_amdgcn_readfirstlane(((a.window > 0 ? max(0, s.pos0 + sw.rr.n - a.window) : 0) + 31) >> 5);
        s.open_hi = __builtin_amdgcn_readfirstlane(max(s.pos0, 0) >> 5);
        if (s.pos0 + first < 0) s.open_hi = 0;
    }
    return s;
}

// What row ci of the sequence sees; for a tree aside from the nodes that its mask hides.
template <bool TREE>
__device__ __forceinline__ TokenRange seen_by(const KvBatch &b, const Kv4Attn &a, const Share &s, int seq, int ci) {
    if constexpr (!TREE) return seen(s.pos0 + ci, s.len, a.causal, a.window);
    TokenRange r{0, s.pos0 + ci >= 0 ? s.len : 0};
    if (a.window > 0) {
        const int nodes = s.len - s.pos0;
        const int path = mask_count(a.mask + static_cast<int64_t>(s.first_row + ci) * a.words(), a.words(), max(0, -s.pos0), nodes);
        r.lo = max(0, min(s.pos0, s.pos0 + path - a.window));    // nodes themselves lie in every window
    }
    return r;
}

// Where a step's tokens lie.  Page ids come through the scalar cache (no kernel writes them
// while this one runs): a vector load here would wait for every code on its way.
struct Pages {
    typedef const __attribute__((address_space(4))) int32_t *Ids;
    Ids table;
    int per_page, end, pages, heads, h, shift;
    __device__ __forceinline__ Pages(const Kv4Cache &c, const KvBatch &b, int seq, int h_, int end_)
        : table((Ids)(b.block_table + static_cast<int64_t>(seq) * b.max_pages)), per_page(b.page_shift - 5), end(end_),
          pages(c.pages), heads(c.heads), h(h_), shift(c.page_shift) {}
    // page of a step, -1 past the end
    __device__ __forceinline__ int id(int step) const { return step < end ? table[step >> per_page] : -1; }
    // index of the step's first token in the cache's [pages][heads][page] order; for a step past the
    // end or on an absent page one that exists
    __device__ __forceinline__ int64_t token(int page, int step) const {
        const int64_t p = page >= 0 && page < pages ? page : 0;
        return ((p * heads + h) << shift) + (step < end ? (step << 5) & ((1 << shift) - 1) : 0);
    }
};

// Where a column's sums go: the output, or among the parts kept apart.
template <int DT, int D, bool TREE>
struct Output {
    const Kv4Attn &a;
    const Plan &pl;
    const Piece &pc;
    float *part_o, *part_ml;
    int first_row, tile0, cols, h, G;
    // four dims from d of the tile's column cc, with its reference exponent and normaliser
    __device__ __forceinline__ void put(int cc, int d, f4 o, float m, float l) const {
        if (pc.parts == 1) {
            const float inv = l > 0.0f ? 1.0f / l : 0.0f;
            const int cp = tile0 + cc;
            const int64_t at = (static_cast<int64_t>(first_row + cp / G) * a.q_heads + h * G + cp % G) * D + d;
            store4<DT>(a.o, at, make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv));
        } else {
            const int64_t slot = (static_cast<int64_t>(h) * pl.slots + pc.slot) * cols + cc;
            *reinterpret_cast<f4 *>(part_o + slot * D + d) = o;
            if (d == 0) *reinterpret_cast<float2 *>(part_ml + 2 * slot) = make_float2(m, l);
        }
    }
    // the column's statistics, where they are asked for (apart from the outputs, whose loop they slowed down)
    __device__ __forceinline__ bool wants_stats() const { return !TREE && pc.parts == 1 && a.stats; }
    __device__ __forceinline__ void put_stats(int cc, float m, float l) const {
        const int cp = tile0 + cc;
        a.stats[static_cast<int64_t>(first_row + cp / G) * a.q_heads + h * G + cp % G] = make_float2(m, l > 0.0f ? 1.0f / l : 0.0f);
    }
};
// The step groups' sums of n columns become one (each group's taken to the common maximum).
template <int TG, int TM, int D, class Out>
__device__ __forceinline__ void join_groups(const Out &out, float (&lds_o)[TG][TM][D + 4], float (&lds_ml)[TG][TM][2], int n) {
    for (int e = threadIdx.x; e < n * (D / 4); e += 64 * kWaves) {
        const int cc = e / (D / 4), d = 4 * (e % (D / 4));
        f4 o{0.f, 0.f, 0.f, 0.f};
        float m = kLowest, l = 0.0f;
#pragma unroll
        for (int k = 0; k < TG; ++k) m = fmaxf(m, lds_ml[k][cc][0]);
#pragma unroll
        for (int k = 0; k < TG; ++k) {
            o += *reinterpret_cast<const f4 *>(&lds_o[k][cc][d]);
            l += lds_ml[k][cc][1] * __builtin_amdgcn_exp2f(lds_ml[k][cc][0] - m);
        }
        out.put(cc, d, o, m, l);
    }
    if (out.wants_stats() && static_cast<int>(threadIdx.x) < n) {
        const int cc = threadIdx.x;
        float m = kLowest, l = 0.0f;
        for (int k = 0; k < TG; ++k) m = fmaxf(m, lds_ml[k][cc][0]);
        for (int k = 0; k < TG; ++k) l += lds_ml[k][cc][1] * __builtin_amdgcn_exp2f(lds_ml[k][cc][0] - m);
        out.put_stats(cc, m, l);
    }
}

// blockIdx: x piece, y KV head.  A tile has 16 columns, `cols` of them in use at most.  Parts of a tile in several leave their sums in part_o [heads][slots][cols][D] and
// part_ml [..][cols][2]; the others write the outputs.  ONCE: no other workgroup reads the
// codes, so they are loaded nontemporally (200K tokens 50 -> 46 us; with several tiles of heads
// of 256 4096 tokens take 246 us that way, 219 us without).  Three waves a SIMD where 168 registers do for
// them (64 sequences 98 us, 102 us with two).
template <int DT, int D, int HL, bool ONCE, bool TREE>
__global__ __launch_bounds__(256, D == 128 && HL != 2 ? 3 : 2) void attn_kernel(Kv4Cache c, KvBatch b, Kv4Attn a, Plan pl, int cols,
                                                      float *part_o, float *part_ml) {
    constexpr int TG = kWaves, TM = 16, NK = D / 32;
    __shared__ float lds_o[TG][TM][D + 4], lds_ml[TG][TM][2];
    const int lane = threadIdx.x & 63, tg = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int g = lane >> 4, col = lane & 15;
    const Place place = ONCE ? Place{static_cast<int>(blockIdx.x), static_cast<int>(blockIdx.y)} : piece_place(pl, c.heads);
    const int h = place.h, G = a.q_heads / c.heads;
    const Piece pc = find_piece<false, ONCE, TREE>(b, a, pl, c.heads, G, place.x);
    if (pc.parts == 0) return;
    const int seq = __builtin_amdgcn_readfirstlane(pc.seq);
    const Share sh = wave_share<TM, TREE>(b, a, pc, seq, G, tg);

    // this lane's column: pair cp is row cp / G of the sequence, head h * G + cp % G
    const int cp = sh.tile0 + (HL == 1 ? col & 7 : col);
    const bool used = cp < sh.pairs;
    const int ci = used ? cp / G : 0, cg = used ? cp % G : 0;
    const TokenRange tr = used ? seen_by<TREE>(b, a, sh, seq, ci) : sh.tile_r;
    // Bytes of the masks, fewer than 2^22 rows of at most 64 words, count in 32 bits: as an address it is a register
    // too many (32 chains of three, 16000 tokens: 64 us, 61 us so; attn_wide_kernel has no such limit, and
    // 8 nodes over 500 tokens lose 0.3 us to it).
    const uint8_t *const masks = reinterpret_cast<const uint8_t *>(a.mask);
    const uint32_t mask = TREE ? static_cast<uint32_t>(sh.first_row + ci) * static_cast<uint32_t>(8 * a.words()) : 0u;
    const int64_t qrow = (static_cast<int64_t>(sh.first_row + ci) * a.q_heads + h * G + cg) * D;
    // the query's values are asked for first, then the first steps
    float qv[NK][8];
#pragma unroll
    for (int j = 0; j < NK; ++j) {
        const int64_t at = qrow + g * (D / 4) + 8 * j;
        const float4 x = load4<DT>(a.q, at), y = load4<DT>(a.q, at + 4);
        qv[j][0] = x.x; qv[j][1] = x.y; qv[j][2] = x.z; qv[j][3] = x.w;
        qv[j][4] = y.x; qv[j][5] = y.y; qv[j][6] = y.z; qv[j][7] = y.w;
    }

    // A wave's steps go through a ring: two (one, where the sums fill the registers) on
    // their way while one is worked on.  Past the end the loads go on, to a page that exists
    // (cached, unused): were they conditional, the wait for a step's codes would have to be
    // a wait for the later ones too.
    const Pages pages(c, b, seq, h, sh.end);
    constexpr int NB = D == 256 ? 2 : 3;
    Step<D> ring[NB];
    int page[NB];
#pragma unroll
    for (int k = 0; k < NB; ++k) page[k] = pages.id(sh.begin + k * TG);
#pragma unroll
    for (int k = 0; k < NB - 1; ++k) load_step<D, ONCE>(ring[k], c, pages.token(page[k], sh.begin + k * TG), g, col);

    u4 qf[NK], ql[HL == 2 ? NK : 1];
    float scale;
    {
        float big = 0.0f;
#pragma unroll
        for (int j = 0; j < NK; ++j)
#pragma unroll
            for (int i = 0; i < 8; ++i) big = fmaxf(big, fabsf(qv[j][i]));
        big = col_max(big);
        // largest value to [2^9, 2^10), undone in the scores' factor (both exact)
        const int e = big > 0.0f ? 10 - __builtin_amdgcn_frexp_expf(big) : 0;
#pragma unroll
        for (int j = 0; j < NK; ++j) {
#pragma unroll
            for (int i = 0; i < 8; ++i) qv[j][i] = used ? __builtin_amdgcn_ldexpf(qv[j][i], e) : 0.0f;
            if constexpr (HL == 0) {
                qf[j] = f16_pack8(qv[j]);
            } else {
                u4 hi, low;
                f16_split8(qv[j], hi, low);
                if constexpr (HL == 2) ql[j] = low;
                qf[j] = HL == 1 && col >= 8 ? low : hi;
            }
        }
        scale = score_factor(a.sm_scale, e);
    }

    float m = kLowest, l = 0.0f;
    f4 acc[D / 16];
#pragma unroll
    for (int j = 0; j < D / 16; ++j) acc[j] = f4{0.f, 0.f, 0.f, 0.f};

    auto work = [&](Step<D> &cur, int step) {
        float s[8];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            f4 x{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int j = 0; j < NK; ++j) {
                const u4 kf = levels8(cur.k[u][j]);
                if constexpr (HL == 2) x = mma16(kf, ql[j], x);
                x = mma16(kf, qf[j], x);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                float y = x[i];
                if constexpr (HL == 1) y += lane_xor<8>(y);          // high and low part of the query
                s[4 * u + i] = times_half(y, cur.ks, 4 * u + i);
            }
        }
        if (step < sh.open_lo || step >= sh.open_hi) {
            const int t0 = (step << 5) + 8 * g;
            const uint32_t bits = TREE ? mask_bits8(masks, mask, 8 * a.words(), t0 - sh.pos0) : 0u;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const bool on = t0 + i >= tr.lo && t0 + i < tr.hi && (!TREE || t0 + i < sh.pos0 || (bits >> i & 1));
                s[i] = on ? s[i] : -INFINITY;
                // a scale past the sequence's end may be anything
                cur.vs[i >> 1] &= on ? 0xFFFFFFFFu : (i & 1 ? 0x0000FFFFu : 0xFFFF0000u);
            }
        }
        float w[8], sum = 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float p = __builtin_amdgcn_exp2f(fmaf(s[i], scale, -m));
            sum += p;
            w[i] = times_half(p, cur.vs, i);
        }
        if (__any(!(max8(w) <= kMost && sum <= kMostP && fabsf(m) <= kNear))) {         // also the first step: m is the lowest
            float most = -INFINITY;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float vs = times_half(1.0f, cur.vs, i);
                most = fmaxf(most, fmaf(s[i], scale, scale_log2(vs)));
            }
            const float mn = reference<DT>(m, col_max(most)), shrink = __builtin_amdgcn_exp2f(m - mn);
            m = mn;
            l *= shrink;
#pragma unroll
            for (int j = 0; j < D / 16; ++j) acc[j] *= shrink;
            const float top = most_power(m);
            sum = 0.0f;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float p = __builtin_amdgcn_exp2f(fminf(fmaf(s[i], scale, -m), top));
                sum += p;
                w[i] = times_half(p, cur.vs, i);
            }
        }
        l += sum;
        u4 wf, wl;
        if constexpr (HL == 0) {
            wf = f16_pack8(w);
        } else {
            u4 hi;
            f16_split8(w, hi, wl);
            wf = HL == 1 && col >= 8 ? wl : hi;
        }
#pragma unroll
        for (int j = 0; j < D / 64; ++j) {
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                const u4 vf = levels8(cur.v[j][x]);
                if constexpr (HL == 2) acc[4 * j + x] = mma16(vf, wl, acc[4 * j + x]);
                acc[4 * j + x] = mma16(vf, wf, acc[4 * j + x]);
            }
        }
    };
    for (int step = sh.begin; step < sh.end;) {
#pragma unroll
        for (int k = 0; k < NB; ++k) {
            constexpr int ahead = NB - 1;
            const int in = (k + ahead) % NB;
            load_step<D, ONCE>(ring[in], c, pages.token(page[in], step + ahead * TG), g, col);
            const int now = page[k];
            page[k] = pages.id(step + NB * TG);
            if (now >= 0 && now < c.pages) work(ring[k], step);
            step += TG;
            if (step >= sh.end) break;
        }
    }

    // lane (g, c) holds dims 64 j + 16 g .. + 15 of column c: acc[4 j + x][i] is 4 i + x of them
    auto dims4 = [&](int j, int i) { return f4{acc[4 * j][i], acc[4 * j + 1][i], acc[4 * j + 2][i], acc[4 * j + 3][i]}; };
    const Output<DT, D, TREE> out{a, pl, pc, part_o, part_ml, sh.first_row, sh.tile0, cols, h, G};
    l = col_sum(l);
    if (g == 0) {
        lds_ml[tg][col][0] = m;
        lds_ml[tg][col][1] = l;
    }
    __syncthreads();
    float top = kLowest;
#pragma unroll
    for (int k = 0; k < TG; ++k) top = fmaxf(top, lds_ml[k][col][0]);
    const float mine = __builtin_amdgcn_exp2f(m - top);
#pragma unroll
    for (int j = 0; j < D / 64; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f4 o = dims4(j, i);
            if constexpr (HL == 1) o = f4{o.x + lane_xor<8>(o.x), o.y + lane_xor<8>(o.y), o.z + lane_xor<8>(o.z), o.w + lane_xor<8>(o.w)};
            *reinterpret_cast<f4 *>(&lds_o[tg][col][64 * j + 16 * g + 4 * i]) = o * mine;
        }
    __syncthreads();
    join_groups<TG, TM, D>(out, lds_o, lds_ml, min(TM, sh.pairs - sh.tile0));
}

// ---- 32 columns a wave -------------------------------------------------------
//
// The same two products with 32x32x16 matrix operations, half as many, one column and 16
// tokens a lane (g = lane / 32, c = lane % 32):
//
//   S^T [32 tokens][32 cols]: A: a lane holds D/2 dims of one token, one dword a product
//   O^T [D][32 cols]: D/32 tiles, two products each of 16 tokens; A: a lane holds one dim of
//                     eight tokens, one dword
//
// Row r of S^T is token 16 (r / 16) + 8 (r / 4 % 2) + 4 (r / 8 % 2) + r % 4, so that lane (g,
// c) comes out with octets g and 2 + g of column c, what O^T's two products take.
typedef float f16v __attribute__((ext_vector_type(16)));
__device__ __forceinline__ f16v mma32(u4 a, u4 b, f16v c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(h8, a), __builtin_bit_cast(h8, b), c, 0, 0, 0);
}

template <int D>
struct WideStep {
    uint32_t k[D / 16];         // D / 2 dims of a token
    uint32_t v[2][D / 32];      // octets g and 2 + g: dims D / 32 * r ..
    u4 ks[2], vs[2];            // f16 scales of the octets
};
template <int D>
__device__ __forceinline__ void load_step(WideStep<D> &s, const Kv4Cache &c, int64_t tok, int g, int r) {
    const int row = 16 * (r >> 4) + 8 * ((r >> 2) & 1) + 4 * ((r >> 3) & 1) + (r & 3);
    const u4 *kp = reinterpret_cast<const u4 *>(c.k_codes + (tok + row) * (D / 2) + g * (D / 4));
#pragma unroll
    for (int j = 0; j < D / 64; ++j) {
        const u4 x = kp[j];
#pragma unroll
        for (int i = 0; i < 4; ++i) s.k[4 * j + i] = x[i];
    }
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        const uint32_t *vp = reinterpret_cast<const uint32_t *>(c.v_codes) + ((tok >> 3) + 2 * e + g) * D + D / 32 * r;
        if constexpr (D == 64) {
            const u2 x = *reinterpret_cast<const u2 *>(vp);
            s.v[e][0] = x.x;
            s.v[e][1] = x.y;
        } else {
            const u4 x = *reinterpret_cast<const u4 *>(vp);
#pragma unroll
            for (int i = 0; i < 4; ++i) s.v[e][i] = x[i];
        }
        s.ks[e] = *reinterpret_cast<const u4 *>(c.k_scale + tok + 16 * e + 8 * g);
        s.vs[e] = *reinterpret_cast<const u4 *>(c.v_scale + tok + 16 * e + 8 * g);
    }
}
__device__ __forceinline__ float max16(const float (&s)[16]) {
    float m = fmaxf(s[0], s[1]);
#pragma unroll
    for (int i = 2; i < 16; i += 2) m = fmaxf(m, fmaxf(s[i], s[i + 1]));
    return m;
}

// Four dims in a row of a lane's column, from register r of the tiles.
template <int D>
__device__ __forceinline__ f4 wide_dims(const f16v (&acc)[D / 32], int r) {
    if constexpr (D == 64) return f4{acc[0][r], acc[1][r], acc[0][r + 1], acc[1][r + 1]};
    else return f4{acc[0][r], acc[1][r], acc[2][r], acc[3][r]};
}

// As attn_kernel, with 32 columns a tile.  SP: f32 queries and weights in two parts.
template <int DT, int D, bool SP, bool TREE>
__global__ __launch_bounds__(256, 2) void attn_wide_kernel(Kv4Cache c, KvBatch b, Kv4Attn a, Plan pl, int cols,
                                                           float *part_o, float *part_ml) {
    constexpr int TG = kWaves, TM = 32, NK = D / 16, ND = D / 32;
    __shared__ float lds_o[TG][TM][D + 4], lds_ml[TG][TM][2];
    const int lane = threadIdx.x & 63, tg = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int g = lane >> 5, col = lane & 31;
    const Place place = piece_place(pl, c.heads);
    const int h = place.h, G = a.q_heads / c.heads;
    const Piece pc = find_piece<false, false, TREE>(b, a, pl, c.heads, G, place.x);
    if (pc.parts == 0) return;
    const int seq = __builtin_amdgcn_readfirstlane(pc.seq);
    const Share sh = wave_share<TM, TREE>(b, a, pc, seq, G, tg);

    // this lane's column: pair cp is row cp / G of the sequence, head h * G + cp % G
    const int cp = sh.tile0 + col;
    const bool used = cp < sh.pairs;
    const int ci = used ? cp / G : 0, cg = used ? cp % G : 0;
    const TokenRange tr = used ? seen_by<TREE>(b, a, sh, seq, ci) : sh.tile_r;
    const uint8_t *const mask = TREE ? reinterpret_cast<const uint8_t *>(a.mask + static_cast<int64_t>(sh.first_row + ci) * a.words()) : nullptr;
    const int64_t qrow = (static_cast<int64_t>(sh.first_row + ci) * a.q_heads + h * G + cg) * D;
    float qv[NK][8];
#pragma unroll
    for (int j = 0; j < NK; ++j) {
        const int64_t at = qrow + g * (D / 2) + 8 * j;
        const float4 x = load4<DT>(a.q, at), y = load4<DT>(a.q, at + 4);
        qv[j][0] = x.x; qv[j][1] = x.y; qv[j][2] = x.z; qv[j][3] = x.w;
        qv[j][4] = y.x; qv[j][5] = y.y; qv[j][6] = y.z; qv[j][7] = y.w;
    }

    const Pages pages(c, b, seq, h, sh.end);
    constexpr int NB = 2;
    WideStep<D> ring[NB];
    int page[NB];
#pragma unroll
    for (int k = 0; k < NB; ++k) page[k] = pages.id(sh.begin + k * TG);
#pragma unroll
    for (int k = 0; k < NB - 1; ++k) load_step<D>(ring[k], c, pages.token(page[k], sh.begin + k * TG), g, col);

    u4 qf[NK], ql[SP ? NK : 1];
    float scale;
    {
        float big = 0.0f;
#pragma unroll
        for (int j = 0; j < NK; ++j)
#pragma unroll
            for (int i = 0; i < 8; ++i) big = fmaxf(big, fabsf(qv[j][i]));
        big = fmaxf(big, __shfl_xor(big, 32));
        const int e = big > 0.0f ? 10 - __builtin_amdgcn_frexp_expf(big) : 0;
#pragma unroll
        for (int j = 0; j < NK; ++j) {
#pragma unroll
            for (int i = 0; i < 8; ++i) qv[j][i] = used ? __builtin_amdgcn_ldexpf(qv[j][i], e) : 0.0f;
            if constexpr (SP) f16_split8(qv[j], qf[j], ql[j]);
            else qf[j] = f16_pack8(qv[j]);
        }
        scale = score_factor(a.sm_scale, e);
    }

    float m = kLowest, l = 0.0f;
    f16v acc[ND];
#pragma unroll
    for (int x = 0; x < ND; ++x)
#pragma unroll
        for (int i = 0; i < 16; ++i) acc[x][i] = 0.0f;

    auto work = [&](WideStep<D> &cur, int step) {
        // the wave with products to issue goes before the one with exponents (8192 tokens
        // 860 -> 827 us)
        __builtin_amdgcn_s_setprio(1);
        f16v st;
#pragma unroll
        for (int i = 0; i < 16; ++i) st[i] = 0.0f;
#pragma unroll
        for (int j = 0; j < NK; ++j) {
            const u4 kf = levels8(cur.k[j]);
            if constexpr (SP) st = mma32(kf, ql[j], st);
            st = mma32(kf, qf[j], st);
        }
        __builtin_amdgcn_s_setprio(0);
        float s[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) s[i] = times_half(st[i], cur.ks[i >> 3], i & 7);
        if (step < sh.open_lo || step >= sh.open_hi) {
            const int t0 = (step << 5) + 8 * g;
            const uint32_t bits = TREE ? mask_bits8(mask, 0, 8 * a.words(), t0 - sh.pos0) |
                                             mask_bits8(mask, 0, 8 * a.words(), t0 + 16 - sh.pos0) << 8 : 0u;
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const int t = t0 + 16 * (i >> 3) + (i & 7);
                const bool on = t >= tr.lo && t < tr.hi && (!TREE || t < sh.pos0 || (bits >> i & 1));
                s[i] = on ? s[i] : -INFINITY;
                // a scale past the sequence's end may be anything
                cur.vs[i >> 3][(i & 7) >> 1] &= on ? 0xFFFFFFFFu : (i & 1 ? 0x0000FFFFu : 0xFFFF0000u);
            }
        }
        float w[16], sum = 0.0f;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const float p = __builtin_amdgcn_exp2f(fmaf(s[i], scale, -m));
            sum += p;
            w[i] = times_half(p, cur.vs[i >> 3], i & 7);
        }
        if (__any(!(max16(w) <= kMost && sum <= kMostP && fabsf(m) <= kNear))) {                        // also the first step: m is the lowest
            float most = -INFINITY;
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const float vs = times_half(1.0f, cur.vs[i >> 3], i & 7);
                most = fmaxf(most, fmaf(s[i], scale, scale_log2(vs)));
            }
            most = fmaxf(most, __shfl_xor(most, 32));
            const float mn = reference<DT>(m, most), shrink = __builtin_amdgcn_exp2f(m - mn);
            m = mn;
            l *= shrink;
#pragma unroll
            for (int x = 0; x < ND; ++x) acc[x] *= shrink;
            const float top = most_power(m);
            sum = 0.0f;
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const float p = __builtin_amdgcn_exp2f(fminf(fmaf(s[i], scale, -m), top));
                sum += p;
                w[i] = times_half(p, cur.vs[i >> 3], i & 7);
            }
        }
        l += sum;
        __builtin_amdgcn_s_setprio(1);
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            float we[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) we[i] = w[8 * e + i];
            u4 wf, wl;
            if constexpr (SP) f16_split8(we, wf, wl);
            else wf = f16_pack8(we);
#pragma unroll
            for (int x = 0; x < ND; ++x) {
                const u4 vf = levels8(cur.v[e][x]);
                if constexpr (SP) acc[x] = mma32(vf, wl, acc[x]);
                acc[x] = mma32(vf, wf, acc[x]);
            }
        }
    };
    for (int step = sh.begin; step < sh.end;) {
#pragma unroll
        for (int k = 0; k < NB; ++k) {
            constexpr int ahead = NB - 1;
            const int in = (k + ahead) % NB;
            load_step<D>(ring[in], c, pages.token(page[in], step + ahead * TG), g, col);
            const int now = page[k];
            page[k] = pages.id(step + NB * TG);
            if (now >= 0 && now < c.pages) work(ring[k], step);
            step += TG;
            if (step >= sh.end) break;
        }
    }

    // lane (g, c): tile x's row 8 q + 4 g + i is dim D / 32 * row + x; four dims in a row from (q, i)
    l += __shfl_xor(l, 32);
    const Output<DT, D, TREE> out{a, pl, pc, part_o, part_ml, sh.first_row, sh.tile0, cols, h, G};
    if (g == 0) {
        lds_ml[tg][col][0] = m;
        lds_ml[tg][col][1] = l;
    }
    __syncthreads();
    float top = kLowest;
#pragma unroll
    for (int k = 0; k < TG; ++k) top = fmaxf(top, lds_ml[k][col][0]);
    const float mine = __builtin_amdgcn_exp2f(m - top);
#pragma unroll
    for (int q = 0; q < 4; ++q)
#pragma unroll
        for (int i = 0; i < 4; i += 128 / D)
            *reinterpret_cast<f4 *>(&lds_o[tg][col][D / 32 * (8 * q + 4 * g + i)]) = wide_dims<D>(acc, 4 * q + i) * mine;
    __syncthreads();
    join_groups<TG, TM, D>(out, lds_o, lds_ml, min(TM, sh.pairs - sh.tile0));
}

// The parts' sums of a tile and KV head become its outputs, `wide` columns (of `cols`) a
// workgroup: D / 4 threads take a part of a column, the rest of the 512 other columns and
// parts, each with a running maximum of its own; LDS joins the parts.
template <int DT, int D, bool TREE>
__global__ __launch_bounds__(512) void attn_join_kernel(Kv4Cache c, KvBatch b, Kv4Attn a, Plan pl, int cols, int wide,
                                                        const float *__restrict__ part_o,
                                                        const float *__restrict__ part_ml) {
    constexpr int L = D / 4, N = 512 / L;
    __shared__ f4 lds_o[N][L];
    __shared__ float lds_ml[N][2];
    const int h = blockIdx.y, G = a.q_heads / c.heads;
    const Piece pc = find_piece<true, false, TREE>(b, a, pl, c.heads, G, blockIdx.x);
    if (pc.parts == 0) return;
    const SeqWork sw = seq_work<TREE>(b, a, pc.seq);
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
        if (!TREE && a.stats && ln == 0) a.stats[at / D] = make_float2(top, inv);
    }
}

// The bounds of a plan (see above) for tiles of tm pairs.
Plan make_plan(const KvBatch &b, int heads, int G, int tm, int target, int min_chunk) {
    const int64_t steps = ((static_cast<int64_t>(b.max_pages) << b.page_shift) + 31) >> 5;
    const int64_t rows = static_cast<int64_t>(b.max_q) * G <= tm ? b.B : static_cast<int64_t>(b.rows) * G / tm + b.B;
    // Each tile may add a part to the even share: where tiles are few, the parts still fit one
    // round of workgroups; where they are many, twice as many parts even the rounds out.
    const int64_t tiles = rows * heads;
    // Contexts that fit few steps a wave are not cut, the longer the more tiles there are: a second
    // launch costs more than it saves (f32, 40 query and 8 KV heads: one sequence of 997 tokens 9.5
    // against 10.3 us, but 14.2 against 10.7 us for 1990; 8 of 1990 14.0 against 15.6 us; 8 of 3900
    // 20.5 against 17.4 us; 64 of 3900 34.6 against 42.9 us).
    const int64_t whole = kWaves * (tiles < 64 ? 8 : tiles < 256 ? 16 : 32);
    target = 2 * tiles <= target ? target - static_cast<int>(tiles) : 2 * target;
    Plan p{tm, target, min_chunk, 0, 0, 0, 0, 0};
    p.split = b.B <= kMostScanned && steps > whole;
    const int64_t even = (target + heads - 1) / heads, cuts = (steps + min_chunk - 1) / min_chunk;
    const int64_t extra = p.split ? (even < rows * cuts ? even : rows * cuts) : 0;
    p.pieces = static_cast<int>(rows + extra);
    p.items = static_cast<int>(extra < rows ? extra : rows);
    p.slots = static_cast<int>(2 * extra < rows + extra ? 2 * extra : rows + extra);
    return p;
}

// The kernel's shape for a call: by the pairs of one sequence and KV head, so that no wave
// multiplies mostly padding (more than 16 pairs in tiles of 32: an 8192-token prompt 861 us,
// 874 us in tiles of 16, which keep twice the conversions a product).  Heads of 256 fill the
// registers with 16 columns a wave.  One tile a workgroup, its waves sharing the context, beat
// two or four tiles side by side (8 x 16 rows 41 -> 37 us, a 4096-token window 199 -> 182 us;
// with 80 pairs a fourth wave had none) though an 8192-token prompt takes 3% less with two.
struct Shape {
    bool once;              // a sequence and KV head is one tile
    Plan plan;
    int cols;               // columns kept for a part
    int64_t sums, stats;    // bytes of the parts' sums and of their statistics
};
Shape attn_shape(const KvBatch &b, const Kv4Cache &c, int q_heads) {
    Shape s;
    const int G = q_heads / c.heads;
    const int64_t pairs = static_cast<int64_t>(b.max_q) * G;
    s.once = pairs <= 16;
    const int tm = s.once || c.D == 256 ? 16 : 32;
    // workgroups that the chip's 256 CUs hold at once; cutting finer costs more in the join (199999
    // tokens 50 us at 3 a CU, 60 at 6, 68 at 9)
    const int held = !s.once || c.D == 256 ? 2 : c.D == 128 ? 3 : 5;
    s.plan = make_plan(b, c.heads, G, tm, 256 * held, kWaves);
    if (!s.once) {
        const int each = 8 >> common8(c.heads), per = (s.plan.pieces + each - 1) / each;
        if (static_cast<int64_t>(per) * 8 * 64 * kWaves < int64_t(1) << 32) s.plan.per = per;
    }
    s.cols = static_cast<int>(pairs < tm ? pairs : tm);
    s.sums = static_cast<int64_t>(c.heads) * s.plan.slots * s.cols * c.D * 4;
    s.stats = static_cast<int64_t>(c.heads) * s.plan.slots * s.cols * 8;
    return s;
}

template <int DT, int D, bool TREE>
hipError_t launch_d(const Kv4Cache &c, const KvBatch &b, const Kv4Attn &a, void *workspace, hipStream_t st) {
    const Shape s = attn_shape(b, c, a.q_heads);
    float *part_o = static_cast<float *>(workspace), *part_ml = part_o + s.sums / 4;
    const dim3 grid = s.plan.per ? dim3(8 * s.plan.per, c.heads >> common8(c.heads)) : dim3(s.plan.pieces, c.heads), block(64 * kWaves);
    auto go = [&](auto kernel) { hipLaunchKernelGGL(kernel, grid, block, 0, st, c, b, a, s.plan, s.cols, part_o, part_ml); };
    constexpr int HL = DT == kDtF32 ? 2 : 0;
    if (s.once) {
        if (DT == kDtF32 && s.cols <= 8) go(attn_kernel<DT, D, DT == kDtF32 ? 1 : 0, true, TREE>);
        else go(attn_kernel<DT, D, HL, true, TREE>);
    } else {
        if constexpr (D == 256) go(attn_kernel<DT, D, HL, false, TREE>);
        else go(attn_wide_kernel<DT, D, DT == kDtF32, TREE>);
    }
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || s.plan.items == 0) return e;
    // columns a workgroup: few where there are few tiles, so that many parts are read side
    // by side, up to what its threads hold
    const int64_t most = s.cols < 2048 / D ? s.cols : 2048 / D, even = static_cast<int64_t>(s.plan.items) * c.heads * s.cols / 512;
    const int wide = static_cast<int>(even < 1 ? 1 : even < most ? even : most);
    hipLaunchKernelGGL((attn_join_kernel<DT, D, TREE>), dim3(s.plan.items, c.heads, (s.cols + wide - 1) / wide), dim3(512), 0, st,
                       c, b, a, s.plan, s.cols, wide, part_o, part_ml);
    return hipGetLastError();
}

template <int DT, bool TREE>
hipError_t launch_t(const Kv4Cache &c, const KvBatch &b, const Kv4Attn &a, void *workspace, hipStream_t st) {
    if (c.D == 64) return launch_d<DT, 64, TREE>(c, b, a, workspace, st);
    if (c.D == 128) return launch_d<DT, 128, TREE>(c, b, a, workspace, st);
    return launch_d<DT, 256, TREE>(c, b, a, workspace, st);
}
template <bool TREE>
hipError_t launch_attn(const Kv4Cache &c, const KvBatch &b, const Kv4Attn &a, void *workspace, int dtype, hipStream_t st) {
    if (dtype == kDtF32) return launch_t<kDtF32, TREE>(c, b, a, workspace, st);
    if (dtype == kDtBf16) return launch_t<kDtBf16, TREE>(c, b, a, workspace, st);
    return launch_t<kDtF16, TREE>(c, b, a, workspace, st);
}

}  // namespace
}  // namespace rad
