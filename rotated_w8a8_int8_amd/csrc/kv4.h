// kv4.h -- the paged 4-bit cache as the kernels see it (layouts and limits in
// include/rad.h), its e2m1 codec, and the ragged batch's bookkeeping (gfx950).
#pragma once

#include "layer_launch.h"
#include "value_types.h"

namespace rad {

// level * 1.0 of the two codes in byte SEL of w, exact
typedef float f2v __attribute__((ext_vector_type(2)));
template <int SEL>
__device__ __forceinline__ f2v e2m1_pair(uint32_t w) {
    return __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, SEL);
}

// Eight quotients -> one dword of e2m1 codes, quotient i in nibble i: nearest
// level, ties to the even code (1/4 -> 0, 3/4 -> 1, 5/4 -> 1, 7/4 -> 2, 5/2 -> 2,
// 7/2 -> 4, 5 -> 4), beyond 6 -> 6, as v_cvt_scalef32_pk_fp4_f32 rounds; then the
// sign of a zero is dropped, so that every value has one code.
__device__ __forceinline__ uint32_t e2m1_pack8(const float (&r)[8]) {
    uint32_t w = 0;
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, r[0], r[1], 1.0f, 0);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, r[2], r[3], 1.0f, 1);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, r[4], r[5], 1.0f, 2);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, r[6], r[7], 1.0f, 3);
    const uint32_t some = (w | (w >> 1) | (w >> 2)) & 0x11111111u;
    return w & ~(0x88888888u & ~(some << 3));
}

// f32 -> f16 bits, nearest even, subnormals kept, saturating at 65504.
__device__ __forceinline__ uint32_t kv4_scale_bits(float s) { return s < 65520.0f ? f16_round(s) : 0x7BFFu; }

// ---- the batch ------------------------------------------------------------
// Tokens of sequence b, as the calls read seq_len.
__device__ __forceinline__ int kv_len(const KvBatch &b, int seq) {
    const int cap = b.max_pages << b.page_shift;
    const int n = b.seq_len[seq];
    return n < 0 ? 0 : (n > cap ? cap : n);
}

// First row and number of rows of a sequence, made to lie inside 0 .. rows
// whatever q_start holds.
struct RowRange {
    int first, n;
};
__device__ __forceinline__ RowRange kv_rows(const KvBatch &b, int seq) {
    if (!b.q_start) return RowRange{seq, 1};
    int lo = b.q_start[seq], hi = b.q_start[seq + 1];
    if (lo < 0 || hi > b.rows || hi <= lo) return RowRange{0, 0};
    return RowRange{lo, hi - lo};
}

// The sequence whose rows hold `row`, or -1 (padding).
__device__ __forceinline__ int kv_seq_of(const KvBatch &b, int row) {
    if (!b.q_start) return row;
    int lo = 0, hi = b.B;                       // the last b with q_start[b] <= row lies in [lo, hi)
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (b.q_start[mid] <= row) lo = mid;
        else hi = mid;
    }
    const RowRange r = kv_rows(b, lo);
    return row >= r.first && row < r.first + r.n ? lo : -1;
}

// A row's sequence with its rows and tokens, for a row that a whole wave (all lanes on)
// asks about: up to 64 sequences are looked at by a lane each, in one trip to memory.
struct SeqOfRow {
    int seq, len;
    RowRange rr;
};
__device__ __forceinline__ SeqOfRow kv_seq_of_wave(const KvBatch &b, int row) {
    SeqOfRow s{-1, 0, RowRange{0, 0}};
    if (b.q_start && b.B <= 64) {
        const int i = min(static_cast<int>(threadIdx.x & 63), b.B - 1);
        const int lo = b.q_start[i], hi = b.q_start[i + 1], len = kv_len(b, i);
        const uint64_t hit = __ballot(row >= lo && row < hi);
        if (hit == 0) return s;
        const int src = __builtin_ctzll(hit);
        s.rr.first = __builtin_amdgcn_readlane(lo, src);
        s.rr.n = __builtin_amdgcn_readlane(hi, src) - s.rr.first;
        if (s.rr.first < 0 || s.rr.first + s.rr.n > b.rows) return s;
        s.seq = src;
        s.len = __builtin_amdgcn_readlane(len, src);
        return s;
    }
    s.seq = kv_seq_of(b, row);
    if (s.seq < 0) return s;
    s.rr = kv_rows(b, s.seq);
    s.len = kv_len(b, s.seq);
    return s;
}

// The page that holds token t of sequence seq, or -1 (absent).  0 <= t < kv_len.
__device__ __forceinline__ int kv_page(const KvBatch &b, int seq, int t, int pages) {
    const int id = b.block_table[static_cast<int64_t>(seq) * b.max_pages + (t >> b.page_shift)];
    return id >= 0 && id < pages ? id : -1;
}

}  // namespace rad
