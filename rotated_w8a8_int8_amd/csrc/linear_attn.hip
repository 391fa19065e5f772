// linear_attn.hip -- linear attention with a decay for each head (gfx950).
//
//   S = exp(g) S + k v^T,  o = scale S^T q, row by row; S [D][D] in f32.
//
// Row by row (single tokens): a workgroup holds 64 of a head's D value columns, D / 16
// of the key's rows a thread, four columns each, and passes over its part of the state once:
// 64 bf16 tokens of 40 heads of 128 stream 338 MB in 56 to 62 us, 5.4 to 6.0 TB/s.
//
// Prompts in chunks of 32 rows: 8192 bf16 rows of 40 heads of 128 take 117 us for the outputs,
// 58 us for what the segments add and 11 us for their states (profiled; 169 us a call), 625 MB in all, 3.7 TB/s of a
// call, with 52% of the cycles of a SIMD of a busy CU on vector and 33% on matrix instructions while outputs are made; f16
// 185 us a call, f32 420 us (its matrix operations 260).
#include <type_traits>

#include "layer_launch.h"
#include "value_types.h"

namespace rad {
namespace {

// First row and number of rows of a sequence, inside 0 .. rows whatever q_start holds.
struct Rows {
    int first, n;
};
__device__ __forceinline__ Rows linear_rows(const Linear &l, int seq) {
    if (!l.q_start) return Rows{seq, 1};
    const int lo = l.q_start[seq], hi = l.q_start[seq + 1];
    if (lo < 0 || hi > l.rows || hi <= lo) return Rows{0, 0};
    return Rows{lo, min(hi - lo, l.max_q)};
}

constexpr int kSlice = 64;        // value columns a workgroup

// blockIdx.x: sequence, blockIdx.y: head * (D / kSlice) + slice.  Thread: columns 4 (tid % 16) ..,
// key rows R (tid / 16) ..
template <int DT, int D>
__global__ __launch_bounds__(256) void recurrent_kernel(Linear l) {
    constexpr int R = D / 16, NS = D / kSlice;
    __shared__ float4 sums[2][4][16];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int seq = blockIdx.x, h = blockIdx.y / NS, c0 = kSlice * (blockIdx.y % NS) + 4 * (tid & 15), r0 = R * (tid >> 4);
    const int hk = h / (l.heads / l.qk_heads);
    const Rows rows = linear_rows(l, seq);
    const int64_t at = ((static_cast<int64_t>(seq) * l.heads + h) * D + r0) * D + c0;
    if (rows.n == 0 && (!l.state_out || l.state == l.state_out)) return;
    float4 s[R];
#pragma unroll
    for (int i = 0; i < R; ++i)
        s[i] = l.state ? load4<kDtF32, true>(l.state, at + static_cast<int64_t>(i) * D) : make_float4(0.f, 0.f, 0.f, 0.f);
    const float decay = expf(l.log_decay[h]);
    for (int t = 0; t < rows.n; ++t) {
        const int64_t row = rows.first + t;
        const float4 v = load4<DT>(l.v, row * l.ldv + static_cast<int64_t>(h) * D + c0);
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int j = 0; j < R / 4; ++j) {
            const float4 k4 = load4<DT>(l.k, row * l.ldk + static_cast<int64_t>(hk) * D + r0 + 4 * j);
            const float4 q4 = load4<DT>(l.q, row * l.ldq + static_cast<int64_t>(hk) * D + r0 + 4 * j);
            const float k[4] = {k4.x, k4.y, k4.z, k4.w}, q[4] = {q4.x, q4.y, q4.z, q4.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                float4 &x = s[4 * j + i];
                x.x = fmaf(x.x, decay, k[i] * v.x);
                x.y = fmaf(x.y, decay, k[i] * v.y);
                x.z = fmaf(x.z, decay, k[i] * v.z);
                x.w = fmaf(x.w, decay, k[i] * v.w);
                o.x = fmaf(x.x, q[i], o.x);
                o.y = fmaf(x.y, q[i], o.y);
                o.z = fmaf(x.z, q[i], o.z);
                o.w = fmaf(x.w, q[i], o.w);
            }
        }
        auto both = [](float x) {
            x += __shfl_xor(x, 16);
            return x + __shfl_xor(x, 32);
        };
        o = make_float4(both(o.x), both(o.y), both(o.z), both(o.w));
        if (lane < 16) sums[t & 1][wave][lane] = o;
        __syncthreads();
        if (tid < 16) {
            const float4 a = sums[t & 1][0][tid], b = sums[t & 1][1][tid], c = sums[t & 1][2][tid], d = sums[t & 1][3][tid];
            auto sum = [&](float x, float y, float z, float w) { return ((x + y) + (z + w)) * l.scale; };
            store4<DT>(l.o, (row * l.heads + h) * D + c0,
                       make_float4(sum(a.x, b.x, c.x, d.x), sum(a.y, b.y, c.y, d.y), sum(a.z, b.z, c.z, d.z), sum(a.w, b.w, c.w, d.w)));
        }
    }
    if (l.state_out)
#pragma unroll
        for (int i = 0; i < R; ++i) store4<kDtF32, true>(l.state_out, at + static_cast<int64_t>(i) * D, s[i]);
}

// ---- chunks of 32 rows ---------------------------------------------------------
//
// With a = exp(g), S the state before a chunk and i, j its rows from 0:
//
//   O = (Q K^T . a^(i - j) [j <= i]) V + a^(i + 1) Q S,   S' = a^n S + K^T (a^(n - 1 - j) V)
//
// A wave holds 32 of the head's value columns of the state, [D][32] in accumulators, and
// does all four products for them, transposed so that what one product leaves is what the
// next takes, lane by lane:
//
//   P^T [32 j][32 i] = K Q^T           a lane comes out with 16 rows j of one column i,
//   O^T [32 v][32 i] = V^T P^T         which are the second operand's rows here
//                    + S^T Q^T         and a lane's dims of one column v the first operand's
//   S [D][32 v]     += K^T (a.. V)     V as read for O^T, aged
//
// Rows r = 8 q + 4 g + e of a tile (q = 0 .. 3, g = lane / 32, e = 0 .. 3) are held by lane half
// g.  Value column r of the wave is v = 16 g + 4 q + e, so that a lane stores 16
// consecutive values of a row.
//
// A sequence is cut into segments of `each` rows, a workgroup each: where it has several, a first
// kernel works out what each adds to the state, a second hands the states on, and the last
// one begins each segment with its state.  Sequence b's segments have the places from
// q_start[b] / each + b on, which leaves room for max(1, ceil(n / each)) of them, so that places
// need no other sequence's length (empty sequences at the end have the last places).
typedef float f16v __attribute__((ext_vector_type(16)));
typedef __bf16 b8 __attribute__((ext_vector_type(8)));
typedef _Float16 h8 __attribute__((ext_vector_type(8)));
typedef unsigned int u4 __attribute__((ext_vector_type(4)));
typedef unsigned int u2 __attribute__((ext_vector_type(2)));
typedef unsigned short us2 __attribute__((ext_vector_type(2)));

constexpr int kChunk = 32;
constexpr float kLog2e = 1.44269504088896340736f;
template <int D>
constexpr int kLinWaves = D >= 128 ? 4 : 2;              // of 32 value columns
template <int D>
constexpr int kSlices = D / (32 * kLinWaves<D>);         // workgroups a head

struct Segments {
    int each, places;         // rows a segment, a multiple of kChunk; places a head
    float *states;            // [places][heads][D][D]: state before each segment of a sequence of several
};
__device__ __forceinline__ int first_place(const Linear &l, const Segments &sg, int seq) {
    return min((l.q_start ? l.q_start[seq] : seq) / sg.each, sg.places - l.B) + seq;
}

// What a workgroup takes: all rows are whole chunks but the sequence's last.
struct SegRows {
    int seq, first, n;        // the sequence; the call's rows
    int segs;                 // the sequence's segments; 0: nothing lies in this place
    bool last;
};
// Segment seg of a sequence.
__device__ __forceinline__ SegRows segment_rows(const Linear &l, const Segments &sg, int seq, int seg) {
    const Rows r = linear_rows(l, seq);
    const int segs = max(1, (r.n + sg.each - 1) / sg.each), lo = min(seg * sg.each, r.n);
    return SegRows{seq, r.first + lo, min(sg.each, r.n - lo), seg < segs ? segs : 0, seg == segs - 1};
}
// The segment in a place: its sequence is the last one whose first place is not past it; 64 are looked at a trip.
// Every lane of the wave calls it and gets the same answer.
__device__ __forceinline__ SegRows segment_in(const Linear &l, const Segments &sg, int place) {
    int seq = 0;
    for (int n = l.B; n > 1;) {                               // it lies in [seq, seq + n)
        const int each = (n + 63) >> 6, i = (threadIdx.x & 63) * each;
        const int at = max(__popcll(__ballot(i < n && first_place(l, sg, seq + min(i, n - 1)) <= place)) - 1, 0) * each;
        seq += at;
        n = min(each, n - at);
    }
    seq = __builtin_amdgcn_readfirstlane(seq);
    const int seg = place - first_place(l, sg, seq);
    return seg >= 0 ? segment_rows(l, sg, seq, seg) : SegRows{seq, 0, 0, 0, false};
}

// What a workgroup is about.  Workgroups go to the eight XCDs in turn: those that read the same queries and keys
// (slices of a head, heads that share a key head) follow each other on one, where its L2 serves them
// (8192 bf16 rows of 16 heads of 256: 292 us, 435 us spread over the XCDs, when this was chosen).
struct Item {
    int place, hk, h, slice;
};
__device__ __forceinline__ Item item_of(const Linear &l, const Segments &sg, int slices) {
    const int each = l.heads / l.qk_heads, sub = each * slices, x = blockIdx.x;
    const int u = x / (8 * sub) * 8 + (x & 7), j = (x >> 3) % sub, hk = u / sg.places;
    return Item{u % sg.places, hk, hk * each + j / slices, j % slices};
}
int64_t items(const Linear &l, const Segments &sg, int slices) {
    return (static_cast<int64_t>(sg.places) * l.qk_heads + 7) / 8 * 8 * (l.heads / l.qk_heads) * slices;
}

// a^k, a = 2^l2
__device__ __forceinline__ float power(float l2, int k) { return __builtin_amdgcn_exp2f(l2 * static_cast<float>(k)); }
__device__ __forceinline__ float log2_decay(const Linear &l, int h) { return fmaxf(l.log_decay[h] * kLog2e, -1e30f); }

// State columns of a wave: lane r = lane % 32 holds column v(r), rows 32 T + 8 q + 4 g + e in s[T][4 q + e].
__device__ __forceinline__ int value_of(int r) { return 16 * ((r >> 2) & 1) + 4 * (r >> 3) + (r & 3); }
template <int D>
__device__ __forceinline__ void load_state(f16v (&s)[D / 32], const float *from, int g, int col) {
#pragma unroll
    for (int T = 0; T < D / 32; ++T)
#pragma unroll
        for (int i = 0; i < 16; ++i) s[T][i] = from ? from[static_cast<int64_t>(32 * T + 8 * (i >> 2) + 4 * g + (i & 3)) * D + col] : 0.0f;
}
template <int D>
__device__ __forceinline__ void store_state(const f16v (&s)[D / 32], float *to, int g, int col) {
#pragma unroll
    for (int T = 0; T < D / 32; ++T)
#pragma unroll
        for (int i = 0; i < 16; ++i) to[static_cast<int64_t>(32 * T + 8 * (i >> 2) + 4 * g + (i & 3)) * D + col] = s[T][i];
}

// A lane's i-th row of a chunk, j = 8 q + 4 g + e.
__device__ __forceinline__ int row_of(int i, int g) { return 8 * (i >> 2) + 4 * g + (i & 3); }
// Ages of a chunk of n rows, as a lane meets its rows.
struct Ages {
    float w[16], all;         // a^(n - 1 - j), 0 from row n on; a^n
    __device__ __forceinline__ void set(float l2, int n, int g) {
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const int j = row_of(i, g);
            w[i] = j < n ? power(l2, n - 1 - j) : 0.0f;
        }
        all = power(l2, n);
    }
};

// A value v_j that is not finite reaches rows i >= j of its column, and the state's column; a product with the 0 that hides it
// from rows before would bring it there.  A chunk that holds one works with 0 in its place, and makes those outputs and the
// state's column NaN: from_row is the first such row of each of a wave's columns.
__device__ __forceinline__ void hide_lost(f16v &o, const int *from_row, int g, int col) {
#pragma unroll
    for (int i = 0; i < 16; ++i) o[i] = col >= from_row[row_of(i, g)] ? NAN : o[i];
}
__device__ __forceinline__ bool keep_lost(int *from_row, int first, int g, int col) {
    first = min(first, __shfl_xor(first, 32));
    if (g == 0) from_row[col] = first;
    __builtin_amdgcn_wave_barrier();
    return first < kChunk;
}

// ---- f32 products -----------------------------------------------------------------
//
// 32x32x2 matrix operations (154 TFLOP/s where the 16-bit ones reach 1228): 160 of them a wave and chunk
// for D = 128.  They read two values a lane and take 64 cycles, so that tiles lie in LDS as they come, f32.
template <int D>
struct TileF32 {
    float q[kChunk][D + 4], k[kChunk][D + 4], v[kChunk][32 * kLinWaves<D> + 4];
    f16v p[kLinWaves<D>][64];                             // shares of P^T, by dims of the products
    int lost, from_row[kLinWaves<D>][32];                 // the last chunk with a value that is not finite; see hide_lost
};

template <int DT, int D, bool OUT>
__global__ __launch_bounds__(64 * kLinWaves<D>, D == 256 ? 1 : 2) void chunk_f32_kernel(Linear l, Segments sg) {
    constexpr int NW = kLinWaves<D>, NT = 64 * NW, VC = 32 * NW, NS = kSlices<D>, PQ = D / (NT / 2);
    __shared__ TileF32<D> tile;
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int g = lane >> 5, col = lane & 31;
    const Item it = item_of(l, sg, NS);
    if (it.hk >= l.qk_heads) return;
    const int h = it.h, v0 = VC * it.slice, hk = it.hk;
    const SegRows sr = segment_in(l, sg, it.place);
    const int64_t pair = static_cast<int64_t>(sr.seq) * l.heads + h, mat = static_cast<int64_t>(D) * D;
    float *const kept = sg.states + (static_cast<int64_t>(it.place) * l.heads + h) * mat;
    const int vcol = v0 + 32 * wave + value_of(col);
    if (sr.segs == 0 || (!OUT && sr.last)) return;
    if (OUT && sr.n == 0 && (!l.state_out || l.state == l.state_out)) return;

    f16v s[D / 32];
    load_state<D>(s, OUT ? (sr.segs > 1 ? kept : l.state ? l.state + pair * mat : nullptr) : nullptr, g, vcol);
    const float l2 = log2_decay(l, h), from = power(l2, col + 1);
    auto sees = [&](int i) { return row_of(i, g) <= col; };
    float near[16];                                       // a^(i - j) of the lane's column i = col
    Ages age;
    age.set(l2, kChunk, g);
    if (OUT)
#pragma unroll
        for (int i = 0; i < 16; ++i) near[i] = sees(i) ? power(l2, col - row_of(i, g)) : 0.0f;

    const int br = 4 * (tid & 7), bc = 4 * (tid >> 3);
    float4 bq[PQ][4], bk[PQ][4], bv[4];
    auto fetch = [&](int c0) {
#pragma unroll
        for (int x = 0; x < 4; ++x) {
            const bool on = c0 + br + x < sr.n;
            const int64_t row = sr.first + c0 + br + x;
            const float4 none = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int y = 0; y < PQ; ++y) {
                const int d = bc + (NT / 2) * y;
                bk[y][x] = on ? load4<DT>(l.k, row * l.ldk + static_cast<int64_t>(hk) * D + d) : none;
                if (OUT) bq[y][x] = on ? load4<DT>(l.q, row * l.ldq + static_cast<int64_t>(hk) * D + d) : none;
            }
            bv[x] = on ? load4<DT>(l.v, row * l.ldv + static_cast<int64_t>(h) * D + v0 + bc) : none;
        }
    };
    // value column v of a wave lies at its r: 4 of them in a row stay together
    const int vr = 32 * (bc >> 5) + 8 * ((bc >> 2) & 3) + 4 * ((bc >> 4) & 1);
    auto put = [&](int c0) {
        float zero = 0.0f;                                // NaN where a value is not finite
#pragma unroll
        for (int x = 0; x < 4; ++x) {
            if (OUT) zero = fmaf(bv[x].x, 0.0f, fmaf(bv[x].y, 0.0f, fmaf(bv[x].z, 0.0f, fmaf(bv[x].w, 0.0f, zero))));
#pragma unroll
            for (int y = 0; y < PQ; ++y) {
                *reinterpret_cast<float4 *>(&tile.k[br + x][bc + (NT / 2) * y]) = bk[y][x];
                if (OUT) *reinterpret_cast<float4 *>(&tile.q[br + x][bc + (NT / 2) * y]) = bq[y][x];
            }
            *reinterpret_cast<float4 *>(&tile.v[br + x][vr]) = bv[x];
        }
        if (OUT && zero != 0.0f) tile.lost = c0;
    };
    if (OUT && tid == 0) tile.lost = -1;
    fetch(0);
    for (int c0 = 0; c0 < sr.n; c0 += kChunk) {
        const int n = min(kChunk, sr.n - c0);
        __syncthreads();                                  // the tile before is read
        put(c0);
        __syncthreads();
        if (c0 + kChunk < sr.n) fetch(c0 + kChunk);
        if (n < kChunk) age.set(l2, n, g);
        bool lost = false;                                // the lane's column has a value that is not finite
        if (OUT) {
            if (tile.lost == c0) {                        // rare; the wave's columns are its own
                int first = kChunk;
#pragma unroll 1
                for (int i = 15; i >= 0; --i) {
                    float &v = tile.v[row_of(i, g)][32 * wave + col];
                    if (!(fabsf(v) < INFINITY)) v = 0.0f, first = row_of(i, g);
                }
                lost = keep_lost(tile.from_row[wave], first, g, col);
            }
            // P^T: each wave sums over its share of the dims, all of them add the shares up
            f16v p{};
#pragma unroll
            for (int m = 0; m < D / NW / 8; ++m) {
                const int d = D / NW * wave + 8 * m + 4 * g;
                const float4 a = *reinterpret_cast<const float4 *>(&tile.k[col][d]), b = *reinterpret_cast<const float4 *>(&tile.q[col][d]);
                p = __builtin_amdgcn_mfma_f32_32x32x2f32(a.x, b.x, p, 0, 0, 0);
                p = __builtin_amdgcn_mfma_f32_32x32x2f32(a.y, b.y, p, 0, 0, 0);
                p = __builtin_amdgcn_mfma_f32_32x32x2f32(a.z, b.z, p, 0, 0, 0);
                p = __builtin_amdgcn_mfma_f32_32x32x2f32(a.w, b.w, p, 0, 0, 0);
            }
            tile.p[wave][lane] = p;
            // S^T Q^T meanwhile
            f16v o{};
#pragma unroll
            for (int T = 0; T < D / 32; ++T)
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const float4 b = *reinterpret_cast<const float4 *>(&tile.q[col][32 * T + 8 * q + 4 * g]);
                    o = __builtin_amdgcn_mfma_f32_32x32x2f32(s[T][4 * q], b.x, o, 0, 0, 0);
                    o = __builtin_amdgcn_mfma_f32_32x32x2f32(s[T][4 * q + 1], b.y, o, 0, 0, 0);
                    o = __builtin_amdgcn_mfma_f32_32x32x2f32(s[T][4 * q + 2], b.z, o, 0, 0, 0);
                    o = __builtin_amdgcn_mfma_f32_32x32x2f32(s[T][4 * q + 3], b.w, o, 0, 0, 0);
                }
            __syncthreads();
            p = tile.p[0][lane];
#pragma unroll
            for (int x = 1; x < NW; ++x) p += tile.p[x][lane];
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                p[i] = sees(i) ? p[i] * near[i] : 0.0f;       // a product with a later row's key may be anything
                o[i] *= from;
            }
#pragma unroll
            for (int i = 0; i < 16; ++i)
                o = __builtin_amdgcn_mfma_f32_32x32x2f32(tile.v[8 * (i >> 2) + 4 * g + (i & 3)][32 * wave + col], p[i], o, 0, 0, 0);
            if (tile.lost == c0) hide_lost(o, tile.from_row[wave], g, col);
            if (col < n) {
                const int64_t at = (static_cast<int64_t>(sr.first + c0 + col) * l.heads + h) * D + v0 + 32 * wave + 16 * g;
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    store4<DT>(l.o, at + 4 * q, make_float4(o[4 * q] * l.scale, o[4 * q + 1] * l.scale, o[4 * q + 2] * l.scale, o[4 * q + 3] * l.scale));
            }
        }
#pragma unroll
        for (int T = 0; T < D / 32; ++T) s[T] *= age.all;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const int j = 8 * (i >> 2) + 4 * g + (i & 3);
            const float b = i == 0 && lost ? NAN : tile.v[j][32 * wave + col] * age.w[i];
#pragma unroll
            for (int T = 0; T < D / 32; ++T) s[T] = __builtin_amdgcn_mfma_f32_32x32x2f32(tile.k[j][32 * T + col], b, s[T], 0, 0, 0);
        }
    }
    if (!OUT) store_state<D>(s, kept, g, vcol);
    else if (l.state_out && sr.last) store_state<D>(s, l.state_out + pair * mat, g, vcol);
}

// ---- 16-bit products ---------------------------------------------------------------
//
// 32x32x16 matrix operations, 8 values a lane.  Rows (and dims) of a step of 16 are taken in the order
// 16 m + 8 b + 4 g + e -> 16 m + 8 g + 4 b + e that accumulators have, so that a lane's values lie together;
// K and V are transposed on their way into LDS, 4 x 4 values a thread.  q, k and v are exact.  P and
// S are taken as two 16-bit parts (bf16 16 bits, f16 22), aged values as as many as make the
// state good to 2^-22 or better (bf16 three, f16 two).  f16 parts are taken at the power of two that puts the
// largest of their column of the state, or of their row's weights, in [2^14, 2^15): what is 2^-17 of that keeps 22
// bits.  One power for a wave's 32 columns left columns 2^-26 of another's a few bits.
template <int DT>
__device__ __forceinline__ f16v mma(u4 a, u4 b, f16v c) {
    if constexpr (DT == kDtBf16) return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(b8, a), __builtin_bit_cast(b8, b), c, 0, 0, 0);
    else return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(h8, a), __builtin_bit_cast(h8, b), c, 0, 0, 0);
}
// Two values to the type, in a word.
template <int DT>
__device__ __forceinline__ uint32_t pack16(float a, float b) {
    typedef float f2 __attribute__((ext_vector_type(2)));
    if constexpr (DT == kDtBf16) {
        typedef __bf16 b2 __attribute__((ext_vector_type(2)));
        return __builtin_bit_cast(uint32_t, __builtin_convertvector(f2{a, b}, b2));
    } else {
        typedef _Float16 h2 __attribute__((ext_vector_type(2)));
        return __builtin_bit_cast(uint32_t, h2{static_cast<_Float16>(a), static_cast<_Float16>(b)});
    }
}
// Eight values to the type; what that leaves of them.
template <int DT>
__device__ __forceinline__ u4 part8(float (&x)[8]) {
    u4 r;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        r[i] = pack16<DT>(x[2 * i], x[2 * i + 1]);
        x[2 * i] -= widen16<DT>(r[i] & 0xFFFFu);
        x[2 * i + 1] -= widen16<DT>(r[i] >> 16);
    }
    return r;
}
// The larger of what the two lanes of a column hold.
__device__ __forceinline__ float both_max(float m) { return fmaxf(m, __shfl_xor(m, 32)); }
// Exponent that takes m, the largest magnitude of a column, to [2^14, 2^15), at most `most` (what meets the products
// in f32 is taken along and has to stay finite).
__device__ __forceinline__ int room(float m, int most) { return m > 0.0f ? min(15 - __builtin_amdgcn_frexp_expf(m), most) : 0; }
template <int N>
__device__ __forceinline__ float largest(const float (&x)[N]) {
    float m = 0.0f;
#pragma unroll
    for (int i = 0; i < N; ++i) m = fmaxf(m, fabsf(x[i]));
    return both_max(m);
}
template <int T>
__device__ __forceinline__ float largest(const f16v (&s)[T]) {
    float m = 0.0f;
#pragma unroll
    for (int t = 0; t < T; ++t)
#pragma unroll
        for (int i = 0; i < 16; ++i) m = fmaxf(m, fabsf(s[t][i]));
    return both_max(m);
}
constexpr float kLazy = 0x1p-8f;
__device__ __forceinline__ float pow2(int e) { return __builtin_amdgcn_ldexpf(1.0f, e); }

template <int D, bool OUT>
struct Tile16 {
    uint16_t q[OUT ? kChunk : 1][D + 8], k[OUT ? kChunk : 1][D + 8];      // [row][dim]
    uint16_t kt[D][kChunk + 8], vt[32 * kLinWaves<D>][kChunk + 8];        // [dim][row], [value column][row]
};
// Place of four values in a row of the order above.
__device__ __forceinline__ int place(int i) { return (i & ~15) + 8 * ((i >> 2) & 1) + 4 * ((i >> 3) & 1); }
// Four rows of four values -> four columns of four.
__device__ __forceinline__ void turn4(const u2 (&x)[4], u2 (&y)[4]) {
#pragma unroll
    for (int c = 0; c < 4; ++c) {
        const uint32_t sel = c & 1 ? 0x07060302u : 0x05040100u;
        y[c] = u2{__builtin_amdgcn_perm(x[1][c >> 1], x[0][c >> 1], sel), __builtin_amdgcn_perm(x[3][c >> 1], x[2][c >> 1], sel)};
    }
}

template <int DT, int D, bool OUT>
__global__ __launch_bounds__(64 * kLinWaves<D>, D == 256 ? 1 : 2) void chunk_kernel(Linear l, Segments sg) {
    constexpr int NW = kLinWaves<D>, NT = 64 * NW, VC = 32 * NW, NS = kSlices<D>, PQ = D / (NT / 2), NA = DT == kDtBf16 ? 3 : 2;
    constexpr bool kScaled = DT == kDtF16;                // bf16 has f32's range
    __shared__ Tile16<D, OUT> tiles[2];
    alignas(16) __shared__ float undo[kScaled && OUT ? NW : 1][32];   // of a wave's state columns, what their parts were scaled by
    __shared__ int from_row[OUT ? NW : 1][32];            // see hide_lost
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int g = lane >> 5, col = lane & 31;
    const Item it = item_of(l, sg, NS);
    if (it.hk >= l.qk_heads) return;
    const int h = it.h, v0 = VC * it.slice, hk = it.hk;
    const SegRows sr = segment_in(l, sg, it.place);
    const int64_t pair = static_cast<int64_t>(sr.seq) * l.heads + h, mat = static_cast<int64_t>(D) * D;
    float *const kept = sg.states + (static_cast<int64_t>(it.place) * l.heads + h) * mat;
    const int vcol = v0 + 32 * wave + value_of(col);
    if (sr.segs == 0 || (!OUT && sr.last)) return;
    if (OUT && sr.n == 0 && (!l.state_out || l.state == l.state_out)) return;

    const int br = 4 * (tid & 7), bc = 4 * (tid >> 3);
    u2 bq[PQ][4], bk[PQ][4], bv[4];
    // the thread's block of the next chunk: four values from column bc of rows br .. br + 3
    const int64_t row0 = sr.first + br;
    const uint16_t *pk = static_cast<const uint16_t *>(l.k) + row0 * l.ldk + hk * D + bc;
    const uint16_t *pq = static_cast<const uint16_t *>(l.q) + row0 * l.ldq + hk * D + bc;
    const uint16_t *pv = static_cast<const uint16_t *>(l.v) + row0 * l.ldv + h * D + v0 + bc;
    auto fetch = [&](int c0) {
        auto rows4 = [&](auto on) {
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                auto four = [&](const uint16_t *at) { return on(x) ? *reinterpret_cast<const u2 *>(at) : u2{0u, 0u}; };
#pragma unroll
                for (int y = 0; y < PQ; ++y) {
                    bk[y][x] = four(pk + x * l.ldk + (NT / 2) * y);
                    if (OUT) bq[y][x] = four(pq + x * l.ldq + (NT / 2) * y);
                }
                bv[x] = four(pv + x * l.ldv);
            }
        };
        rows4([&](int x) { return c0 + br + x < sr.n; });
        pk += kChunk * l.ldk;
        pq += kChunk * l.ldq;
        pv += kChunk * l.ldv;
    };
    const int vr = 32 * (bc >> 5) + 8 * ((bc >> 2) & 3) + 4 * ((bc >> 4) & 1), at_r = place(br);
    auto put = [&](Tile16<D, OUT> &t) {
        u2 y4[4];
#pragma unroll
        for (int y = 0; y < PQ; ++y) {
            const int d = bc + (NT / 2) * y;
            if (OUT)
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    *reinterpret_cast<u2 *>(&t.k[br + x][place(d)]) = bk[y][x];
                    *reinterpret_cast<u2 *>(&t.q[br + x][place(d)]) = bq[y][x];
                }
            turn4(bk[y], y4);
#pragma unroll
            for (int x = 0; x < 4; ++x) *reinterpret_cast<u2 *>(&t.kt[d + x][at_r]) = y4[x];
        }
        turn4(bv, y4);
#pragma unroll
        for (int x = 0; x < 4; ++x) *reinterpret_cast<u2 *>(&t.vt[vr + x][at_r]) = y4[x];
    };
    fetch(0);
    f16v s[D / 32];
    load_state<D>(s, OUT ? (sr.segs > 1 ? kept : l.state ? l.state + pair * mat : nullptr) : nullptr, g, vcol);
    const float l2 = log2_decay(l, h), from = power(l2, col + 1) * l.scale;
    auto sees = [&](int i) { return row_of(i, g) <= col; };
    float near[16];                                       // a^(i - j) of the lane's column i = col
    Ages age;
    age.set(l2, kChunk, g);
    if (OUT)
#pragma unroll
        for (int i = 0; i < 16; ++i) near[i] = sees(i) ? power(l2, col - row_of(i, g)) * l.scale : 0.0f;
    // The lane's column of the state is a^aged_by 2^-es s.  Where the products have f32's range (bf16) it ages by the
    // count of rows alone, and is multiplied out once that comes to kLazy.  f16 products add less than 2^54 to a state
    // (2^22 rows of 2^32 each), so that only one that begins past that may leave no room for its exponent.
    int es = 0, aged_by = 0, most_es = 32;
    if constexpr (kScaled) {
        const float big = largest(s);
        if (big > 0x1p60f) most_es = min(32, 126 - __builtin_amdgcn_frexp_expf(big));
    }
    put(tiles[0]);
    __syncthreads();
    for (int c0 = 0, at = 0; c0 < sr.n; c0 += kChunk, at ^= 1) {
        const Tile16<D, OUT> &t = tiles[at];
        const int n = min(kChunk, sr.n - c0);
        const bool more = c0 + kChunk < sr.n;
        if (more) fetch(c0 + kChunk);
        u4 vf[2];
        auto values = [&]() {
#pragma unroll
            for (int m = 0; m < 2; ++m) vf[m] = *reinterpret_cast<const u4 *>(&t.vt[32 * wave + col][16 * m + 8 * g]);
        };
        bool lost = false;                                // the lane's column has a value that is not finite
        if (OUT) {
            u4 qf[D / 16];
#pragma unroll
            for (int m = 0; m < D / 16; ++m) qf[m] = *reinterpret_cast<const u4 *>(&t.q[col][16 * m + 8 * g]);
            f16v p{};
#pragma unroll
            for (int m = 0; m < D / 16; ++m) p = mma<DT>(*reinterpret_cast<const u4 *>(&t.k[col][16 * m + 8 * g]), qf[m], p);
            float fs = 1.0f;
            if constexpr (kScaled) {
                const int ef = room(largest(s), 90);
                fs = pow2(ef);
                if (g == 0) undo[wave][col] = pow2(-ef - es);
                __builtin_amdgcn_wave_barrier();
            }
            f16v o{};
#pragma unroll
            for (int T = 0; T < D / 32; ++T)
#pragma unroll
                for (int m = 0; m < 2; ++m) {
                    float x[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i) x[i] = kScaled ? s[T][8 * m + i] * fs : s[T][8 * m + i];
                    const u4 hi = part8<DT>(x), lo = part8<DT>(x);
                    o = mma<DT>(lo, qf[2 * T + m], o);
                    o = mma<DT>(hi, qf[2 * T + m], o);
                }
            float pw[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) pw[i] = sees(i) ? p[i] * near[i] : 0.0f;       // a product with a later row's key may be anything
            const int ep = kScaled ? room(largest(pw), 64) : 0;
            const float fo = __builtin_amdgcn_ldexpf(from * power(l2, aged_by), ep), fp = pow2(ep);
            if constexpr (kScaled)                        // a product's row is a column of the state
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const float4 u = *reinterpret_cast<const float4 *>(&undo[wave][8 * q + 4 * g]);
                    o[4 * q] *= u.x, o[4 * q + 1] *= u.y, o[4 * q + 2] *= u.z, o[4 * q + 3] *= u.w;
                }
            __builtin_amdgcn_wave_barrier();
#pragma unroll
            for (int i = 0; i < 16; ++i) o[i] *= fo;
            values();
            constexpr uint32_t kExp = DT == kDtBf16 ? 0x7F80u : 0x7C00u;
            us2 most = __builtin_bit_cast(us2, vf[0][0] & 0x7FFF7FFFu);
#pragma unroll
            for (int i = 1; i < 8; ++i) most = __builtin_elementwise_max(most, __builtin_bit_cast(us2, vf[i >> 2][i & 3] & 0x7FFF7FFFu));
            const bool any_lost = __any(most.x >= kExp || most.y >= kExp);
            if (any_lost) {                               // rare
                int first = kChunk;                       // the wave's columns are its own
#pragma unroll 1
                for (int i = 15; i >= 0; --i) {
                    uint16_t &x = tiles[at].vt[32 * wave + col][16 * (i >> 3) + 8 * g + (i & 7)];
                    if ((x & kExp) == kExp) x = 0, first = row_of(i, g);
                }
                lost = keep_lost(from_row[wave], first, g, col);
                values();
            }
#pragma unroll
            for (int m = 0; m < 2; ++m) {
                float x[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) x[i] = kScaled ? pw[8 * m + i] * fp : pw[8 * m + i];
                const u4 hi = part8<DT>(x), lo = part8<DT>(x);
                o = mma<DT>(vf[m], lo, o);
                o = mma<DT>(vf[m], hi, o);
            }
            if (any_lost) hide_lost(o, from_row[wave], g, col);
            if (col < n) {
                const int64_t to = (static_cast<int64_t>(sr.first + c0 + col) * l.heads + h) * D + v0 + 32 * wave + 16 * g;
                u4 y[2];
                const float f = pow2(-ep);
#pragma unroll
                for (int i = 0; i < 8; ++i) y[i >> 2][i & 3] = kScaled ? pack16<DT>(o[2 * i] * f, o[2 * i + 1] * f) : pack16<DT>(o[2 * i], o[2 * i + 1]);
                u4 *q = reinterpret_cast<u4 *>(static_cast<uint16_t *>(l.o) + to);
                q[0] = y[0];
                q[1] = y[1];
            }
        }
        if (!OUT) values();
        if (n < kChunk) age.set(l2, n, g);
        float aged[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) aged[i] = widen16<DT>(i & 1 ? vf[i >> 3][(i & 7) >> 1] >> 16 : vf[i >> 3][(i & 7) >> 1] & 0xFFFFu) * age.w[i];
        if (lost) aged[0] = NAN;
        const int ea = kScaled ? room(largest(aged), most_es) : 0;
        aged_by += n;
        const float gone = power(l2, aged_by);
        if (kScaled || gone < kLazy) {
            const float keep = __builtin_amdgcn_ldexpf(gone, ea - es);
#pragma unroll
            for (int T = 0; T < D / 32; ++T) s[T] *= keep;
            aged_by = 0;
            es = ea;
        }
        const float fa = __builtin_amdgcn_ldexpf(power(-l2, aged_by), es);
#pragma unroll
        for (int m = 0; m < 2; ++m) {
            float x[8];
            u4 part[NA];
#pragma unroll
            for (int i = 0; i < 8; ++i) x[i] = aged[8 * m + i] * fa;
#pragma unroll
            for (int y = 0; y < NA; ++y) part[y] = part8<DT>(x);
#pragma unroll
            for (int T = 0; T < D / 32; ++T) {
                const u4 kf = *reinterpret_cast<const u4 *>(&t.kt[32 * T + col][16 * m + 8 * g]);
#pragma unroll
                for (int y = NA - 1; y >= 0; --y) s[T] = mma<DT>(kf, part[y], s[T]);
            }
        }
        if (more) put(tiles[at ^ 1]);
        __syncthreads();
    }
#pragma unroll
    for (int T = 0; T < D / 32; ++T) s[T] *= __builtin_amdgcn_ldexpf(power(l2, aged_by), -es);
    if (!OUT) store_state<D>(s, kept, g, vcol);
    else if (l.state_out && sr.last) store_state<D>(s, l.state_out + pair * mat, g, vcol);
}

// States before each segment, in place of what each adds: blockIdx.x: sequence * heads + head, blockIdx.y: 1024 values.
__global__ __launch_bounds__(256) void states_kernel(Linear l, Segments sg) {
    const int64_t pair = blockIdx.x;
    const int seq = static_cast<int>(pair / l.heads), h = static_cast<int>(pair % l.heads);
    const int segs = segment_rows(l, sg, seq, 0).segs;
    if (segs == 1) return;                                    // its state is read where it is
    const int64_t mat = static_cast<int64_t>(l.D) * l.D, next = mat * l.heads, at = blockIdx.y * 1024 + 4 * threadIdx.x;
    const float a = power(log2_decay(l, h), sg.each);         // the last segment's is of no use here
    float *w = sg.states + first_place(l, sg, seq) * next + h * mat + at;
    float4 s = l.state ? load4<kDtF32>(l.state, pair * mat + at) : make_float4(0.f, 0.f, 0.f, 0.f);
    for (int seg = 0; seg < segs; ++seg, w += next) {
        const float4 add = seg + 1 < segs ? load4<kDtF32>(w, 0) : s;
        store4<kDtF32>(w, 0, s);
        s = make_float4(fmaf(a, s.x, add.x), fmaf(a, s.y, add.y), fmaf(a, s.z, add.z), fmaf(a, s.w, add.w));
    }
}

// Rows a segment: so many that the segments fill the chip once (an 8192-row bf16 prompt of 40 heads takes 176 us
// with 12, 196 with 9, 207 with 19; 8 x 1000 rows 147 us whole, 207 us in halves, when this was chosen), 128 at least
// (600 rows 36 us, 53 with 256).  Places that stay empty count too: 288 workgroups of which 32 had nothing to do took
// 440 us where the 256 others take 296.
//
// Sequences within a tenth of the longest's length share the segments evenly; else these are sized by all rows (bf16, 40
// heads of 128: 8 x 1000 rows 148 us so, 312 by all rows; 4 of 500 to 1000 rows 78 us by all rows, 92 evenly; 4 ragged of up to
// 1500 91 and 118), less half a workgroup for each sequence but the first, whose last segment is short (6 ragged 146 us; 149
// with none less, 176 with a whole one; 4 91, 91 and 98).  Where that leaves one segment the longest sequence goes whole: 8
// ragged of up to 1500 rows take 225 us, 156 with none less, and of many single rows and one long sequence
// only that one's heads keep workgroups busy.
template <int DT, int D>
Segments make_segments(const Linear &l, void *ws) {
    constexpr int kHeld = D == 256 ? 256 : D == 128 ? 512 : DT == kDtF32 ? 1024 : 768;
    const int64_t a_head = kHeld / (l.heads * kSlices<D>), all = static_cast<int64_t>(l.B) * l.max_q;
    int64_t even;
    if (10 * static_cast<int64_t>(l.rows) >= 9 * all) {
        const int64_t segs = a_head / l.B > 1 ? a_head / l.B : 1;
        even = (l.max_q + segs - 1) / segs;
    } else {
        const int64_t segs = a_head - (l.B - 1) / 2 > 1 ? a_head - (l.B - 1) / 2 : 1;
        even = (l.rows + segs - 1) / segs;
    }
    const int64_t most = (static_cast<int64_t>(l.max_q) + kChunk - 1) / kChunk * kChunk;
    const int64_t each = ((even > 128 ? even : 128) + kChunk - 1) / kChunk * kChunk;
    Segments sg{static_cast<int>(each < most ? each : most), 0, static_cast<float *>(ws)};
    sg.places = (l.rows + sg.each - 1) / sg.each + l.B - 1;
    return sg;
}
// Few rows are done one by one: 32 sequences of 8 bf16 rows and 16 heads of 128 take 17 us either way, f32 18 and 25 us.
template <int DT>
bool row_by_row(const Linear &l) { return l.max_q <= (DT == kDtF32 ? 12 : 8); }

template <int DT, int D>
hipError_t launch_d(const Linear &l, void *ws, hipStream_t st) {
    if (row_by_row<DT>(l)) {
        hipLaunchKernelGGL((recurrent_kernel<DT, D>), dim3(l.B, l.heads * (D / kSlice)), dim3(256), 0, st, l);
        return hipGetLastError();
    }
    const Segments sg = make_segments<DT, D>(l, ws);
    const dim3 grid(static_cast<uint32_t>(items(l, sg, kSlices<D>))), block(64 * kLinWaves<D>);
    auto go = [&](auto kernel) {
        hipLaunchKernelGGL(kernel, grid, block, 0, st, l, sg);
        return hipGetLastError();
    };
    auto chunks = [&](auto out) {
        if constexpr (DT == kDtF32) return go(chunk_f32_kernel<DT, D, decltype(out)::value>);
        else return go(chunk_kernel<DT, D, decltype(out)::value>);
    };
    if (l.max_q > sg.each) {
        if (hipError_t e = chunks(std::false_type{}); e != hipSuccess) return e;
        hipLaunchKernelGGL(states_kernel, dim3(l.B * l.heads, D * D / 1024), dim3(256), 0, st, l, sg);
        if (hipError_t e = hipGetLastError(); e != hipSuccess) return e;
    }
    return chunks(std::true_type{});
}
template <int DT>
hipError_t launch_t(const Linear &l, void *ws, hipStream_t st) {
    if (l.D == 64) return launch_d<DT, 64>(l, ws, st);
    if (l.D == 128) return launch_d<DT, 128>(l, ws, st);
    return launch_d<DT, 256>(l, ws, st);
}
template <int DT, int D>
bool fits_d(const Linear &l) {
    return row_by_row<DT>(l) || items(l, make_segments<DT, D>(l, nullptr), kSlices<D>) * 64 * kLinWaves<D> < int64_t(1) << 32;
}
template <int DT>
bool fits_t(const Linear &l) {
    return l.D == 64 ? fits_d<DT, 64>(l) : l.D == 128 ? fits_d<DT, 128>(l) : fits_d<DT, 256>(l);
}
template <int DT, int D>
int64_t workspace_d(const Linear &l) {
    if (row_by_row<DT>(l)) return 0;
    const Segments sg = make_segments<DT, D>(l, nullptr);
    return l.max_q > sg.each ? static_cast<int64_t>(sg.places) * l.heads * D * D * 4 : 0;
}
template <int DT>
int64_t workspace_t(const Linear &l) {
    return l.D == 64 ? workspace_d<DT, 64>(l) : l.D == 128 ? workspace_d<DT, 128>(l) : workspace_d<DT, 256>(l);
}

}  // namespace

bool linear_fits(const Linear &l, int dtype) {
    return dtype == kDtF32 ? fits_t<kDtF32>(l) : dtype == kDtBf16 ? fits_t<kDtBf16>(l) : fits_t<kDtF16>(l);
}

int64_t linear_workspace(const Linear &l, int dtype) {
    return dtype == kDtF32 ? workspace_t<kDtF32>(l) : dtype == kDtBf16 ? workspace_t<kDtBf16>(l) : workspace_t<kDtF16>(l);
}

hipError_t launch_linear(const Linear &l, int dtype, void *workspace, hipStream_t st) {
    if (dtype == kDtF32) return launch_t<kDtF32>(l, workspace, st);
    if (dtype == kDtBf16) return launch_t<kDtBf16>(l, workspace, st);
    return launch_t<kDtF16>(l, workspace, st);
}

}  // namespace rad
