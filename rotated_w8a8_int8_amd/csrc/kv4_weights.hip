// kv4_weights.hip -- attention weight of the cached tokens (gfx950).
//
// Behind an attention call that left each row's reference exponent m and normaliser l:
//
//   weight[t] = factor * weight[t] + sum over observed rows i and heads j of the group of
//               exp2(f_ij q_ij.k_t - m_ij) / l_ij
//
// The keys are read a second time, the values not at all.  A wave takes 32 tokens at a
// time against tiles of 32 (row, head) pairs:
//
//   S [32 pairs][32 tokens] = Q K^T, 32x32x16 matrix operations; a lane comes out with 16
//   pairs of one token, so that pairs are summed within the lane, and the two lanes of a
//   token meet once at the end.  Nothing is atomic: a token belongs to one wave.
//
// Few rows leave it to the memory: 32 bf16 rows over up to 30000 tokens each read 222 MB of
// keys and move 27 MB of weights in 56 us, 4.4 TB/s; 4096 tokens of one row take 5 us, latency.  Many rows are
// bound by a SIMD's vector work, about eight instructions and an exponent a pair and token: 288 f32 rows of
// 48 heads over 2913 tokens 87 us and 7 us for their pairs, beside 49 us for the attention; four ragged f16 prompts of up
// to 3000 rows, 32 heads of 64, 571 and 14 us beside 146 us with every row observed, 13 and 8 us beside 226 us (of other
// lengths) with the last 32, the pairs being made ready for every row of the call.
#include "kv4_attn.h"

namespace rad {
namespace {

// A step's key codes: D / 2 dims of token lane % 32, and its scale.
template <int D>
struct Codes {
    u4 k[D / 64];
    uint16_t scale;
};
template <int D>
__device__ __forceinline__ void load_codes(Codes<D> &s, const Kv4Cache &c, int64_t tok, int g, int r) {
    const u4 *p = reinterpret_cast<const u4 *>(c.k_codes + (tok + r) * (D / 2) + g * (D / 4));
#pragma unroll
    for (int j = 0; j < D / 64; ++j) s.k[j] = p[j];
    s.scale = c.k_scale[tok + r];
}

// What a pair's row brings to its scores: their factor, reference exponent, 1 / normaliser, position.  A row
// that sees nothing, and a pair that is none, has no statistics: it counts 0 times 2^0.
struct PairRow {
    float f, m, inv;
    int pos;
};

// The sequence as the call counts it: its rows row0 .. row1 - 1 are observed.
struct Observed {
    RowRange rr;
    int len, base, pair0, pair1;
    __device__ __forceinline__ Observed(const KvBatch &b, const Kv4Attn &a, const Kv4Weights &w, int heads, int seq)
        : rr(kv_rows(b, seq)), len(kv_len(b, seq)), base(len - rr.n) {
        const int G = a.q_heads / heads, row0 = w.observe > 0 ? max(0, rr.n - w.observe) : 0;
        pair0 = row0 * G;
        pair1 = max(min(rr.n, b.max_q), row0) * G;
    }
};

template <int DT, int D>
struct Tile {                                             // 32 pairs as the matrix operations take them
    u4 hi[D / 16][64], lo[DT == kDtF32 ? D / 16 : 1][64];
    PairRow row[32];
    int far;                                              // a reference exponent past kNear is among them
};
// Eight threads a pair, D / 8 dims each (lane8 the thread's place): queries to f16, their largest value in [2^9,
// 2^10) as in attn_wide_kernel, and the pair's row.  at: the pair's index in [rows][q_heads]; ci: its row of the sequence.
template <int DT, int D>
__device__ __forceinline__ PairRow ready(const Kv4Attn &a, const Observed &ob, int64_t at, int ci, bool used, int lane8, u4 (&hi)[D / 64],
                                         u4 (&lo)[D / 64]) {
    constexpr int N = D / 64;                             // runs of 8 dims
    float x[N][8], big = 0.0f;
#pragma unroll
    for (int n = 0; n < N; ++n) {
        const float4 u = load4<DT>(a.q, at * D + 8 * (N * lane8 + n)), v = load4<DT>(a.q, at * D + 8 * (N * lane8 + n) + 4);
        x[n][0] = u.x; x[n][1] = u.y; x[n][2] = u.z; x[n][3] = u.w;
        x[n][4] = v.x; x[n][5] = v.y; x[n][6] = v.z; x[n][7] = v.w;
    }
    const float2 st = a.stats[at];
#pragma unroll
    for (int n = 0; n < N; ++n)
#pragma unroll
        for (int i = 0; i < 8; ++i) big = fmaxf(big, fabsf(x[n][i]));
    big = fmaxf(big, lane_xor<1>(big));
    big = fmaxf(big, lane_xor<2>(big));
    big = fmaxf(big, lane_xor<4>(big));
    const int e = big > 0.0f ? 10 - __builtin_amdgcn_frexp_expf(big) : 0;
    const bool token = used && ob.base + ci >= 0;             // else its values may be anything: scores of 0
#pragma unroll
    for (int n = 0; n < N; ++n) {
#pragma unroll
        for (int i = 0; i < 8; ++i) x[n][i] = token ? __builtin_amdgcn_ldexpf(x[n][i], e) : 0.0f;
        if constexpr (DT == kDtF32) f16_split8(x[n], hi[n], lo[n]);
        else hi[n] = f16_pack8(x[n]);
    }
    const bool on = token && st.y > 0.0f;
    return PairRow{on ? score_factor(a.sm_scale, e) : 0.0f, on ? st.x : 0.0f, on ? st.y : 0.0f, ob.base + ci};
}
template <int DT, int D>
__device__ __forceinline__ void stage(Tile<DT, D> &t, const Kv4Attn &a, const Observed &ob, int h, int G, int p0) {
    const int r = threadIdx.x >> 3, c = threadIdx.x & 7, cp = p0 + r;
    const bool used = cp < ob.pair1;
    const int ci = used ? cp / G : 0, cg = used ? cp % G : 0;
    u4 hi[D / 64], lo[D / 64];
    const PairRow pr = ready<DT, D>(a, ob, static_cast<int64_t>(ob.rr.first + ci) * a.q_heads + h * G + cg, ci, used, c, hi, lo);
#pragma unroll
    for (int n = 0; n < D / 64; ++n) {
        const int d = 8 * (D / 64 * c + n), slot = (d >= D / 2 ? 32 : 0) + r, j = (d & (D / 2 - 1)) >> 3;
        t.hi[j][slot] = hi[n];
        if constexpr (DT == kDtF32) t.lo[j][slot] = lo[n];
    }
    if (c == 0) {
        t.row[r] = pr;
        if (fabsf(pr.m) > kNear) t.far = 1;
    }
}

// A pair's probability of a token: s its product with the key, ks the key's scale.
__device__ __forceinline__ float probability(const PairRow &r, float s, float ks, bool far, bool causal, int window, int t) {
    float x = fmaf(s * ks, r.f, -r.m);
    if (far) x = fminf(x, most_power(r.m));
    const bool on = (!causal || t <= r.pos) && (window == 0 || t > r.pos - window);
    return on ? __builtin_amdgcn_exp2f(x) * r.inv : 0.0f;
}
// One lane's tokens: the sum of the two lanes that share one, added to what is there.
__device__ __forceinline__ void add_weight(const Kv4Weights &w, float *row, const Observed &ob, int t, int g, float total, float old) {
    total += __shfl_xor(total, 32);
    if (g == 0 && t < ob.len) row[t] = (w.factor != 0.0f && t < ob.base ? w.factor * old : 0.0f) + total;
}

// How the workgroups of a KV head share the steps, four at a time.  even 0: `parts` to every sequence.  Else (2 to 64
// sequences) parts of equal length, about `even` of them, found from all lengths: even + B workgroups hold them.
struct Split {
    int even, parts;
};
struct PartOf {
    int seq, part, parts;                                 // parts 0: none
};
// Every lane of the wave calls it and gets the same answer.
__device__ __forceinline__ PartOf part_of(const KvBatch &b, const Split &sp, int x) {
    if (sp.even == 0) return PartOf{x / sp.parts, x % sp.parts, sp.parts};
    const int lane = threadIdx.x & 63, i = min(lane, b.B - 1);
    const int fours = lane < b.B && kv_rows(b, i).n > 0 ? (kv_len(b, i) + 127) >> 7 : 0;
    const int all = __builtin_amdgcn_readlane(wave_scan(fours), 63), each = max(1, (all + sp.even - 1) / sp.even);
    const int parts = (fours + each - 1) / each, sum = wave_scan(parts);
    const uint64_t hit = __ballot(x >= sum - parts && x < sum);
    if (hit == 0) return PartOf{0, 0, 0};
    const int src = __builtin_ctzll(hit);
    return PartOf{src, x - __builtin_amdgcn_readlane(sum - parts, src), __builtin_amdgcn_readlane(parts, src)};
}

// At most 8 NQ pairs: queries stay in registers, the steps of a wave go through a ring of kRing on
// their way.  Rows 8 q + .. of the products are looked at for q < NQ alone.  blockIdx.x: a part,
// blockIdx.y: KV head; wave w of part x takes steps 4 x + w, 4 (x + parts) + w, ..
constexpr int kRing = 4;
template <int DT, int D, int NQ>
__global__ __launch_bounds__(256, NQ == 4 || D == 256 || (D == 128 && DT == kDtF32) ? 2 : 3) void weights_few_kernel(Kv4Cache c, KvBatch b, Kv4Attn a, Kv4Weights w, Split split) {
    constexpr int NK = D / 16;
    constexpr bool SP = DT == kDtF32;
    __shared__ Tile<DT, D> tile;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int g = lane >> 5, col = lane & 31;
    const int h = blockIdx.y, G = a.q_heads / c.heads;
    const PartOf mine = part_of(b, split, blockIdx.x);
    if (mine.parts == 0) return;
    const int seq = mine.seq;
    const Observed ob(b, a, w, c.heads, seq);
    if (ob.rr.n == 0) return;
    const Pages pages(c, b, seq, h, (ob.len + 31) >> 5);
    const int stride = 4 * mine.parts;
    int step = 4 * mine.part + wave;
    Codes<D> ring[kRing];
    int page[kRing + 1];
    float old[kRing];
    float *const row = w.weight + (static_cast<int64_t>(seq) * c.heads + h) * w.ldw;
    const int most = w.factor != 0.0f ? static_cast<int>(w.ldw) - 1 : 0;          // what is there does not matter: one line of it
    auto load = [&](int k, int p, int st) {
        load_codes<D>(ring[k], c, pages.token(p, st), g, col);
        old[k] = row[min((st << 5) + col, most)];
    };
#pragma unroll
    for (int k = 0; k < kRing + 1; ++k) page[k] = pages.id(step + k * stride);
#pragma unroll
    for (int k = 0; k < kRing - 1; ++k) load(k, page[k], step + k * stride);
    if (threadIdx.x == 0) tile.far = 0;
    __syncthreads();
    stage<DT, D>(tile, a, ob, h, G, ob.pair0);
    __syncthreads();
    u4 qf[NK], ql[SP ? NK : 1];
#pragma unroll
    for (int j = 0; j < NK; ++j) {
        qf[j] = tile.hi[j][lane];
        if constexpr (SP) ql[j] = tile.lo[j][lane];
    }
    PairRow rows[4 * NQ];
#pragma unroll
    for (int i = 0; i < 4 * NQ; ++i) rows[i] = tile.row[8 * (i >> 2) + 4 * g + (i & 3)];
    const bool far = tile.far;
    while (step < pages.end) {
#pragma unroll
        for (int k = 0; k < kRing; ++k) {
            constexpr int ahead = kRing - 1;
            load((k + ahead) % kRing, page[ahead], step + ahead * stride);
            const int t0 = step << 5, now = page[0];
#pragma unroll
            for (int i = 0; i < kRing; ++i) page[i] = page[i + 1];
            page[kRing] = pages.id(step + (kRing + 1) * stride);
            float total = 0.0f;
            if (now >= 0 && now < c.pages) {
                f16v s;
#pragma unroll
                for (int i = 0; i < 16; ++i) s[i] = 0.0f;
#pragma unroll
                for (int j = 0; j < NK; ++j) {
                    const u4 kf = levels8(ring[k].k[j >> 2][j & 3]);
                    if constexpr (SP) s = mma32(ql[j], kf, s);
                    s = mma32(qf[j], kf, s);
                }
                const float ks = f16_widen(ring[k].scale);
#pragma unroll
                for (int i = 0; i < 4 * NQ; ++i) total += probability(rows[i], s[i], ks, far, a.causal, a.window, t0 + col);
            }
            add_weight(w, row, ob, t0 + col, g, total, old[k]);
            step += stride;
            if (step >= pages.end) break;
        }
    }
}

// More pairs: their queries are made ready once (pairs_kernel), as f16 in the order in which a lane takes them,
// and their rows; every wave reads them as they lie.  A KV head's pairs follow each other row by row.
template <int DT, int D>
struct Pairs {
    u4 *hi, *lo;                      // [heads][rows * G][D / 16][2]: eight dims each
    PairRow *row;                     // [heads][rows * G]
    int64_t each;                     // rows * G
    __host__ __device__ Pairs(void *p, int64_t rows, int heads, int G) : each(rows * G) {
        row = static_cast<PairRow *>(p);
        hi = reinterpret_cast<u4 *>(row + each * heads);
        lo = hi + each * heads * (D / 8);
    }
};
// Eight threads a pair, D / 8 dims each; blockIdx.x: 32 pairs, blockIdx.y: KV head.
template <int DT, int D>
__global__ __launch_bounds__(256) void pairs_kernel(Kv4Cache c, KvBatch b, Kv4Attn a, Kv4Weights w) {
    const int h = blockIdx.y, G = a.q_heads / c.heads, lane8 = threadIdx.x & 7;
    const Pairs<DT, D> to(w.pairs, b.rows, c.heads, G);
    const int64_t cp = static_cast<int64_t>(blockIdx.x) * 32 + (threadIdx.x >> 3);
    const int row = static_cast<int>(min(cp / G, static_cast<int64_t>(b.rows) - 1)), seq = kv_seq_of(b, row);
    if (cp >= to.each || seq < 0) return;
    const Observed ob(b, a, w, c.heads, seq);
    const int64_t mine = cp - static_cast<int64_t>(ob.rr.first) * G;
    if (mine < ob.pair0 || mine >= ob.pair1) return;
    u4 hi[D / 64], lo[D / 64];
    const PairRow r = ready<DT, D>(a, ob, static_cast<int64_t>(row) * a.q_heads + h * G + cp % G, row - ob.rr.first, true, lane8, hi, lo);
    const int64_t at = h * to.each + cp;
#pragma unroll
    for (int n = 0; n < D / 64; ++n) {
        const int d = 8 * (D / 64 * lane8 + n), half = d >= D / 2, j = (d & (D / 2 - 1)) >> 3;
        to.hi[at * (D / 8) + 2 * j + half] = hi[n];
        if constexpr (DT == kDtF32) to.lo[at * (D / 8) + 2 * j + half] = lo[n];
    }
    if (lane8 == 0) to.row[at] = r;
}

// SPLIT 1: a wave takes a step and all its tiles of pairs; 4: the workgroup's waves take every fourth tile of one
// step, and their sums meet in LDS.
template <int DT, int D, int SPLIT>
__global__ __launch_bounds__(256, 2) void weights_many_kernel(Kv4Cache c, KvBatch b, Kv4Attn a, Kv4Weights w, int parts) {
    constexpr int NK = D / 16;
    constexpr bool SP = DT == kDtF32;
    __shared__ PairRow tile_rows[4][32];
    __shared__ float sums[SPLIT == 4 ? 4 : 1][32];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int g = lane >> 5, col = lane & 31;
    const int h = blockIdx.y, G = a.q_heads / c.heads;
    const int seq = blockIdx.x / parts, part = blockIdx.x % parts;
    const Observed ob(b, a, w, c.heads, seq);
    if (ob.rr.n == 0) return;
    const Pages pages(c, b, seq, h, (ob.len + 31) >> 5);
    const Pairs<DT, D> from(w.pairs, b.rows, c.heads, G);
    const int64_t pair_at = h * from.each + static_cast<int64_t>(ob.rr.first) * G;
    float *const row = w.weight + (static_cast<int64_t>(seq) * c.heads + h) * w.ldw;
    for (int first = 4 / SPLIT * part; first < pages.end; first += 4 / SPLIT * parts) {
        const int step = SPLIT == 4 ? first : first + wave, t = (step << 5) + col, page = pages.id(step);
        const bool here = page >= 0 && page < c.pages;
        Codes<D> codes;
        load_codes<D>(codes, c, pages.token(page, step), g, col);
        const float old = row[min(t, w.factor != 0.0f ? static_cast<int>(w.ldw) - 1 : 0)];
        // rows before the first token see none of the step
        int p0 = ob.pair0;
        if (a.causal && (step << 5) - ob.base > 0) p0 += max(0, ((step << 5) - ob.base) * G - ob.pair0) & ~31;
        if (SPLIT == 4) p0 += 32 * wave;
        u4 kf[NK];
#pragma unroll
        for (int j = 0; j < NK; ++j) kf[j] = levels8(codes.k[j >> 2][j & 3]);
        const float ks = f16_widen(codes.scale);
        float total = 0.0f;
        if (here)
            for (; p0 < ob.pair1; p0 += 32 * SPLIT) {
                const int cp = min(p0 + col, ob.pair1 - 1);
                const int64_t at = (pair_at + cp) * (D / 8) + g;
                u4 hi[NK], lo[SP ? NK : 1];
#pragma unroll
                for (int j = 0; j < NK; ++j) {
                    hi[j] = from.hi[at + 2 * j];
                    if constexpr (SP) lo[j] = from.lo[at + 2 * j];
                }
                PairRow r = from.row[pair_at + cp];
                if (p0 + col >= ob.pair1) r.inv = 0.0f;       // past the last pair: its scores again, which count nothing
                const bool far = __any(fabsf(r.m) > kNear);
                if (g == 0) tile_rows[wave][col] = r;
                __builtin_amdgcn_wave_barrier();
                f16v s;
#pragma unroll
                for (int i = 0; i < 16; ++i) s[i] = 0.0f;
#pragma unroll
                for (int j = 0; j < NK; ++j) {
                    if constexpr (SP) s = mma32(lo[j], kf[j], s);
                    s = mma32(hi[j], kf[j], s);
                }
                float sum = 0.0f;
#pragma unroll
                for (int i = 0; i < 16; ++i) sum += probability(tile_rows[wave][8 * (i >> 2) + 4 * g + (i & 3)], s[i], ks, far, a.causal, a.window, t);
                total += sum;
                __builtin_amdgcn_wave_barrier();
            }
        if (SPLIT == 4) {
            total += __shfl_xor(total, 32);
            if (g == 0) sums[wave][col] = total;
            __syncthreads();
            total = 0.5f * (sums[0][col] + sums[1][col] + sums[2][col] + sums[3][col]);      // add_weight adds both halves
            __syncthreads();
            if (wave != 0) continue;
        }
        add_weight(w, row, ob, t, g, total, old);
    }
}

// Pairs of a sequence and KV head that a call observes at most.
int64_t most_pairs(const KvBatch &b, int G, int observe) { return static_cast<int64_t>(observe > 0 && observe < b.max_q ? observe : b.max_q) * G; }
// Pairs that weights_few_kernel holds.
template <int D>
constexpr int kFew = D == 256 ? 8 : 32;

template <int DT, int D>
hipError_t launch_d(const Kv4Cache &c, const KvBatch &b, const Kv4Attn &a, const Kv4Weights &w, hipStream_t st) {
    const int64_t steps = ((static_cast<int64_t>(b.max_pages) << b.page_shift) + 31) >> 5, all = static_cast<int64_t>(b.B) * c.heads;
    if (steps == 0) return hipSuccess;
    const int G = a.q_heads / c.heads;
    // workgroups, of `held` steps each: about 2048, fewer where there are fewer steps
    auto go = [&](auto kernel, int held) {
        const int64_t most = (steps + held - 1) / held, even = 2048 / all;
        const int parts = static_cast<int>(even < 1 ? 1 : even < most ? even : most);
        hipLaunchKernelGGL(kernel, dim3(static_cast<uint32_t>(b.B) * parts, c.heads), dim3(64 * kWaves), 0, st, c, b, a, w, parts);
        return hipGetLastError();
    };
    // few pairs: several sequences by their lengths, in one round of the workgroups that 256 CUs hold, half a part a
    // sequence more than even counted in (bf16, one row each: 32 of up to 30000 tokens 156 -> 148 us a call, 8 of
    // 2000 20.3 -> 18.9; four rows, 16 of 8000 54 -> 44; two rounds 150, 19.2 and 46)
    auto go_few = [&](auto kernel, int held) {
        const int64_t most = (steps + 3) / 4, even = 2048 / all;
        Split sp{0, static_cast<int>(even < 1 ? 1 : even < most ? even : most)};
        int64_t pieces = static_cast<int64_t>(b.B) * sp.parts;
        if (b.B > 1 && b.B <= 64 && most > 1) {
            const int64_t round = 256 * held / c.heads, half = (round + 1) / 2, share = round - b.B / 2 > half ? round - b.B / 2 : half;
            sp.even = static_cast<int>(share < 1 ? 1 : share < b.B * most ? share : b.B * most);
            pieces = sp.even + b.B;
        }
        hipLaunchKernelGGL(kernel, dim3(static_cast<uint32_t>(pieces), c.heads), dim3(64 * kWaves), 0, st, c, b, a, w, sp);
        return hipGetLastError();
    };
    const int64_t pairs = most_pairs(b, G, w.observe);
    constexpr int held = D == 256 || (D == 128 && DT == kDtF32) ? 2 : 3;
    if (pairs <= 8) return go_few(weights_few_kernel<DT, D, 1>, held);
    if (pairs <= kFew<D>) return go_few(weights_few_kernel<DT, D <= 128 ? D : 64, 4>, 2);
    const int64_t each = static_cast<int64_t>(b.rows) * G;
    hipLaunchKernelGGL((pairs_kernel<DT, D>), dim3(static_cast<uint32_t>((each + 31) / 32), c.heads), dim3(256), 0, st, c, b, a, w);
    if (hipError_t e = hipGetLastError(); e != hipSuccess) return e;
    // few steps: four waves to a step
    if ((steps + 3) / 4 * all >= 1024) return go(weights_many_kernel<DT, D, 1>, 4);
    return go(weights_many_kernel<DT, D, 4>, 1);
}
template <int DT>
hipError_t launch_t(const Kv4Cache &c, const KvBatch &b, const Kv4Attn &a, const Kv4Weights &w, hipStream_t st) {
    if (c.D == 64) return launch_d<DT, 64>(c, b, a, w, st);
    if (c.D == 128) return launch_d<DT, 128>(c, b, a, w, st);
    return launch_d<DT, 256>(c, b, a, w, st);
}

}  // namespace

int64_t kv4_weights_workspace(const Kv4Cache &c, const KvBatch &b, int q_heads, int dtype) {
    const int64_t pairs = static_cast<int64_t>(b.rows) * q_heads, most = static_cast<int64_t>(b.max_q) * (q_heads / c.heads);
    if (most <= (c.D == 256 ? kFew<256> : kFew<128>)) return 0;
    return pairs * (c.D * (dtype == kDtF32 ? 4 : 2) + static_cast<int64_t>(sizeof(PairRow)));
}

hipError_t launch_kv4_weights(const Kv4Cache &c, const KvBatch &b, const Kv4Attn &a, const Kv4Weights &w, int dtype, hipStream_t st) {
    if (dtype == kDtF32) return launch_t<kDtF32>(c, b, a, w, st);
    if (dtype == kDtBf16) return launch_t<kDtBf16>(c, b, a, w, st);
    return launch_t<kDtF16>(c, b, a, w, st);
}

}  // namespace rad
