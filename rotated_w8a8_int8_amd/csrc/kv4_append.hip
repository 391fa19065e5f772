// kv4_append.hip -- new keys and values into the paged 4-bit cache, with the
// position rotation and the 128-point rotation on the way, and the read-back
// (gfx950).
//
// Append, per head vector x of a token at position p: pairs (a, b) become (a cos -
// b sin, b cos + a sin); y = x rotated per 128; scale = f16(amax / 6); codes =
// e2m1(y / scale).  An HBM stream for a prompt (the projection's output in, the
// turned queries and a few bytes of codes out), a chain of loads and one
// reduction for a few tokens.
//
// Values lie in octets of tokens (a dword = one dimension of eight tokens), so
// the work is split by octets: a workgroup takes up to eight consecutive tokens
// of one octet of one sequence and a few heads, each token's head held by D / 8
// lanes, 8 values each (lane layout of rotate_quant.h).  The codes of a head's
// values cross LDS once to become dwords; a dword that the call fills only
// partly is read and merged.  No other workgroup of the call writes that dword,
// so nothing is atomic.  Where every sequence has one row no octet has two tokens
// to bring together: a kernel of its own holds a head a 16-lane group (1024
// sequences 100 us by octets, 14.6 us, read-back counted).
//
// 8192 f32 tokens of 40 query and 8 KV heads of 128 take 94 us, 4.4 TB/s of the
// 412 MB it moves, its mix of reads and writes being a copy's (4.9 TB/s); one
// token of 8 sequences 3.1 us, 8 x 16 bf16 tokens 7.9 us.  The read-back is a
// stream: 12 us for the 8192 tokens.
#include "kv4.h"
#include "rotate_quant.h"

namespace rad {
namespace {

// (a cos - b sin, b cos + a sin), every operation rounded by itself.
__device__ __forceinline__ float turn_first(float a, float b, float cs, float sn) {
#pragma clang fp contract(off)
    return a * cs - b * sn;
}
__device__ __forceinline__ float turn_second(float a, float b, float cs, float sn) {
#pragma clang fp contract(off)
    return b * cs + a * sn;
}

// A lane's two runs of four values of a head vector.
struct Runs {
    float4 lo, hi;
};

// The position rotation of a lane's runs at d0 and d1.  Where a pair's halves lie d1 - d0
// apart (style 0, dim = 2 (d1 - d0): the usual whole-head rotation for D = 64 and 128)
// the lane holds both, and lo and hi share one set of angles; style 1 pairs neighbours;
// otherwise the other half is read again.
struct Angles {
    float4 c0, s0, c1, s1;      // cosines and sines for lo and for hi
};
template <int D>
__device__ __forceinline__ Angles angles(const float *tab, int dim, int style, int d0, int d1) {
    const int half = dim >> 1;
    Angles a{};
    if (style == 1) {
        auto two = [&](int d, float4 &c, float4 &s) {
            if (d >= dim) return;
            const float2 x = *reinterpret_cast<const float2 *>(tab + (d >> 1)), y = *reinterpret_cast<const float2 *>(tab + half + (d >> 1));
            c = make_float4(x.x, x.y, 0.f, 0.f);
            s = make_float4(y.x, y.y, 0.f, 0.f);
        };
        two(d0, a.c0, a.s0);
        two(d1, a.c1, a.s1);
    } else {
        if (d0 < dim) {
            const int j = d0 < half ? d0 : d0 - half;
            a.c0 = load4<kDtF32>(tab, j);
            a.s0 = load4<kDtF32>(tab, half + j);
        }
        if (half == d1 - d0) return a;
        if (d1 < dim) {
            const int j = d1 < half ? d1 : d1 - half;
            a.c1 = load4<kDtF32>(tab, j);
            a.s1 = load4<kDtF32>(tab, half + j);
        }
    }
    return a;
}
__device__ __forceinline__ float4 firsts(float4 a, float4 b, float4 c, float4 s) {
    return make_float4(turn_first(a.x, b.x, c.x, s.x), turn_first(a.y, b.y, c.y, s.y), turn_first(a.z, b.z, c.z, s.z),
                       turn_first(a.w, b.w, c.w, s.w));
}
__device__ __forceinline__ float4 seconds(float4 a, float4 b, float4 c, float4 s) {
    return make_float4(turn_second(a.x, b.x, c.x, s.x), turn_second(a.y, b.y, c.y, s.y), turn_second(a.z, b.z, c.z, s.z),
                       turn_second(a.w, b.w, c.w, s.w));
}
template <int DT>
__device__ __forceinline__ void turn(Runs &v, const Angles &a, const void *src, int64_t base, int dim, int style, int d0,
                                     int d1) {
    const int half = dim >> 1;
    if (style == 1) {
        auto two = [](float4 x, float4 c, float4 s) {
            return make_float4(turn_first(x.x, x.y, c.x, s.x), turn_second(x.x, x.y, c.x, s.x),
                               turn_first(x.z, x.w, c.y, s.y), turn_second(x.z, x.w, c.y, s.y));
        };
        if (d0 < dim) v.lo = two(v.lo, a.c0, a.s0);
        if (d1 < dim) v.hi = two(v.hi, a.c1, a.s1);
    } else if (half == d1 - d0) {
        if (d0 < half) {                                      // heads of 256: the first 128 alone
            const float4 x = v.lo, y = v.hi;
            v.lo = firsts(x, y, a.c0, a.s0);
            v.hi = seconds(x, y, a.c0, a.s0);
        }
    } else {
        auto one = [&](float4 x, int d, float4 c, float4 s) {
            if (d >= dim) return x;
            const float4 o = load4<DT>(src, base + (d < half ? d + half : d - half));
            return d < half ? firsts(x, o, c, s) : seconds(o, x, c, s);
        };
        v.lo = one(v.lo, d0, a.c0, a.s0);
        v.hi = one(v.hi, d1, a.c1, a.s1);
    }
}

// Maximum over the L lanes of a head vector (L = 8, 16 or 32).
template <int L>
__device__ __forceinline__ float head_max(float a) {
    a = fmaxf(a, lane_xor<1>(a));
    a = fmaxf(a, lane_xor<2>(a));
    a = fmaxf(a, lane_xor<4>(a));
    if constexpr (L >= 16) a = fmaxf(a, lane_xor<8>(a));
    if constexpr (L >= 32) a = fmaxf(a, __shfl_xor(a, 16));
    return a;
}

// One head vector v of a token (kind 0: query, 1: key, 2: value, head h of its kind), by D / 8
// lanes: the turned query stored, or scale and keys' codes; returns the lane's eight codes.
template <int DT, int D>
__device__ __forceinline__ uint32_t append_head(const Kv4Cache &c, const Kv4New &nw, Runs v, const Angles &ang, int kind, int h,
                                                int64_t base, int64_t trow, int page, int off, int lane, int d0, int d1,
                                                float sign) {
    const bool turned_too = D % 128 == 0 && nw.rotate;
    if (kind < 2 && nw.rope) turn<DT>(v, ang, kind == 0 ? nw.q : nw.k, base, nw.rope_dim, nw.rope_style, d0, d1);
    if (turned_too) {
        Blk8 x{v.lo, v.hi};
        fwht128_regs_signed(x, lane & 15);
        v = Runs{x.lo, x.hi};
    }
    if (kind == 0) {
        const float m = turned_too ? sign * 0x1p-7f : 1.0f;
        const int64_t at = (trow * nw.q_heads + h) * D;
        store4<DT>(nw.q_out, at + d0, make_float4(v.lo.x * m, v.lo.y * m, v.lo.z * m, v.lo.w * m));
        store4<DT>(nw.q_out, at + d1, make_float4(v.hi.x * m, v.hi.y * m, v.hi.z * m, v.hi.w * m));
        return 0;
    }
    float r[8] = {v.lo.x, v.lo.y, v.lo.z, v.lo.w, v.hi.x, v.hi.y, v.hi.z, v.hi.w};
    float a = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) a = fmaxf(a, fabsf(r[i]));
    a = head_max<D / 8>(a);
    const uint32_t sb = kv4_scale_bits(a / 6.0f);
    const float s = f16_widen(sb);
    uint32_t w = 0;
    if (s > 0.0f) {
        const float d = sign * s;
#pragma unroll
        for (int i = 0; i < 8; ++i) r[i] = r[i] / d;
        w = e2m1_pack8(r);
    }
    if (page >= 0) {
        const int64_t tok = ((static_cast<int64_t>(page) * c.heads + h) << c.page_shift) + off;
        if (lane == 0) (kind == 1 ? c.k_scale : c.v_scale)[tok] = static_cast<uint16_t>(sb);
        if (kind == 1) {
            uint16_t *q = reinterpret_cast<uint16_t *>(c.k_codes + tok * (D / 2));
            q[d0 >> 2] = static_cast<uint16_t>(w);
            q[d1 >> 2] = static_cast<uint16_t>(w >> 16);
        }
    }
    return w;
}

// A lane's runs of a head vector: d0 .. d0 + 3 and d1 .. d1 + 3.
template <int D>
__device__ __forceinline__ int first_dim(int lane) { return D == 64 ? 4 * lane : (lane >> 4) * 128 + 4 * (lane & 15); }
template <int D>
constexpr int kRunsApart = D == 64 ? 32 : 64;

// One row per sequence: blockIdx.x the row, blockIdx.y 256 / L heads of it (queries, keys,
// values), D / 8 lanes each.  A value's lane puts its eight codes into the octet's dwords itself.
template <int DT, int D>
__global__ __launch_bounds__(256) void kv4_append_one_kernel(Kv4Cache c, KvBatch b, Kv4New nw) {
    constexpr int L = D / 8;
    const int lane = threadIdx.x % L, row = blockIdx.x, hx = blockIdx.y * (256 / L) + threadIdx.x / L;
    const int d0 = first_dim<D>(lane), d1 = d0 + kRunsApart<D>;
    const int H = c.heads, HQ = nw.q_heads;
    const int kind = hx < HQ ? 0 : hx < HQ + H ? 1 : hx < HQ + 2 * H ? 2 : 3;
    if (kind == 3) return;
    const int h = kind == 0 ? hx : kind == 1 ? hx - HQ : hx - HQ - H;
    const int64_t base = row * (kind == 0 ? nw.ldq : kind == 1 ? nw.ldk : nw.ldv) + static_cast<int64_t>(h) * D;
    const void *src = kind == 0 ? nw.q : kind == 1 ? nw.k : nw.v;
    const Runs v{load4<DT>(src, base + d0), load4<DT>(src, base + d1)};
    const int t = kv_len(b, row) - 1;
    if (t < 0 || (nw.rope && t >= nw.rope_rows)) return;
    const int page = kv_page(b, row, t, c.pages), off = t & ((1 << c.page_shift) - 1), sh = 4 * (t & 7);
    const bool merge = kind == 2 && page >= 0;
    uint4 *oct = nullptr, lo{}, hi{};
    if (merge) {
        oct = reinterpret_cast<uint4 *>(c.v_codes) + ((((static_cast<int64_t>(page) * H + h) << c.page_shift) + off) >> 3) * (D / 4);
        lo = oct[d0 >> 2];
        hi = oct[d1 >> 2];
    }
    const Angles ang = nw.rope && kind < 2 ? angles<D>(nw.rope + static_cast<int64_t>(t) * nw.rope_dim, nw.rope_dim, nw.rope_style, d0, d1)
                                           : Angles{};
    const float sign = D % 128 == 0 && nw.rotate ? fwht_lane_sign(lane & 15) : 1.0f;
    const uint32_t w = append_head<DT, D>(c, nw, v, ang, kind, h, base, row, page, off, lane, d0, d1, sign);
    if (merge) {
        auto put = [&](uint32_t &word, int i) { word = (word & ~(15u << sh)) | (((w >> (4 * i)) & 15u) << sh); };
        put(lo.x, 0); put(lo.y, 1); put(lo.z, 2); put(lo.w, 3);
        put(hi.x, 4); put(hi.y, 5); put(hi.z, 6); put(hi.w, 7);
        oct[d0 >> 2] = lo;
        oct[d1 >> 2] = hi;
    }
}

// blockIdx.x: `chunk` consecutive rows, of which the workgroup takes the octets that begin
// there; blockIdx.y: `span` groups of HPB heads of the q_heads + 2 * heads in the order
// queries, keys, values.  A thread's token, and with it its angles, stays while the heads
// go by, the next head's values being on their way.
template <int DT, int D>
__global__ __launch_bounds__(256) void kv4_append_kernel(Kv4Cache c, KvBatch b, Kv4New nw, int chunk, int span) {
    constexpr int L = D / 8, HPB = 32 / L;
    __shared__ uint32_t codes[HPB][8][L];                 // [head][token of the octet][lane]: 8 codes of a lane
    const int lane = threadIdx.x % L, tok = (threadIdx.x / L) % 8, hs = threadIdx.x / (8 * L);
    const int d0 = first_dim<D>(lane), d1 = d0 + kRunsApart<D>;
    const int H = c.heads, HQ = nw.q_heads, heads = HQ + 2 * H;
    const int hb0 = blockIdx.y * span, hb1 = min(hb0 + span, (heads + HPB - 1) / HPB);
    const float sign = D % 128 == 0 && nw.rotate ? fwht_lane_sign(lane & 15) : 1.0f;     // what fwht128_regs_signed leaves on a lane

    const int row_end = min(static_cast<int>(blockIdx.x + 1) * chunk, b.rows);
    for (int row = blockIdx.x * chunk; row < row_end;) {
        const SeqOfRow found = kv_seq_of_wave(b, row);
        const int seq = found.seq;
        if (seq < 0) {
            ++row;
            continue;
        }
        const RowRange rr = found.rr;
        const int pos0 = found.len - rr.n;                   // position of the sequence's first row
        const int seq_end = min(rr.first + rr.n, row_end), last = pos0 + rr.n - 1;
        // the first row here that begins an octet or the sequence's tokens
        int p = max(pos0 + (row - rr.first), 0);
        if ((p & 7) != 0 && p != max(pos0, 0)) p = (p | 7) + 1;
        for (; rr.first + (p - pos0) < seq_end; p = (p | 7) + 1) {
            const int octet = p >> 3;                         // tokens p .. min(last, 8 * octet + 7)
            const int t = octet * 8 + tok;
            const bool here = t >= p && t <= last && (!nw.rope || t < nw.rope_rows);
            const int64_t trow = rr.first + (t - pos0);
            const int page = kv_page(b, seq, octet * 8, c.pages);
            const int off = (octet * 8) & ((1 << c.page_shift) - 1);
            const Angles ang = here && nw.rope ? angles<D>(nw.rope + static_cast<int64_t>(t) * nw.rope_dim, nw.rope_dim, nw.rope_style, d0, d1)
                                               : Angles{};
            auto base_of = [&](int hx) {
                return hx < HQ ? trow * nw.ldq + static_cast<int64_t>(hx) * D
                               : hx < HQ + H ? trow * nw.ldk + static_cast<int64_t>(hx - HQ) * D
                                             : trow * nw.ldv + static_cast<int64_t>(hx - HQ - H) * D;
            };
            auto source = [&](int hx) { return hx < HQ ? nw.q : hx < HQ + H ? nw.k : nw.v; };
            auto fetch = [&](int hx) {
                Runs v{};
                if (here && hx < heads) {
                    v.lo = load4<DT>(source(hx), base_of(hx) + d0);
                    v.hi = load4<DT>(source(hx), base_of(hx) + d1);
                }
                return v;
            };
            Runs next = fetch(hb0 * HPB + hs);
            for (int hb = hb0; hb < hb1; ++hb) {
                const int hx = hb * HPB + hs;
                Runs v = next;
                if (hb + 1 < hb1) next = fetch(hx + HPB);
                const int kind = hx < HQ ? 0 : hx < HQ + H ? 1 : hx < heads ? 2 : 3;       // query, key, value, none
                const int h = kind == 0 ? hx : kind == 1 ? hx - HQ : hx - HQ - H;
                uint32_t w = 0;
                if (here && kind < 3) w = append_head<DT, D>(c, nw, v, ang, kind, h, base_of(hx), trow, page, off + tok, lane, d0, d1, sign);
                if ((hb + 1) * HPB <= HQ + H || page < 0) continue;   // no values among the workgroup's heads
                __syncthreads();                              // the group before is read
                if (kind == 2) codes[hs][tok][lane] = w;
                __syncthreads();
                if (kind == 2) {
                    // one thread per dword: dimension d of head hs, the octet's eight tokens
                    const int d = threadIdx.x % D;
                    const int dl = d % 128, ln = D == 64 ? (d % 32) / 4 : (d / 128) * 16 + (dl % 64) / 4;
                    const int nib = 4 * (d % 4) + (D == 64 ? (d >= 32 ? 16 : 0) : (dl >= 64 ? 16 : 0));
                    uint32_t word = 0, mask = 0;
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const int tj = octet * 8 + j;
                        const bool on = tj >= p && tj <= last && (!nw.rope || tj < nw.rope_rows);
                        word |= ((codes[hs][j][ln] >> nib) & 15u) << (4 * j);
                        mask |= on ? 15u << (4 * j) : 0u;
                    }
                    const int64_t vec = (static_cast<int64_t>(page) * H + h) << c.page_shift;
                    uint32_t *q = reinterpret_cast<uint32_t *>(c.v_codes) + ((vec + off) >> 3) * D + d;
                    *q = mask == 0xFFFFFFFFu ? word : (*q & ~mask) | (word & mask);
                }
            }
        }
        row = rr.first + rr.n;
    }
}

template <int DT, int D>
hipError_t append_d(const Kv4Cache &c, const KvBatch &b, const Kv4New &n, hipStream_t st) {
    const int heads = n.q_heads + 2 * c.heads;
    if (!b.q_start) {
        const dim3 grid(b.rows, (heads * (D / 8) + 255) / 256);
        hipLaunchKernelGGL((kv4_append_one_kernel<DT, D>), grid, dim3(256), 0, st, c, b, n);
        return hipGetLastError();
    }
    // Rows a workgroup: an octet where sequences have that many, else as many as they have on
    // average, so that it does not walk from sequence to sequence (1024 of one row each: 100 us by
    // eights, 88 us by ones; 512 rows of one: 17 us by eights, 53 us by ones).  Heads a workgroup:
    // one group, until that gives more workgroups than the chip takes at once, then up to seven, each
    // token's angles being read once for them (8 x 16 rows 10 us with one, 23 us with seven; 8192
    // rows 111 us with four, 109 us with seven, 119 us with 28).
    constexpr int kSpan = 7, kFew = 1024;
    const int each = b.rows / b.B, chunk = each >= 8 ? 8 : each >= 4 ? 4 : each >= 2 ? 2 : 1;
    constexpr int hpb = 256 / D;
    const int groups = (heads + hpb - 1) / hpb;
    const int64_t all = static_cast<int64_t>((b.rows + chunk - 1) / chunk) * groups;
    const int span = static_cast<int>(all <= kFew ? 1 : all >= kSpan * kFew ? kSpan : all / kFew);
    const dim3 grid((b.rows + chunk - 1) / chunk, (groups + span - 1) / span);
    hipLaunchKernelGGL((kv4_append_kernel<DT, D>), grid, dim3(256), 0, st, c, b, n, chunk, span);
    return hipGetLastError();
}
template <int DT>
hipError_t append_t(const Kv4Cache &c, const KvBatch &b, const Kv4New &n, hipStream_t st) {
    if (c.D == 64) return append_d<DT, 64>(c, b, n, st);
    if (c.D == 128) return append_d<DT, 128>(c, b, n, st);
    return append_d<DT, 256>(c, b, n, st);
}

// One (row, head) vector by D / 8 lanes, eight consecutive values each.
template <int D>
__global__ __launch_bounds__(256) void kv4_read_kernel(Kv4Cache c, KvBatch b, uint16_t *__restrict__ k,
                                                       uint16_t *__restrict__ v) {
    constexpr int L = D / 8;
    const int lane = threadIdx.x % L;
    const int64_t idx = static_cast<int64_t>(blockIdx.x) * (256 / L) + threadIdx.x / L;
    if (idx >= static_cast<int64_t>(b.rows) * c.heads) return;
    const int row = static_cast<int>(idx / c.heads), h = static_cast<int>(idx % c.heads);
    const int seq = kv_seq_of(b, row);
    if (seq < 0) return;
    const RowRange rr = kv_rows(b, seq);
    const int t = kv_len(b, seq) - rr.n + (row - rr.first);
    if (t < 0) return;
    const int page = kv_page(b, seq, t, c.pages);
    if (page < 0) return;
    const int off = t & ((1 << c.page_shift) - 1);
    const int64_t vec = (static_cast<int64_t>(page) * c.heads + h) << c.page_shift;

    const float ks = f16_widen(c.k_scale[vec + off]), vs = f16_widen(c.v_scale[vec + off]);
    const uint32_t kw = reinterpret_cast<const uint32_t *>(c.k_codes + (vec + off) * (D / 2))[lane];
    const uint4 *vp = reinterpret_cast<const uint4 *>(c.v_codes + (((vec + off) >> 3) * D + 8 * lane) * 4);
    const uint4 va = vp[0], vb = vp[1];
    const int sh = 4 * (t & 7);
    const uint32_t vw = ((va.x >> sh) & 15u) | (((va.y >> sh) & 15u) << 4) | (((va.z >> sh) & 15u) << 8) |
                        (((va.w >> sh) & 15u) << 12) | (((vb.x >> sh) & 15u) << 16) | (((vb.y >> sh) & 15u) << 20) |
                        (((vb.z >> sh) & 15u) << 24) | (((vb.w >> sh) & 15u) << 28);
    auto pair = [](f2v x, float s) { return bf16_round(x[0] * s) | (bf16_round(x[1] * s) << 16); };
    auto eight = [&](uint32_t w, float s) {
        return make_uint4(pair(e2m1_pair<0>(w), s), pair(e2m1_pair<1>(w), s), pair(e2m1_pair<2>(w), s),
                          pair(e2m1_pair<3>(w), s));
    };
    reinterpret_cast<uint4 *>(k + idx * D)[lane] = eight(kw, ks);
    reinterpret_cast<uint4 *>(v + idx * D)[lane] = eight(vw, vs);
}

}  // namespace

hipError_t launch_kv4_append(const Kv4Cache &c, const KvBatch &b, const Kv4New &n, int dtype, hipStream_t st) {
    if (dtype == kDtF32) return append_t<kDtF32>(c, b, n, st);
    if (dtype == kDtBf16) return append_t<kDtBf16>(c, b, n, st);
    return append_t<kDtF16>(c, b, n, st);
}

hipError_t launch_kv4_read(const Kv4Cache &c, const KvBatch &b, uint16_t *k, uint16_t *v, hipStream_t st) {
    const int per = 2048 / c.D;
    const dim3 grid(static_cast<uint32_t>((static_cast<int64_t>(b.rows) * c.heads + per - 1) / per)), block(256);
    if (c.D == 64) hipLaunchKernelGGL(kv4_read_kernel<64>, grid, block, 0, st, c, b, k, v);
    else if (c.D == 128) hipLaunchKernelGGL(kv4_read_kernel<128>, grid, block, 0, st, c, b, k, v);
    else hipLaunchKernelGGL(kv4_read_kernel<256>, grid, block, 0, st, c, b, k, v);
    return hipGetLastError();
}

}  // namespace rad
