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
// so nothing is atomic.
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

// Four consecutive values d .. d + 3 (d % 4 == 0) of the head at `base` after
// the position rotation; tab is the position's table row.
template <int DT>
__device__ __forceinline__ float4 turned4(const void *src, int64_t base, int d, const float *tab, int dim, int style) {
    const float4 x = load4<DT>(src, base + d);
    if (d >= dim) return x;
    const int half = dim >> 1;
    if (style == 1) {
        const float2 cs = *reinterpret_cast<const float2 *>(tab + (d >> 1));
        const float2 sn = *reinterpret_cast<const float2 *>(tab + half + (d >> 1));
        return make_float4(turn_first(x.x, x.y, cs.x, sn.x), turn_second(x.x, x.y, cs.x, sn.x),
                           turn_first(x.z, x.w, cs.y, sn.y), turn_second(x.z, x.w, cs.y, sn.y));
    }
    const bool first = d < half;
    const int j = first ? d : d - half;
    const float4 o = load4<DT>(src, base + (first ? d + half : j));
    const float4 cs = load4<kDtF32>(tab, j), sn = load4<kDtF32>(tab, half + j);
    if (first)
        return make_float4(turn_first(x.x, o.x, cs.x, sn.x), turn_first(x.y, o.y, cs.y, sn.y),
                           turn_first(x.z, o.z, cs.z, sn.z), turn_first(x.w, o.w, cs.w, sn.w));
    return make_float4(turn_second(o.x, x.x, cs.x, sn.x), turn_second(o.y, x.y, cs.y, sn.y),
                       turn_second(o.z, x.z, cs.z, sn.z), turn_second(o.w, x.w, cs.w, sn.w));
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

// blockIdx.x: `chunk` consecutive rows; blockIdx.y: HPB heads of the q_heads +
// 2 * heads in the order queries, keys, values.
template <int DT, int D>
__global__ __launch_bounds__(256) void kv4_append_kernel(Kv4Cache c, KvBatch b, Kv4New nw, int chunk) {
    constexpr int L = D / 8, HPB = 32 / L;
    __shared__ uint32_t codes[HPB][8][L];                 // [head][token of the octet][lane]: 8 codes of a lane
    const int lane = threadIdx.x % L, tok = (threadIdx.x / L) % 8, hs = threadIdx.x / (8 * L);
    const int l16 = lane & 15;
    // a lane's two runs of four values: d0 .. d0 + 3 and d1 .. d1 + 3
    const int d0 = D == 64 ? 4 * lane : (lane >> 4) * 128 + 4 * l16, d1 = d0 + (D == 64 ? 32 : 64);
    const int hx = blockIdx.y * HPB + hs, H = c.heads, HQ = nw.q_heads;
    const int kind = hx < HQ ? 0 : hx < HQ + H ? 1 : hx < HQ + 2 * H ? 2 : 3;       // query, key, value, none
    const int h = kind == 0 ? hx : kind == 1 ? hx - HQ : hx - HQ - H;
    const void *src = kind == 0 ? nw.q : kind == 1 ? nw.k : nw.v;
    const int64_t ld = kind == 0 ? nw.ldq : kind == 1 ? nw.ldk : nw.ldv;

    const int row_end = min(static_cast<int>(blockIdx.x + 1) * chunk, b.rows);
    for (int row = blockIdx.x * chunk; row < row_end; ++row) {
        // this row's octet is the workgroup's if the row is its first token in the call
        const int seq = kv_seq_of(b, row);
        if (seq < 0) continue;
        const RowRange rr = kv_rows(b, seq);
        const int pos0 = kv_len(b, seq) - rr.n;              // position of the sequence's first row
        const int pos = pos0 + (row - rr.first);
        if (pos < 0 || !((pos & 7) == 0 || pos == max(pos0, 0))) continue;
        const int octet = pos >> 3, last = pos0 + rr.n - 1;   // tokens pos .. min(last, 8 * octet + 7)
        const int t = octet * 8 + tok;
        const bool live = t >= pos && t <= last && kind < 3 && (!nw.rope || t < nw.rope_rows);
        const int page = kv_page(b, seq, octet * 8, c.pages);
        const int off = (octet * 8) & ((1 << c.page_shift) - 1);

        float r[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
        if (live) {
            const int64_t base = static_cast<int64_t>(rr.first + (t - pos0)) * ld + static_cast<int64_t>(h) * D;
            Blk8 v;
            if (kind < 2 && nw.rope) {
                const float *tab = nw.rope + static_cast<int64_t>(t) * nw.rope_dim;
                v.lo = turned4<DT>(src, base, d0, tab, nw.rope_dim, nw.rope_style);
                v.hi = turned4<DT>(src, base, d1, tab, nw.rope_dim, nw.rope_style);
            } else {
                v.lo = load4<DT>(src, base + d0);
                v.hi = load4<DT>(src, base + d1);
            }
            if (D % 128 == 0 && nw.rotate) fwht128_regs(v, l16);
            if (kind == 0) {
                const float m = D % 128 == 0 && nw.rotate ? 0x1p-7f : 1.0f;
                const int64_t at = (static_cast<int64_t>(rr.first + (t - pos0)) * HQ + h) * D;
                store4<DT>(nw.q_out, at + d0, make_float4(v.lo.x * m, v.lo.y * m, v.lo.z * m, v.lo.w * m));
                store4<DT>(nw.q_out, at + d1, make_float4(v.hi.x * m, v.hi.y * m, v.hi.z * m, v.hi.w * m));
            } else {
                r[0] = v.lo.x; r[1] = v.lo.y; r[2] = v.lo.z; r[3] = v.lo.w;
                r[4] = v.hi.x; r[5] = v.hi.y; r[6] = v.hi.z; r[7] = v.hi.w;
            }
        }
        // a head vector's lanes are live together, so its reduction sees only live lanes
        uint32_t w = 0;
        if (live && kind != 0) {
            float a = 0.0f;
#pragma unroll
            for (int i = 0; i < 8; ++i) a = fmaxf(a, fabsf(r[i]));
            a = head_max<L>(a);
            const uint32_t sb = kv4_scale_bits(a / 6.0f);
            const float s = f16_widen(sb);
            if (s > 0.0f) {
#pragma unroll
                for (int i = 0; i < 8; ++i) r[i] = r[i] / s;
                w = e2m1_pack8(r);
            }
            if (page >= 0) {
                const int64_t vec = (static_cast<int64_t>(page) * H + h) << c.page_shift;    // first token of (page, head)
                if (lane == 0) (kind == 1 ? c.k_scale : c.v_scale)[vec + off + tok] = static_cast<uint16_t>(sb);
                if (kind == 1) {
                    uint16_t *p = reinterpret_cast<uint16_t *>(c.k_codes + (vec + off + tok) * (D / 2));
                    p[d0 >> 2] = static_cast<uint16_t>(w);
                    p[d1 >> 2] = static_cast<uint16_t>(w >> 16);
                }
            }
        }
        __syncthreads();                                     // the last octet's codes are read
        if (kind == 2) codes[hs][tok][lane] = w;
        __syncthreads();
        if (kind == 2 && page >= 0) {
            // one thread per dword: dimension d of head hs, the octet's eight tokens
            const int d = threadIdx.x % D;
            const int dl = d % 128, ln = D == 64 ? (d % 32) / 4 : (d / 128) * 16 + (dl % 64) / 4;
            const int nib = 4 * (d % 4) + (D == 64 ? (d >= 32 ? 16 : 0) : (dl >= 64 ? 16 : 0));
            uint32_t word = 0, mask = 0;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int tj = octet * 8 + j;
                const bool on = tj >= pos && tj <= last && (!nw.rope || tj < nw.rope_rows);
                word |= ((codes[hs][j][ln] >> nib) & 15u) << (4 * j);
                mask |= on ? 15u << (4 * j) : 0u;
            }
            const int64_t vec = (static_cast<int64_t>(page) * H + h) << c.page_shift;
            uint32_t *p = reinterpret_cast<uint32_t *>(c.v_codes) + ((vec + off) >> 3) * D + d;
            *p = mask == 0xFFFFFFFFu ? word : (*p & ~mask) | (word & mask);
        }
    }
}

template <int DT>
hipError_t append_t(const Kv4Cache &c, const KvBatch &b, const Kv4New &n, hipStream_t st) {
    // Few rows: a workgroup for each, so that no octet waits for another.  Many:
    // one for every eight, so that most find one octet to do.
    const int chunk = b.rows <= 512 ? 1 : 8;
    const int hpb = 256 / c.D, heads = n.q_heads + 2 * c.heads;
    const dim3 grid((b.rows + chunk - 1) / chunk, (heads + hpb - 1) / hpb), block(256);
    if (c.D == 64) hipLaunchKernelGGL((kv4_append_kernel<DT, 64>), grid, block, 0, st, c, b, n, chunk);
    else if (c.D == 128) hipLaunchKernelGGL((kv4_append_kernel<DT, 128>), grid, block, 0, st, c, b, n, chunk);
    else hipLaunchKernelGGL((kv4_append_kernel<DT, 256>), grid, block, 0, st, c, b, n, chunk);
    return hipGetLastError();
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
