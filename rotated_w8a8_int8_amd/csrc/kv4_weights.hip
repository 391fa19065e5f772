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
#include "kv4_attn.h"

namespace rad {
namespace {

// A token's keys and their f16 levels, D / 2 dims a lane.
template <int D>
struct Keys {
    u4 f[D / 16];
    float scale;
};
template <int D>
__device__ __forceinline__ void load_keys(Keys<D> &k, const Kv4Cache &c, int64_t tok, int g, int r) {
    const u4 *p = reinterpret_cast<const u4 *>(c.k_codes + (tok + r) * (D / 2) + g * (D / 4));
#pragma unroll
    for (int j = 0; j < D / 64; ++j) {
        const u4 x = p[j];
#pragma unroll
        for (int i = 0; i < 4; ++i) k.f[4 * j + i] = levels8(x[i]);
    }
    k.scale = f16_widen(c.k_scale[tok + r]);
}

// What a pair's row brings to its scores: their factor, reference exponent, 1 / normaliser, position.
struct PairRow {
    float f, m, inv;
    int pos;
};

// blockIdx.x: sequence * parts + part, blockIdx.y: KV head.  Wave w of part x takes steps 4 x + w, 4 (x + parts) + w, ..
template <int DT, int D>
__global__ __launch_bounds__(256) void weights_kernel(Kv4Cache c, KvBatch b, Kv4Attn a, Kv4Weights w, int parts) {
    constexpr int NK = D / 16;
    constexpr bool SP = DT == kDtF32;
    __shared__ PairRow rows[kWaves][32];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int g = lane >> 5, col = lane & 31;
    const int h = blockIdx.y, G = a.q_heads / c.heads;
    const int seq = blockIdx.x / parts, part = blockIdx.x % parts;
    const RowRange rr = kv_rows(b, seq);
    if (rr.n == 0) return;
    const int len = kv_len(b, seq), base = len - rr.n;
    const int row0 = w.observe > 0 ? max(0, rr.n - w.observe) : 0, row1 = min(rr.n, b.max_q);
    const int pair0 = row0 * G, pair1 = max(row1, row0) * G;
    const Pages pages(c, b, seq, h, (len + 31) >> 5);

    u4 qf[NK], ql[SP ? NK : 1];
    bool far = false;
    // tile of pairs p0 ..: queries to f16 (as in attn_wide_kernel), rows to LDS
    auto load_tile = [&](int p0) {
        const int cp = p0 + col;
        const bool used = cp < pair1;
        const int ci = used ? cp / G : row0, cg = used ? cp % G : 0;
        const int64_t qrow = (static_cast<int64_t>(rr.first + ci) * a.q_heads + h * G + cg) * D;
        float qv[NK][8], big = 0.0f;
#pragma unroll
        for (int j = 0; j < NK; ++j) {
            const int64_t at = qrow + g * (D / 2) + 8 * j;
            const float4 x = load4<DT>(a.q, at), y = load4<DT>(a.q, at + 4);
            qv[j][0] = x.x; qv[j][1] = x.y; qv[j][2] = x.z; qv[j][3] = x.w;
            qv[j][4] = y.x; qv[j][5] = y.y; qv[j][6] = y.z; qv[j][7] = y.w;
        }
        const float2 st = a.stats[qrow / D];
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
        // a row that sees nothing has no statistics: it counts 0 times 1
        const bool on = used && base + ci >= 0 && st.y > 0.0f;
        far = __any(on && fabsf(st.x) > kNear);
        if (g == 0)
            rows[wave][col] = PairRow{on ? score_factor(a.sm_scale, e) : 0.0f, on ? st.x : 0.0f, on ? st.y : 0.0f, base + ci};
        __builtin_amdgcn_wave_barrier();
    };
    const bool one = pair1 - pair0 <= 32;
    if (one && pair1 > pair0) load_tile(pair0);

    for (int step = 4 * part + wave; step < pages.end; step += 4 * parts) {
        const int t0 = step << 5, t = t0 + col, page = pages.id(step);
        float total = 0.0f;
        if (page >= 0 && page < c.pages) {
            Keys<D> k;
            load_keys<D>(k, c, pages.token(page, step), g, col);
            // rows before the step's first token see none of it
            int p0 = pair0;
            if (a.causal && t0 > base + row0) p0 += (t0 - base - row0) * G & ~31;
            for (; p0 < pair1; p0 += 32) {
                if (!one) load_tile(p0);
                f16v s;
#pragma unroll
                for (int i = 0; i < 16; ++i) s[i] = 0.0f;
#pragma unroll
                for (int j = 0; j < NK; ++j) {
                    if constexpr (SP) s = mma32(ql[j], k.f[j], s);
                    s = mma32(qf[j], k.f[j], s);
                }
                float sum = 0.0f;
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    const PairRow r = rows[wave][8 * (i >> 2) + 4 * g + (i & 3)];
                    float x = fmaf(s[i] * k.scale, r.f, -r.m);
                    if (far) x = fminf(x, most_power(r.m));
                    const bool on = (!a.causal || t <= r.pos) && (a.window == 0 || t > r.pos - a.window);
                    sum += on ? __builtin_amdgcn_exp2f(x) * r.inv : 0.0f;
                }
                total += sum;
            }
        }
        total += __shfl_xor(total, 32);
        if (g == 0 && t < len) {
            float *at = w.weight + (static_cast<int64_t>(seq) * c.heads + h) * w.ldw + t;
            const float old = w.factor != 0.0f && t < base ? w.factor * *at : 0.0f;
            *at = old + total;
        }
    }
}

template <int DT>
hipError_t launch_t(const Kv4Cache &c, const KvBatch &b, const Kv4Attn &a, const Kv4Weights &w, hipStream_t st) {
    const int64_t steps = ((static_cast<int64_t>(b.max_pages) << b.page_shift) + 31) >> 5, all = static_cast<int64_t>(b.B) * c.heads;
    const int64_t most = (steps + 3) / 4, even = 2048 / all;
    const int parts = static_cast<int>(even < 1 ? 1 : even < most ? even : most);
    if (parts == 0) return hipSuccess;
    const dim3 grid(static_cast<uint32_t>(b.B) * parts, c.heads), block(64 * kWaves);
    auto go = [&](auto kernel) { hipLaunchKernelGGL(kernel, grid, block, 0, st, c, b, a, w, parts); };
    if (c.D == 64) go(weights_kernel<DT, 64>);
    else if (c.D == 128) go(weights_kernel<DT, 128>);
    else go(weights_kernel<DT, 256>);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_kv4_weights(const Kv4Cache &c, const KvBatch &b, const Kv4Attn &a, const Kv4Weights &w, int dtype, hipStream_t st) {
    if (dtype == kDtF32) return launch_t<kDtF32>(c, b, a, w, st);
    if (dtype == kDtBf16) return launch_t<kDtBf16>(c, b, a, w, st);
    return launch_t<kDtF16>(c, b, a, w, st);
}

}  // namespace rad
