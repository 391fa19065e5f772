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

// One workgroup per (row, query head); tiles of 256 tokens, a thread a token
// for the scores and a thread a dimension (of 256 / D token groups) for the sum.
template <int DT, int D>
__global__ __launch_bounds__(256) void attn_plain_kernel(Kv4Cache c, KvBatch b, Kv4Attn a) {
    __shared__ float qs[D], ps[256], red[8], part[256];
    const int row = blockIdx.x, hq = blockIdx.y, tid = threadIdx.x;
    const int h = hq / (a.q_heads / c.heads);
    const int seq = kv_seq_of(b, row);
    if (seq < 0) return;
    const RowRange rr = kv_rows(b, seq);
    if (row - rr.first >= b.max_q) return;
    const int len = kv_len(b, seq), pos = len - rr.n + (row - rr.first);
    const TokenRange tr = seen(pos, len, a.causal, a.window);
    const int64_t at = (static_cast<int64_t>(row) * a.q_heads + hq) * D;
    if (tid < D / 4) {
        const float4 x = load4<DT>(a.q, at + 4 * tid);
        const float f = a.sm_scale * kLog2e;
        qs[4 * tid] = x.x * f; qs[4 * tid + 1] = x.y * f; qs[4 * tid + 2] = x.z * f; qs[4 * tid + 3] = x.w * f;
    }
    __syncthreads();
    float m = -INFINITY, l = 0.0f, acc = 0.0f;
    const int d = tid % D, group = tid / D, per = 256 / (256 / D);         // tokens of a tile for a group
    for (int t0 = tr.lo & ~31; t0 < tr.hi; t0 += 256) {
        const int t = t0 + tid;
        const int page = t < tr.hi && t >= tr.lo ? kv_page(b, seq, t, c.pages) : -1;
        float s = -INFINITY, sv = 0.0f;
        if (page >= 0) {
            const int64_t vec = (static_cast<int64_t>(page) * c.heads + h) << c.page_shift;
            const int64_t tok = vec + (t & ((1 << c.page_shift) - 1));
            const uint32_t *kp = reinterpret_cast<const uint32_t *>(c.k_codes + tok * (D / 2));
            float sum = 0.0f;
            for (int j = 0; j < D / 8; ++j) {
                const uint32_t w = kp[j];
                const f2v x0 = e2m1_pair<0>(w), x1 = e2m1_pair<1>(w), x2 = e2m1_pair<2>(w), x3 = e2m1_pair<3>(w);
                const float *qq = qs + 8 * j;
                sum += qq[0] * x0[0] + qq[1] * x0[1] + qq[2] * x1[0] + qq[3] * x1[1] + qq[4] * x2[0] + qq[5] * x2[1] +
                       qq[6] * x3[0] + qq[7] * x3[1];
            }
            s = sum * f16_widen(c.k_scale[tok]);
            sv = f16_widen(c.v_scale[tok]);
        }
        const float wm = wave_max_f32(s);
        if ((tid & 63) == 0) red[tid >> 6] = wm;
        __syncthreads();
        const float mt = fmaxf(m, fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3])));
        const float p = s > -INFINITY ? __builtin_amdgcn_exp2f(s - mt) : 0.0f;
        const float ws = wave_sum_f32(p);
        if ((tid & 63) == 0) red[4 + (tid >> 6)] = ws;
        ps[tid] = s > -INFINITY ? p * sv : 0.0f;
        __syncthreads();
        const float scale = m > -INFINITY ? __builtin_amdgcn_exp2f(m - mt) : 0.0f;
        l = l * scale + ((red[4] + red[5]) + (red[6] + red[7]));
        acc *= scale;
        m = mt;
        for (int j = 0; j < per; j += 8) {
            const int tj = t0 + group * per + j;
            const int pg = tj < tr.hi ? kv_page(b, seq, tj, c.pages) : -1;
            if (pg < 0) continue;
            const int64_t vec = (static_cast<int64_t>(pg) * c.heads + h) << c.page_shift;
            const int64_t oct = (vec + (tj & ((1 << c.page_shift) - 1))) >> 3;
            const uint32_t w = reinterpret_cast<const uint32_t *>(c.v_codes)[oct * D + d];
            const f2v x0 = e2m1_pair<0>(w), x1 = e2m1_pair<1>(w), x2 = e2m1_pair<2>(w), x3 = e2m1_pair<3>(w);
            const float *pp = ps + group * per + j;
            acc += pp[0] * x0[0] + pp[1] * x0[1] + pp[2] * x1[0] + pp[3] * x1[1] + pp[4] * x2[0] + pp[5] * x2[1] +
                   pp[6] * x3[0] + pp[7] * x3[1];
        }
        __syncthreads();
    }
    part[tid] = acc;
    __syncthreads();
    if (tid < D / 4) {
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int g = 0; g < 256 / D; ++g) {
            const float *pp = part + g * D + 4 * tid;
            o.x += pp[0]; o.y += pp[1]; o.z += pp[2]; o.w += pp[3];
        }
        const float inv = l > 0.0f ? 1.0f / l : 0.0f;
        store4<DT>(a.o, at + 4 * tid, make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv));
    }
}

template <int DT>
hipError_t launch_t(const Kv4Cache &c, const KvBatch &b, const Kv4Attn &a, hipStream_t st) {
    const dim3 grid(b.rows, a.q_heads), block(256);
    if (c.D == 64) hipLaunchKernelGGL((attn_plain_kernel<DT, 64>), grid, block, 0, st, c, b, a);
    else if (c.D == 128) hipLaunchKernelGGL((attn_plain_kernel<DT, 128>), grid, block, 0, st, c, b, a);
    else hipLaunchKernelGGL((attn_plain_kernel<DT, 256>), grid, block, 0, st, c, b, a);
    return hipGetLastError();
}

}  // namespace

int64_t kv4_attn_workspace(const Kv4Cache &, const KvBatch &, int, int) { return 0; }

hipError_t launch_kv4_attn(const Kv4Cache &c, const KvBatch &b, const Kv4Attn &a, int dtype, hipStream_t st) {
    if (dtype == kDtF32) return launch_t<kDtF32>(c, b, a, st);
    if (dtype == kDtBf16) return launch_t<kDtBf16>(c, b, a, st);
    return launch_t<kDtF16>(c, b, a, st);
}

}  // namespace rad
