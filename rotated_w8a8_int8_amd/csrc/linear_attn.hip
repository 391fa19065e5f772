// linear_attn.hip -- linear attention with a decay for each head (gfx950).
//
//   S = exp(g) S + k v^T,  o = scale S^T q, row by row; S [D][D] in f32.
//
// Row by row (single tokens): a workgroup holds 64 of a head's D value columns, D / 16
// of the key's rows a thread, four columns each, and passes over its part of the state once.
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

template <int DT, int D>
hipError_t launch_d(const Linear &l, void *, hipStream_t st) {
    hipLaunchKernelGGL((recurrent_kernel<DT, D>), dim3(l.B, l.heads * (D / kSlice)), dim3(256), 0, st, l);
    return hipGetLastError();
}
template <int DT>
hipError_t launch_t(const Linear &l, void *ws, hipStream_t st) {
    if (l.D == 64) return launch_d<DT, 64>(l, ws, st);
    if (l.D == 128) return launch_d<DT, 128>(l, ws, st);
    return launch_d<DT, 256>(l, ws, st);
}

}  // namespace

int64_t linear_workspace(const Linear &, int) { return 0; }

hipError_t launch_linear(const Linear &l, int dtype, void *workspace, hipStream_t st) {
    if (dtype == kDtF32) return launch_t<kDtF32>(l, workspace, st);
    if (dtype == kDtBf16) return launch_t<kDtBf16>(l, workspace, st);
    return launch_t<kDtF16>(l, workspace, st);
}

}  // namespace rad
