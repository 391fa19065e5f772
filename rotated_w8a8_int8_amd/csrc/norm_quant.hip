// norm_quant.hip -- residual addition, root-mean-square norm, 128-point
// rotation and per-token int8 quantisation in one pass (gfx950).
//
// Per token of K values: h = round_to_type(residual + x); r = 1 / sqrt(mean(h^2)
// + eps); n = (h * r) * gamma; n~ = n rotated per 128; s = max |n~| / 127;
// codes = rne(n~ / s).  The rotation mixes gamma's products, so two reductions
// over the row are needed, the sum of squares before it and the maximum after
// it; the row stays in registers between them.  The call reads x, the residual
// and gamma and writes h, codes and a scale: an HBM stream for many tokens, a
// chain of two reductions for few.
//
// A workgroup holds one token, each wave four 128-blocks a step (the lane layout
// of rotate_quant.h), NITER steps.  8192 tokens of 5120 f32 values with a residual
// take 93 to 94 us for the 545 MB that it reads and writes, 5.8 TB/s, where a copy that
// moves as much reaches 5.3, one of 4 GB 4.9 and a read-only stream 5.8.  Nontemporal
// accesses are no faster here and leave the codes out of the caches for the contraction
// (the call and a pass over its codes 203 us, 210 us with them).  128 bf16 tokens take
// 4.1 us and one f32 token 3.8 us: the launch, a trip to memory and the two reductions.
// A row whose squares leave f32's range takes two reductions more.
#include "layer_launch.h"
#include "rotate_quant.h"
#include "value_types.h"

namespace rad {
namespace {

// Sum of squares, and maximum, over the workgroup's row; `red` holds a value a wave.
template <int NITER>
__device__ __forceinline__ float row_sum_of_squares(const Blk8 (&v)[NITER], float (&red)[16]) {
    float ss = 0.0f;
#pragma unroll
    for (int it = 0; it < NITER; ++it) {
        const float4 a = v[it].lo, b = v[it].hi;
        ss += ((a.x * a.x + a.y * a.y) + (a.z * a.z + a.w * a.w)) + ((b.x * b.x + b.y * b.y) + (b.z * b.z + b.w * b.w));
    }
    ss = wave_sum_f32(ss);
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = ss;
    __syncthreads();
    float total = 0.0f;
    for (uint32_t w = 0; w < blockDim.x >> 6; ++w) total += red[w];
    return total;
}
__device__ __forceinline__ float row_max(float a, float (&red)[16]) {
    a = wave_max_f32(a);
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = a;
    __syncthreads();
    a = red[0];
    for (uint32_t w = 1; w < blockDim.x >> 6; ++w) a = fmaxf(a, red[w]);
    return a;
}
__device__ __forceinline__ float4 ldexp4(float4 f, int e) {
    return make_float4(__builtin_amdgcn_ldexpf(f.x, e), __builtin_amdgcn_ldexpf(f.y, e), __builtin_amdgcn_ldexpf(f.z, e),
                       __builtin_amdgcn_ldexpf(f.w, e));
}

template <int DT, int NITER>
__global__ __launch_bounds__(1024) void norm_quant_kernel(const void *x, const void *res, void *res_out,
                                                          const float *__restrict__ gamma, float eps,
                                                          int8_t *__restrict__ q, float *__restrict__ scale, int K,
                                                          int rotate) {
    __shared__ float red_sum[16], red_max[16];
    const int lane = threadIdx.x & 63, wid = threadIdx.x >> 6, waves = blockDim.x >> 6;
    const int l16 = lane & 15, nblk = K >> 7;
    const int64_t m = blockIdx.x, row = m * K;

    Blk8 v[NITER];
#pragma unroll
    for (int it = 0; it < NITER; ++it) {
        const int blk = (it * waves + wid) * 4 + (lane >> 4);
        if (blk < nblk) {
            const int64_t at = row + blk * 128 + 4 * l16;
            v[it].lo = load4<DT>(x, at);
            v[it].hi = load4<DT>(x, at + 64);
        } else {
            v[it].lo = make_float4(0.f, 0.f, 0.f, 0.f);
            v[it].hi = v[it].lo;
        }
    }
    if (res) {
#pragma unroll
        for (int it = 0; it < NITER; ++it) {
            const int blk = (it * waves + wid) * 4 + (lane >> 4);
            if (blk < nblk) {
                const int64_t at = row + blk * 128 + 4 * l16;
                const float4 a = load4<DT>(res, at), b = load4<DT>(res, at + 64);
                v[it].lo = make_float4(rounded<DT>(v[it].lo.x + a.x), rounded<DT>(v[it].lo.y + a.y),
                                       rounded<DT>(v[it].lo.z + a.z), rounded<DT>(v[it].lo.w + a.w));
                v[it].hi = make_float4(rounded<DT>(v[it].hi.x + b.x), rounded<DT>(v[it].hi.y + b.y),
                                       rounded<DT>(v[it].hi.z + b.z), rounded<DT>(v[it].hi.w + b.w));
                store4<DT>(res_out, at, v[it].lo);
                store4<DT>(res_out, at + 64, v[it].hi);
            }
        }
    }
    float total = row_sum_of_squares(v, red_sum);
    if constexpr (DT != kDtF16) {
        // Squares that leave f32's range (values past 2^63 or, where eps does not cover them, below
        // 2^-45): the row times a power of two, exactly, with eps to match.  The same for every thread.
        if (!(total < 0x1p127f) || (total < 0x1p-90f && eps < 0x1p-120f)) {
            float big = 0.0f;
#pragma unroll
            for (int it = 0; it < NITER; ++it) big = fmaxf(big, fmaxf(amax4(v[it].lo), amax4(v[it].hi)));
            const int e = max(__builtin_amdgcn_frexp_expf(row_max(big, red_max)), -100);
#pragma unroll
            for (int it = 0; it < NITER; ++it) {
                v[it].lo = ldexp4(v[it].lo, -e);
                v[it].hi = ldexp4(v[it].hi, -e);
            }
            total = row_sum_of_squares(v, red_sum);
            eps = __builtin_amdgcn_ldexpf(eps, -2 * e);
        }
    }
    const float r = 1.0f / __builtin_sqrtf(total / static_cast<float>(K) + eps);

    float amax = 0.0f;
#pragma unroll
    for (int it = 0; it < NITER; ++it) {
        const int blk = (it * waves + wid) * 4 + (lane >> 4);
        if (blk < nblk) {
            const float4 g = load4<kDtF32>(gamma, blk * 128 + 4 * l16), k = load4<kDtF32>(gamma, blk * 128 + 64 + 4 * l16);
            float4 &a = v[it].lo, &b = v[it].hi;
            a = make_float4(a.x * r * g.x, a.y * r * g.y, a.z * r * g.z, a.w * r * g.w);
            b = make_float4(b.x * r * k.x, b.y * r * k.y, b.z * r * k.z, b.w * r * k.w);
        }
        if (rotate) fwht128_regs_signed(v[it], l16);           // values times the lane sign c
        amax = fmaxf(amax, fmaxf(amax4(v[it].lo), amax4(v[it].hi)));
    }
    const float a = row_max(amax, red_max);
    const float s = a / 127.0f;
    if (threadIdx.x == 0) scale[m] = s;

    // codes as in quant_act_kernel: through the reciprocal, near-half ones redone
    // with the division, scales too small for a finite reciprocal divided throughout
    const bool fast = s >= 0x1p-120f;
    const float c = rotate ? fwht_lane_sign(l16) : 1.0f;
    const float rs_c = c * (1.0f / s);
#pragma unroll
    for (int it = 0; it < NITER; ++it) {
        const int blk = (it * waves + wid) * 4 + (lane >> 4);
        if (blk < nblk) {
            uint32_t lo = 0, hi = 0;
            if (fast) {
                lo = pack4_rcp_signed(v[it].lo, s, rs_c, c);
                hi = pack4_rcp_signed(v[it].hi, s, rs_c, c);
            } else if (s != 0.0f) {
                lo = pack4_signed(v[it].lo, s, c);
                hi = pack4_signed(v[it].hi, s, c);
            }
            uint32_t *p = reinterpret_cast<uint32_t *>(q + row + blk * 128 + 4 * l16);
            p[0] = lo;
            p[16] = hi;
        }
    }
}

struct Args {
    const void *x, *res;
    void *res_out;
    const float *gamma;
    float eps;
    int8_t *q;
    float *scale;
    int64_t M;
    int K, rotate;
    hipStream_t st;
};

template <int DT, int NITER>
hipError_t go(const Args &a, int waves) {
    hipLaunchKernelGGL((norm_quant_kernel<DT, NITER>), dim3(static_cast<uint32_t>(a.M)), dim3(waves * 64), 0,
                       a.st, a.x, a.res, a.res_out, a.gamma, a.eps, a.q, a.scale, a.K, a.rotate);
    return hipGetLastError();
}

template <int DT>
hipError_t launch(const Args &a) {
    const int nblk = a.K / 128;
    // As many waves as the row has groups of four blocks, so that each holds one step, up to 16
    // (5120 values: 128 tokens 10.5 us with 10 waves, 11.8 us with 4, codes widened after).  Of many
    // tokens a CU holds more where rows of more than 2048 take half the waves, two steps each (8192
    // bf16 tokens 162 us, 185 us in one step; 16384 x 1024 f32 has no second step to take).
    const int least = (nblk + 63) / 64, niter = a.M >= 1024 && nblk > 16 && least < 2 ? 2 : least;
    const int waves = (nblk + 4 * niter - 1) / (4 * niter);
    if (niter <= 1) return go<DT, 1>(a, waves);
    if (niter <= 2) return go<DT, 2>(a, waves);
    if (niter <= 4) return go<DT, 4>(a, waves);
    return go<DT, 8>(a, waves);                                // K <= 65536
}

}  // namespace

hipError_t launch_norm_quant(const void *x, const void *res, void *res_out, const float *gamma, float eps,
                             int8_t *q, float *scale, int64_t M, int K, int dtype, int rotate, hipStream_t st) {
    const Args a{x, res, res_out, gamma, eps, q, scale, M, K, rotate, st};
    if (dtype == kDtF32) return launch<kDtF32>(a);
    if (dtype == kDtBf16) return launch<kDtBf16>(a);
    return launch<kDtF16>(a);
}

}  // namespace rad
