// kv4_select.hip -- the tokens of greatest weight of each sequence and KV head
// (gfx950).
//
// Weights become 32-bit keys of the same order (NaN lowest).  The budget's least key is
// found digit by digit, 11, 11 and 10 bits: a histogram of the keys that share the digits
// so far, from its top down to where the budget ends.  Every key above it is kept, and of
// those equal to it the first ones.  The list comes out in order because a wave takes a run
// of tokens and knows from the waves before it how many it follows.
#include "layer_launch.h"
#include "rad_device.h"

namespace rad {
namespace {

__device__ __forceinline__ uint32_t key_of(float w) {
    const uint32_t u = __float_as_uint(w + 0.0f);             // -0 is 0
    if ((u & 0x7FFFFFFFu) > 0x7F800000u) return 0u;
    return u >> 31 ? ~u : u | 0x80000000u;
}

constexpr int kSelThreads = 1024, kSelWaves = kSelThreads / 64, kBins = 2048;

// Sums over the lanes above this one, and over all lanes.
__device__ __forceinline__ int wave_suffix(int v, int lane) {
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
        const int o = __shfl_down(v, d);
        v += lane + d < 64 ? o : 0;
    }
    return v;
}

// One workgroup per (head, sequence).
__global__ __launch_bounds__(kSelThreads) void select_kernel(Kv4Select s) {
    __shared__ int hist[kBins];
    __shared__ int part[kSelWaves];
    __shared__ int found[2];                                  // digit, keys above it
    __shared__ int above[kSelWaves], equal[kSelWaves];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int h = blockIdx.y, seq = blockIdx.x;
    const int L = min(max(s.seq_len[seq], 0), s.max_tokens), n = min(L, s.budget);
    const int64_t pair = static_cast<int64_t>(seq) * s.heads + h;
    const float *w = s.weight + pair * s.ldw;
    int32_t *kept = s.kept + pair * s.budget;
    float *kw = s.kept_weight ? s.kept_weight + pair * s.ld_kept : nullptr;
    if (h == 0 && tid == 0) s.count[seq] = n;
    if (n == L) {                                             // everything is kept
        for (int t = tid; t < L; t += kSelThreads) {
            kept[t] = t;
            if (kw) kw[t] = w[t];
        }
        return;
    }
    // the tokens that weights decide about, and how many of them are kept
    const int lo = s.first, hi = L - s.recent, need = n - s.first - s.recent;
    uint32_t prefix = 0, known = 0;                           // digits found, and their bits
    int rest = need;                                          // keys still wanted among those that share them
#pragma unroll 1
    for (int pass = 0; pass < 3; ++pass) {
        const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0, bits = pass == 2 ? 10 : 11;
        for (int i = tid; i < kBins; i += kSelThreads) hist[i] = 0;
        __syncthreads();
        if (rest > 0)
            for (int t = lo + tid; t < hi; t += kSelThreads) {
                const uint32_t k = key_of(w[t]);
                if ((k & known) == prefix) atomicAdd(&hist[(k >> shift) & ((1u << bits) - 1)], 1);
            }
        __syncthreads();
        // digit d with keys in digits above it < rest <= those and its own
        const int h1 = hist[2 * tid + 1], h0 = hist[2 * tid], sum = wave_suffix(h0 + h1, lane);
        if (lane == 0) part[wave] = sum;
        if (tid == 0) found[0] = found[1] = 0;
        __syncthreads();
        int over = sum - h0 - h1;                             // keys in the digits of higher threads
        for (int x = wave + 1; x < kSelWaves; ++x) over += part[x];
        if (rest > over && rest <= over + h1) found[0] = 2 * tid + 1, found[1] = over;
        else if (rest > over + h1 && rest <= over + h1 + h0) found[0] = 2 * tid, found[1] = over + h1;
        __syncthreads();
        prefix |= static_cast<uint32_t>(found[0]) << shift;
        known |= ((1u << bits) - 1) << shift;
        rest -= found[1];
        __syncthreads();
    }
    // rest: how many of the keys equal to prefix are kept.  A wave's run of tokens, whole lines of 64
    const int run = ((L + 63) / 64 + kSelWaves - 1) / kSelWaves * 64, t0 = wave * run, t1 = min(t0 + run, L);
    auto look = [&](int t, bool &up, bool &tie) {
        const bool on = t < t1, sure = t < lo || t >= hi;
        const uint32_t k = on && need > 0 ? key_of(w[t]) : 0u;
        up = on && (sure || (need > 0 && k > prefix));
        tie = on && !sure && need > 0 && k == prefix;
    };
    int ups = 0, ties = 0;
    for (int t = t0; t < t1; t += 64) {
        bool up, tie;
        look(t + lane, up, tie);
        ups += __popcll(__ballot(up));
        ties += __popcll(__ballot(tie));
    }
    if (lane == 0) above[wave] = ups, equal[wave] = ties;
    __syncthreads();
    ups = ties = 0;
    for (int x = 0; x < wave; ++x) ups += above[x], ties += equal[x];
    const uint64_t before = (uint64_t(1) << lane) - 1;
    for (int t = t0; t < t1; t += 64) {
        bool up, tie;
        look(t + lane, up, tie);
        const uint64_t mu = __ballot(up), mt = __ballot(tie);
        const int tb = ties + __popcll(mt & before), at = ups + __popcll(mu & before) + min(tb, rest);
        if (up || (tie && tb < rest)) {
            kept[at] = t + lane;
            if (kw) kw[at] = w[t + lane];
        }
        ups += __popcll(mu);
        ties += __popcll(mt);
    }
}

}  // namespace

int64_t kv4_select_workspace(int64_t, int64_t, int64_t) { return 0; }

hipError_t launch_kv4_select(const Kv4Select &s, void *, hipStream_t st) {
    hipLaunchKernelGGL(select_kernel, dim3(s.B, s.heads), dim3(kSelThreads), 0, st, s);
    return hipGetLastError();
}

}  // namespace rad
