// kv4_select.hip -- the tokens of greatest weight of each sequence and KV head
// (gfx950).
//
// Weights become 32-bit keys of the same order (NaN lowest).  The budget's least key is
// found digit by digit, 11, 11 and 10 bits: a histogram of the keys that share the digits
// so far, from its top down to where the budget ends.  Every key above it is kept, and of
// those equal to it the first ones.  The list comes out in order because a wave takes a run
// of tokens and knows from the runs before it how many it follows.
//
// Up to 65536 tokens a workgroup holds a sequence and head's keys in registers.  Longer ones are cut
// into slices, a workgroup each, and the digits found between launches.  Both are bound by their
// chains of counters, sums and barriers, not by the weights' bytes: 8 heads of 1000 tokens 9.3 us, 64 lists of
// up to 32768 tokens 22 us, 8 of 199999 tokens 37 us in four launches.
#include "layer_launch.h"
#include "rad_device.h"

namespace rad {
namespace {

__device__ __forceinline__ uint32_t key_of(float w) {
    const uint32_t u = __float_as_uint(w + 0.0f);             // -0 is 0
    if ((u & 0x7FFFFFFFu) > 0x7F800000u) return 0u;
    return u >> 31 ? ~u : u | 0x80000000u;
}

constexpr int kBins = 2048;
constexpr int kShift[3] = {21, 10, 0}, kBits[3] = {11, 11, 10};

// Sums over this lane and those above it.
__device__ __forceinline__ int wave_suffix(int v, int lane) {
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
        const int o = __shfl_down(v, d);
        v += lane + d < 64 ? o : 0;
    }
    return v;
}

// A (sequence, head)'s task: tokens lo .. hi - 1 compete for `need` places, those outside are kept.
struct Task {
    int L, n, lo, hi, need;
    int64_t pair;
    const float *w;
    __device__ __forceinline__ Task(const Kv4Select &s, int seq, int h)
        : L(min(max(s.seq_len[seq], 0), s.max_tokens)), n(min(L, s.budget)), lo(s.first), hi(L - s.recent),
          need(n - s.first - s.recent), pair(static_cast<int64_t>(seq) * s.heads + h), w(s.weight + pair * s.ldw) {}
    __device__ __forceinline__ bool competes(int t) const { return t >= lo && t < hi; }
};

// The keys of four tokens from t on (t a multiple of 4): 16 bytes, those past the sequence aside.
__device__ __forceinline__ uint4 keys4(const Task &k, int t) {
    const float4 w = t < k.L ? *reinterpret_cast<const float4 *>(k.w + t) : make_float4(0.f, 0.f, 0.f, 0.f);
    return make_uint4(key_of(w.x), key_of(w.y), key_of(w.z), key_of(w.w));
}

// found: digit d with as many keys in higher digits as `over` < rest <= over + its own, over, and its own, of C counts a digit
// (the lowest thread has the lowest digits); by a workgroup of W waves, 2048 / (64 W) digits a thread.
template <int W, class Count>
__device__ __forceinline__ void find_digit(int rest, int (&part)[W], int (&found)[3], Count count) {
    constexpr int N = kBins / (64 * W);
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    int c[N], all = 0;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        c[i] = count(N * tid + i);
        all += c[i];
    }
    const int sum = wave_suffix(all, lane);
    if (lane == 0) part[wave] = sum;
    if (tid == 0) found[0] = found[1] = found[2] = 0;
    __syncthreads();
    int over = sum - all;
    for (int x = wave + 1; x < W; ++x) over += part[x];
#pragma unroll
    for (int i = N - 1; i >= 0; --i) {
        if (rest > over && rest <= over + c[i]) found[0] = N * tid + i, found[1] = over, found[2] = c[i];
        over += c[i];
    }
    __syncthreads();
}

// A lane's tokens of four in a row: bit c of the low four where token t + c is kept whatever the ties, bit 4 + c
// where its key is the least one.
__device__ __forceinline__ uint32_t look4(const Task &k, int t, uint4 w, uint32_t least) {
    const uint32_t key[4] = {w.x, w.y, w.z, w.w};
    uint32_t m = 0;
#pragma unroll
    for (int c = 0; c < 4; ++c) {
        const bool free = k.competes(t + c);
        const bool up = t + c < k.L && (!free || (k.need > 0 && key[c] > least)), tie = free && k.need > 0 && key[c] == least;
        m |= (up ? 1u << c : 0u) | (tie ? 16u << c : 0u);
    }
    return m;
}
// How many of each kind, in the halves of a word (256 tokens a wave at most, so they stay apart).
__device__ __forceinline__ int counts(uint32_t m) { return __popc(m & 15u) | __popc(m >> 4) << 16; }

// The kept tokens among 256 in a row (four a lane), behind `ups` and `ties` of them that came before.
__device__ __forceinline__ void list256(const Kv4Select &s, const Task &k, int t, uint4 w, uint32_t least, int rest, int &ups, int &ties) {
    const uint32_t m = look4(k, t, w, least);
    const int mine = counts(m), sum = wave_scan(mine), all = __builtin_amdgcn_readlane(sum, 63);
    int u = ups + ((sum - mine) & 0xFFFF), e = ties + ((sum - mine) >> 16);
    if (m)
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            const bool up = m >> c & 1, tie = m >> (4 + c) & 1;
            if (up || (tie && e < rest)) {
                const int at = u + min(e, rest);
                s.kept[k.pair * s.budget + at] = t + c;
                if (s.kept_weight) s.kept_weight[k.pair * s.ld_kept + at] = k.w[t + c];
            }
            u += up;
            e += tie;
        }
    ups += all & 0xFFFF;
    ties += all >> 16;
}
// Their numbers alone, a lane's own.
__device__ __forceinline__ void count4(const Task &k, int t, uint4 w, uint32_t least, int &ups, int &ties) {
    const int c = counts(look4(k, t, w, least));
    ups += c & 0xFFFF;
    ties += c >> 16;
}

// ---- keys in registers ---------------------------------------------------------
//
// blockIdx.x: sequence * shares + share, blockIdx.y: head; 4 NV keys a thread, 4096 tokens in a row at a time.  Every
// share finds the least key, and lists its share of the tokens.  Weights crowd into few digits (a binade is four of them), so a digit has four counters, by lane; the
// keys that share the first digit are few and go on in LDS, where kHeldKeys hold them (32 us without).
constexpr int kSelWaves = 16, kRun = 256 * kSelWaves, kHeldKeys = 4096;
// A token's number, hidden from the compiler, which would keep what it once found out about each
// (whether it competes: 64 of them spilled 430 scalar registers).
__device__ __forceinline__ int anew(int t) {
    asm volatile("" : "+v"(t));
    return t;
}
template <int NV>
__global__ __launch_bounds__(64 * kSelWaves) void select_kernel(Kv4Select s, int shares) {
    constexpr int kCopies = NV == 1 ? 2 : 4, kBlocks = NV * kSelWaves;       // blocks of 256 tokens
    __shared__ int hist[kBins * kCopies];
    __shared__ uint32_t held[kHeldKeys];
    __shared__ int part[kSelWaves], found[3], n_held, ups_of[kBlocks], ties_of[kBlocks];
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int seq = blockIdx.x / shares, share = blockIdx.x % shares;
    const Task k(s, seq, blockIdx.y);
    if (share == 0 && blockIdx.y == 0 && tid == 0) s.count[seq] = k.n;
    if (k.L == k.n) {                                         // everything is kept
        for (int t = tid + 64 * kSelWaves * share; t < k.L; t += 64 * kSelWaves * shares) {
            s.kept[k.pair * s.budget + t] = t;
            if (s.kept_weight) s.kept_weight[k.pair * s.ld_kept + t] = k.w[t];
        }
        return;
    }
    const int t0 = 256 * wave + 4 * lane, runs = (k.L + kRun - 1) / kRun;
    uint4 w[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) w[i] = keys4(k, t0 + kRun * i);
    uint32_t least = 0, known = 0;
    int rest = k.need;
    bool few = false;                                         // the keys still in question are in `held`
    if (tid == 0) n_held = 0;
#pragma unroll
    for (int pass = 0; pass < 3; ++pass) {
        const int shift = kShift[pass], mask = (1 << kBits[pass]) - 1;
        for (int i = tid; i < (few ? kBins : kBins * kCopies); i += 64 * kSelWaves) hist[i] = 0;
        __syncthreads();
        if (few) {
            for (int i = tid; i < found[2]; i += 64 * kSelWaves)
                if ((held[i] & known) == least) atomicAdd(&hist[held[i] >> shift & mask], 1);
        } else if (rest > 0) {
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                if (i >= runs) continue;
                const uint32_t key[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
                const int t = anew(t0 + kRun * i);
#pragma unroll
                for (int c = 0; c < 4; ++c)
                    if (k.competes(t + c) && (key[c] & known) == least)
                        atomicAdd(&hist[(key[c] >> shift & mask) * kCopies + (lane & (kCopies - 1))], 1);
            }
        }
        const int before = few ? found[2] : 0;
        __syncthreads();
        find_digit<kSelWaves>(rest, part, found, [&](int d) {
            if (few) return hist[d];
            int c = 0;
#pragma unroll
            for (int x = 0; x < kCopies; x += 2) {
                const int2 a = *reinterpret_cast<const int2 *>(&hist[kCopies * d + x]);
                c += a.x + a.y;
            }
            return c;
        });
        least |= static_cast<uint32_t>(found[0]) << shift;
        known |= static_cast<uint32_t>(mask) << shift;
        rest -= found[1];
        const int same = found[2];
        __syncthreads();
        if (few) {
            if (tid == 0) found[2] = before;                  // the list stays as long as it is
        } else if (pass == 0 && rest > 0 && same <= kHeldKeys) {       // with no place left no digit was found: `same` counts nothing
            few = true;
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                if (i >= runs) continue;
                const uint32_t key[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
                const int t = anew(t0 + kRun * i);
#pragma unroll
                for (int c = 0; c < 4; ++c)
                    if (k.competes(t + c) && (key[c] & known) == least) held[atomicAdd(&n_held, 1)] = key[c];
            }
        }
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        if (i >= runs) continue;
        int ups = 0, ties = 0;
        count4(k, anew(t0 + kRun * i), w[i], least, ups, ties);
        const int sum = wave_scan(ups | ties << 16);
        if (lane == 63) {
            ups_of[i * kSelWaves + wave] = sum & 0xFFFF;
            ties_of[i * kSelWaves + wave] = sum >> 16;
        }
    }
    __syncthreads();
    if (wave == 0) {                                          // of the blocks before each
        int u[NV / 4 + 1], e[NV / 4 + 1], all_u = 0, all_e = 0;
        constexpr int N = (kBlocks + 63) / 64;
#pragma unroll
        for (int x = 0; x < N; ++x) {
            const int at = N * lane + x;
            u[x] = at < runs * kSelWaves ? ups_of[at] : 0;
            e[x] = at < runs * kSelWaves ? ties_of[at] : 0;
            all_u += u[x];
            all_e += e[x];
        }
        all_u = wave_scan(all_u) - all_u;
        all_e = wave_scan(all_e) - all_e;
#pragma unroll
        for (int x = 0; x < N; ++x) {
            const int at = N * lane + x;
            if (at < runs * kSelWaves) ups_of[at] = all_u, ties_of[at] = all_e;
            all_u += u[x];
            all_e += e[x];
        }
    }
    __syncthreads();
    const int i0 = runs * share / shares, i1 = runs * (share + 1) / shares;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        if (i < i0 || i >= i1) continue;
        int ups = ups_of[i * kSelWaves + wave], ties = ties_of[i * kSelWaves + wave];
        list256(s, k, anew(t0 + kRun * i), w[i], anew(least), rest, ups, ties);
    }
}

// ---- slices ----------------------------------------------------------------------
//
// blockIdx.x: sequence * slices + slice, blockIdx.y: head.  Launch p = 0 .. 2 counts the p-th digit of
// its slice's keys that share the digits found; launch 3 lists.  Each finds the digit before it from
// every slice's counts; slice 0 keeps it for the launches after that.  Of a slice's keys those above the
// digits found so far are counted on the way.
constexpr int kSliceWaves = 16, kSliceCopies = 4, kMostSlices = 64, kManySlices = 96;
struct Slices {
    int slices, each;                 // tokens a slice, a multiple of 256 * kSliceWaves
    int *hist;                        // [3][pairs][slices][kBins]
    int *above;                       // [2][pairs][slices]: keys above the first digit, above the second
    int *state;                       // [2][pairs][2]: digits found, places left among the keys that share them
    int64_t pairs;
};
template <int PASS>
__global__ __launch_bounds__(64 * kSliceWaves) void slice_kernel(Kv4Select s, Slices sl) {
    __shared__ int hist[PASS < 3 ? kBins * kSliceCopies : 1];
    __shared__ int part[kSliceWaves], found[3], sums[kSliceWaves][2];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, slice = blockIdx.x % sl.slices, seq = blockIdx.x / sl.slices;
    const Task k(s, seq, blockIdx.y);
    if (PASS == 0 && slice == 0 && blockIdx.y == 0 && tid == 0) s.count[seq] = k.n;
    const int t0 = slice * sl.each, t1 = min(t0 + sl.each, k.L);
    if (k.L == k.n) {                                         // everything is kept
        if (PASS == 3)
            for (int t = t0 + tid; t < t1; t += 64 * kSliceWaves) {
                s.kept[k.pair * s.budget + t] = t;
                if (s.kept_weight) s.kept_weight[k.pair * s.ld_kept + t] = k.w[t];
            }
        return;
    }
    // the first keys are asked for before the digits are looked for: PASS < 3 takes 4096 tokens at a time, the list
    // a run a wave
    constexpr int N = 4, kStep = PASS < 3 ? 4 * 64 * kSliceWaves : 256;
    const int run = sl.each / kSliceWaves, r0 = PASS < 3 ? t0 + 4 * tid : t0 + wave * run + 4 * lane;
    uint4 w[N];
    auto load = [&](int t) {
#pragma unroll
        for (int i = 0; i < N; ++i) w[i] = keys4(k, t + kStep * i);
    };
    load(r0);
    auto hists = [&](int pass) { return sl.hist + (static_cast<int64_t>(pass) * sl.pairs + k.pair) * sl.slices * kBins; };
    uint32_t least = 0, known = 0;
    int rest = k.need, ups = 0, ties = 0;                     // above and equal to the least key in the slices before
    if (PASS > 0) {
        if (PASS > 1) {
            const int *st = sl.state + ((PASS - 2) * sl.pairs + k.pair) * 2;
            least = static_cast<uint32_t>(st[0]);
            rest = st[1];
        }
        for (int p = 0; p < PASS; ++p) known |= ((1u << kBits[p]) - 1) << kShift[p];
        const int *from = hists(PASS - 1);
        constexpr int N = kBins / (64 * kSliceWaves);
        int c[N] = {}, cb[N] = {};                            // all slices' counts, those of the slices before
#pragma unroll 8
        for (int x = 0; x < sl.slices; ++x) {
            const bool before = PASS == 3 && x < slice;
#pragma unroll
            for (int i = 0; i < N; i += 2) {
                const int2 v = *reinterpret_cast<const int2 *>(from + static_cast<int64_t>(x) * kBins + N * tid + i);
                c[i] += v.x;
                c[i + 1] += v.y;
                if (PASS == 3) {
                    cb[i] += before ? v.x : 0;
                    cb[i + 1] += before ? v.y : 0;
                }
            }
        }
        find_digit<kSliceWaves>(rest, part, found, [&](int d) { return c[d % N]; });
        least |= static_cast<uint32_t>(found[0]) << kShift[PASS - 1];
        rest -= found[1];
        if (PASS == 3) {
#pragma unroll
            for (int i = 0; i < N; ++i) {
                ups += N * tid + i > found[0] ? cb[i] : 0;
                ties += N * tid + i == found[0] ? cb[i] : 0;
            }
        }
        if (PASS < 3) {
            if (slice == 0 && tid == 0) {
                int *st = sl.state + ((PASS - 1) * sl.pairs + k.pair) * 2;
                st[0] = static_cast<int>(least);
                st[1] = rest;
            }
            // this slice's keys above the digit
            int up = 0;
#pragma unroll
            for (int i = 0; i < N; ++i)
                if (N * tid + i > found[0]) up += from[static_cast<int64_t>(slice) * kBins + N * tid + i];
            up = wave_suffix(up, lane);
            if (lane == 0) sums[wave][0] = up;
            __syncthreads();
            if (tid == 0) {
                up = 0;
                for (int x = 0; x < kSliceWaves; ++x) up += sums[x][0];
                sl.above[((PASS - 1) * sl.pairs + k.pair) * sl.slices + slice] = up;
            }
        }
    }
    if constexpr (PASS < 3) {
        for (int i = tid; i < kBins * kSliceCopies; i += 64 * kSliceWaves) hist[i] = 0;
        __syncthreads();
        auto count = [&](int t, uint4 w4) {
            const uint32_t key[4] = {w4.x, w4.y, w4.z, w4.w};
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                if (t + c < t1 && k.competes(t + c) && (PASS == 0 || (key[c] & known) == least))
                    atomicAdd(&hist[(key[c] >> kShift[PASS] & ((1u << kBits[PASS]) - 1)) * kSliceCopies + (lane & (kSliceCopies - 1))], 1);
            }
        };
        if (rest > 0)
            for (int t = r0; t < t1; t += N * kStep) {
                if (t != r0) load(t);
#pragma unroll
                for (int i = 0; i < N; ++i) count(t + kStep * i, w[i]);
            }
        __syncthreads();
        int *to = hists(PASS) + static_cast<int64_t>(slice) * kBins;
        for (int d = tid; d < kBins; d += 64 * kSliceWaves) {
            const int4 a = *reinterpret_cast<const int4 *>(&hist[kSliceCopies * d]);
            to[d] = a.x + a.y + a.z + a.w;
        }
    } else {
        if (tid < slice) ups += sl.above[k.pair * sl.slices + tid] + sl.above[(sl.pairs + k.pair) * sl.slices + tid];
        ups = wave_suffix(ups, lane);
        ties = wave_suffix(ties, lane);
        if (lane == 0) sums[wave][0] = ups, sums[wave][1] = ties;
        __syncthreads();
        // before t0, tokens below lo and from hi on are kept whatever they weigh
        ups = min(t0, k.lo) + max(0, t0 - max(k.hi, k.lo));
        ties = 0;
        for (int x = 0; x < kSliceWaves; ++x) ups += sums[x][0], ties += sums[x][1];
        __syncthreads();
        const int r1 = min(t0 + (wave + 1) * run, t1);        // the end of the wave's run
        int u = 0, e = 0;
        for (int t = r0; t - 4 * lane < r1; t += N * kStep) {
            if (t != r0) load(t);
#pragma unroll
            for (int i = 0; i < N; ++i)
                if (t - 4 * lane + kStep * i < r1) count4(k, t + kStep * i, w[i], least, u, e);
        }
        u = wave_suffix(u, lane);
        e = wave_suffix(e, lane);
        if (lane == 0) sums[wave][0] = u, sums[wave][1] = e;
        __syncthreads();
        for (int x = 0; x < wave; ++x) ups += sums[x][0], ties += sums[x][1];
        const bool once = run <= N * kStep;                   // the run is still in registers
        for (int t = r0; t - 4 * lane < r1; t += N * kStep) {
            if (!once) load(t);
#pragma unroll
            for (int i = 0; i < N; ++i)
                if (t - 4 * lane + kStep * i < r1) list256(s, k, t + kStep * i, w[i], least, rest, ups, ties);
        }
    }
}

// Tokens of a slice whose list is still in registers when it is written; up to 1024 slices for all lists, as long as a list
// has no more than 96 of them, whose counts every slice adds up: else 64 longer ones (one list of 1300000 tokens 57 us
// in 80, 62 in 64, of 2 million 72 us in 123, 66 in 64, of 8 million 373 us in 489, 144 in 64; 8 lists of 2 million 250
// and 128).
constexpr int kSliceTokens = 16384;
// Tokens that a workgroup's registers hold; sequences that may be longer are cut into slices (8 lists of 65536 tokens 35 us
// held, 33 in slices; 64 of them 43 and 36, 256 of them 64 and 129; 8 of 40960 25 and 32).
constexpr int kMostHeld = 64 * kSelWaves * 4 * 16;

Slices make_slices(int64_t pairs, int64_t max_tokens, void *workspace) {
    constexpr int kUnit = 256 * kSliceWaves;
    Slices sl{};
    sl.pairs = pairs;
    const int64_t most = (max_tokens + kSliceTokens - 1) / kSliceTokens, want = pairs < 1024 ? 1024 / pairs : 1;
    const int64_t n = most < want && most <= kManySlices ? most : want < kMostSlices ? want : kMostSlices;
    const int64_t each = ((max_tokens + n - 1) / n + kUnit - 1) / kUnit * kUnit;
    sl.each = static_cast<int>(each);
    sl.slices = static_cast<int>((max_tokens + each - 1) / each);
    sl.hist = static_cast<int *>(workspace);
    sl.above = sl.hist ? sl.hist + 3 * pairs * sl.slices * kBins : nullptr;
    sl.state = sl.above ? sl.above + 2 * pairs * sl.slices : nullptr;
    return sl;
}

}  // namespace

int64_t kv4_select_workspace(int64_t B, int64_t heads, int64_t max_tokens) {
    if (max_tokens <= kMostHeld) return 0;
    const Slices sl = make_slices(B * heads, max_tokens, nullptr);
    return 4 * (sl.pairs * sl.slices * (3 * kBins + 2) + 4 * sl.pairs);
}

hipError_t launch_kv4_select(const Kv4Select &s, void *workspace, hipStream_t st) {
    if (s.max_tokens <= kMostHeld) {
        const int64_t pairs = static_cast<int64_t>(s.B) * s.heads;
        // As many shares as find a CU of their own (lists of 32768: 8 of them 28 us with one share, 24 with two, 22 with
        // four, 80 of them 29, 25 and 46, 136 of them 29, 49 and 69).  A list's registers go by its room, in rungs
        // (8 lists of 32768 tokens 22 us with 40 keys a thread, 23.5 with 64; 32 keys would serve 32768 in 21.7 and
        // leave 40960, 25.5, to 64, 26.9).
        const int shares = s.max_tokens <= 4096 || pairs > 128 ? 1 : pairs > 64 ? 2 : 4;
        auto go = [&](auto kernel) { hipLaunchKernelGGL(kernel, dim3(s.B * shares, s.heads), dim3(64 * kSelWaves), 0, st, s, shares); };
        if (s.max_tokens <= 4096) go(select_kernel<1>);
        else if (s.max_tokens <= 16384) go(select_kernel<4>);
        else if (s.max_tokens <= 32768 + 8192) go(select_kernel<10>);
        else go(select_kernel<16>);
        return hipGetLastError();
    }
    const Slices sl = make_slices(static_cast<int64_t>(s.B) * s.heads, s.max_tokens, workspace);
    auto go = [&](auto kernel) {
        hipLaunchKernelGGL(kernel, dim3(static_cast<uint32_t>(s.B) * sl.slices, s.heads), dim3(64 * kSliceWaves), 0, st, s, sl);
        return hipGetLastError();
    };
    if (hipError_t e = go(slice_kernel<0>); e != hipSuccess) return e;
    if (hipError_t e = go(slice_kernel<1>); e != hipSuccess) return e;
    if (hipError_t e = go(slice_kernel<2>); e != hipSuccess) return e;
    return go(slice_kernel<3>);
}

}  // namespace rad
