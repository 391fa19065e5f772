// kv4_move.hip -- cached tokens to other places of the paged 4-bit cache (gfx950).
//
// Values lie in octets of tokens (a dword = one dimension of eight tokens), so a wave
// makes an octet of targets: for its eight entries it reads their keys' codes (D/2
// bytes each, D bytes a lane group), their scales, and of each entry's octet of values the
// dwords of its own dimensions, D/64 a lane, from which it takes a nibble each.  Octets
// that the list fills only partly are merged with what is there.
//
// Bound by the trips to memory of an octet (list, page, codes, a scale of two bytes from each of 16 lines) more than
// by bytes: 8 sequences' 4096 of 13000 tokens (8 heads of 128) take 32 us for 44 MB fetched and 35 MB written; the
// loads of the eight entries one behind the other took 41 us, several octets a wave with the next one's places
// looked up ahead the same 32.  16384 of 199999 tokens 19 us, 256 of 1000 3.2 us; in place 8 paths of 8 of 60
// drafted tokens 3.4 us.
//
// Into pages of their own the octets are independent.  In place a workgroup has all
// of a sequence and head's octets (at most 33): it reads them all, meets, and writes.
#include "kv4.h"

namespace rad {
namespace {

// What a wave holds of an octet of targets.
template <int D>
struct Octet {
    uint2 key[D / 128 > 0 ? D / 128 : 1];     // entry lane / 8: D / 16 bytes from D / 16 * (lane % 8)
    uint32_t value[D / 64];                   // dims D / 64 * lane ..
    uint32_t mask;                            // nibbles of entries that move
    uint32_t scales;                          // lane < 8: entry lane's key and value scale
};


// The source of entry i of the list (all lanes may ask for different ones).
__device__ __forceinline__ int64_t source_of(const Kv4Cache &c, const KvBatch &b, const int32_t *list, int seq, int h, int len, int i, int n) {
    if (i < 0 || i >= n) return -1;
    const int t = list[i];
    if (t < 0 || t >= len) return -1;
    const int page = kv_page(b, seq, t, c.pages);
    return page < 0 ? -1 : ((static_cast<int64_t>(page) * c.heads + h) << c.page_shift) + (t & ((1 << c.page_shift) - 1));
}

__device__ __forceinline__ int64_t lane_of(int64_t v, int lane) {
    return static_cast<uint32_t>(__builtin_amdgcn_readlane(static_cast<int>(v), lane)) |
           static_cast<int64_t>(__builtin_amdgcn_readlane(static_cast<int>(v >> 32), lane)) << 32;
}
template <int D>
__device__ __forceinline__ void read_octet(Octet<D> &o, const Kv4Cache &c, const KvBatch &b, const int32_t *list, int seq, int h, int len, int i0, int n) {
    constexpr int KB = D / 16, NV = D / 64;                   // bytes of a key and dwords of values a lane
    const int lane = threadIdx.x & 63;
    const int64_t mine = source_of(c, b, list, seq, h, len, i0 + (lane & 7), n);
    const uint64_t moves = __ballot(mine >= 0);
    o.mask = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) o.mask |= moves >> j & 1 ? 15u << (4 * j) : 0u;
    o.scales = 0;
    if (lane < 8 && mine >= 0) o.scales = c.k_scale[mine] | static_cast<uint32_t>(c.v_scale[mine]) << 16;
    if (moves == 0) return;
    // entries that do not move read another's, so that every load is under way before the first is waited for
    const int64_t some = lane_of(mine, __builtin_ctzll(moves)), ke = __shfl(mine, lane >> 3);
    const uint8_t *p = c.k_codes + (ke >= 0 ? ke : some) * (D / 2) + KB * (lane & 7);
    if constexpr (D == 64) o.key[0].x = *reinterpret_cast<const uint32_t *>(p);
    else {
#pragma unroll
        for (int x = 0; x < D / 128; ++x) o.key[x] = reinterpret_cast<const uint2 *>(p)[x];
    }
    uint32_t v[8][NV];
    int shift[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const int64_t ve = moves >> j & 1 ? lane_of(mine, j) : some;
        const uint32_t *q = reinterpret_cast<const uint32_t *>(c.v_codes) + (ve >> 3) * D + NV * lane;
        shift[j] = 4 * static_cast<int>(ve & 7);
#pragma unroll
        for (int x = 0; x < NV; ++x) v[j][x] = q[x];
    }
#pragma unroll
    for (int x = 0; x < NV; ++x) {
        o.value[x] = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) o.value[x] |= ((v[j][x] >> shift[j]) & 15u) << (4 * j);
        o.value[x] &= o.mask;
    }
}

// Targets: tokens 8 * octet .. of the sequence's target pages.
template <int D>
__device__ __forceinline__ void write_octet(const Octet<D> &o, const Kv4Cache &to, int page, int h, int octet) {
    constexpr int KB = D / 16, NV = D / 64;
    if (o.mask == 0 || page < 0 || page >= to.pages) return;
    const int lane = threadIdx.x & 63;
    const int64_t vec = ((static_cast<int64_t>(page) * to.heads + h) << to.page_shift) + ((8 * octet) & ((1 << to.page_shift) - 1));
    if (lane < 8 && (o.mask >> (4 * lane) & 1)) {
        to.k_scale[vec + lane] = static_cast<uint16_t>(o.scales);
        to.v_scale[vec + lane] = static_cast<uint16_t>(o.scales >> 16);
    }
    const int e = lane >> 3;
    if (o.mask >> (4 * e) & 1) {
        uint8_t *p = to.k_codes + (vec + e) * (D / 2) + KB * (lane & 7);
        if constexpr (D == 64) *reinterpret_cast<uint32_t *>(p) = o.key[0].x;
        else {
#pragma unroll
            for (int x = 0; x < D / 128; ++x) reinterpret_cast<uint2 *>(p)[x] = o.key[x];
        }
    }
    uint32_t *q = reinterpret_cast<uint32_t *>(to.v_codes) + (vec >> 3) * D + NV * lane;
#pragma unroll
    for (int x = 0; x < NV; ++x) q[x] = o.mask == 0xFFFFFFFFu ? o.value[x] : (q[x] & ~o.mask) | o.value[x];
}

constexpr int kFar = (1 << 30) - 16, kBefore = -(1 << 30);   // past every table's last octet, and before any entry's token
struct List {
    const int32_t *list;
    int len, n, start;
    __device__ __forceinline__ List(const KvBatch &b, const Kv4Move &m, int seq, int h)
        : list(m.from + (static_cast<int64_t>(seq) * m.lists + (m.lists == 1 ? 0 : h)) * m.entries), len(kv_len(b, seq)),
          n(min(max(m.count[seq], 0), m.entries)),
          start(m.to_start ? min(max(m.to_start[seq], kBefore), kFar) : 0) {}      // no token lies that far: sums stay in 32 bits
};
// Page of the octet's targets, or -1.
__device__ __forceinline__ int target_page(const int32_t *table, int pages, int shift, int octet) {
    if (octet < 0) return -1;
    const int p = static_cast<int>((static_cast<int64_t>(octet) * 8) >> shift);
    return p < pages ? table[p] : -1;
}

// blockIdx.x: sequence * parts + part, blockIdx.y: head.  Wave w of a part takes octets 4 part + w, 4 (part + parts) + w, ..
template <int D>
__global__ __launch_bounds__(256) void move_kernel(Kv4Cache c, KvBatch b, Kv4Cache to, Kv4Move m, int parts) {
    const int seq = blockIdx.x / parts, part = blockIdx.x % parts, h = blockIdx.y, wave = threadIdx.x >> 6;
    const List l(b, m, seq, h);
    const int first = l.start >> 3, octets = l.n > 0 ? ((l.start + l.n + 7) >> 3) - first : 0;
    for (int x = 4 * part + wave; x < octets; x += 4 * parts) {
        Octet<D> o{};
        read_octet<D>(o, c, b, l.list, seq, h, l.len, 8 * (first + x) - l.start, l.n);
        write_octet<D>(o, to, target_page(m.to_table + static_cast<int64_t>(seq) * m.to_pages, m.to_pages, to.page_shift, first + x), h, first + x);
    }
}

// In place: blockIdx.x sequence, blockIdx.y head; wave w holds octets w, 12 + w, 24 + w.
constexpr int kInPlaceWaves = 12;
template <int D>
__global__ __launch_bounds__(64 * kInPlaceWaves) void move_in_place_kernel(Kv4Cache c, KvBatch b, Kv4Move m) {
    constexpr int N = 3;
    const int seq = blockIdx.x, h = blockIdx.y, wave = threadIdx.x >> 6;
    const List l(b, m, seq, h);
    const int first = l.start >> 3, octets = l.n > 0 ? ((l.start + l.n + 7) >> 3) - first : 0;
    Octet<D> o[N] = {};
#pragma unroll
    for (int k = 0; k < N; ++k) {
        const int x = wave + kInPlaceWaves * k;
        if (x < octets) read_octet<D>(o[k], c, b, l.list, seq, h, l.len, 8 * (first + x) - l.start, l.n);
    }
    // every wave's reads have come back before any wave writes
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    __syncthreads();
#pragma unroll
    for (int k = 0; k < N; ++k) {
        const int x = wave + kInPlaceWaves * k;
        if (x < octets)
            write_octet<D>(o[k], c, target_page(b.block_table + static_cast<int64_t>(seq) * b.max_pages, b.max_pages, c.page_shift, first + x), h, first + x);
    }
}

template <int D>
hipError_t launch_d(const Kv4Cache &c, const KvBatch &b, const Kv4Cache &to, const Kv4Move &m, hipStream_t st) {
    if (!m.to_table) {
        hipLaunchKernelGGL(move_in_place_kernel<D>, dim3(b.B, c.heads), dim3(64 * kInPlaceWaves), 0, st, c, b, m);
        return hipGetLastError();
    }
    const int64_t all = static_cast<int64_t>(b.B) * c.heads, most = (static_cast<int64_t>(m.entries) + 8 + 31) / 32, even = 16384 / all;
    const int parts = static_cast<int>(even < 1 ? 1 : even < most ? even : most);
    hipLaunchKernelGGL(move_kernel<D>, dim3(static_cast<uint32_t>(b.B) * parts, c.heads), dim3(256), 0, st, c, b, to, m, parts);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_kv4_move(const Kv4Cache &c, const KvBatch &b, const Kv4Cache &to, const Kv4Move &m, hipStream_t st) {
    if (c.D == 64) return launch_d<64>(c, b, to, m, st);
    if (c.D == 128) return launch_d<128>(c, b, to, m, st);
    return launch_d<256>(c, b, to, m, st);
}

}  // namespace rad
