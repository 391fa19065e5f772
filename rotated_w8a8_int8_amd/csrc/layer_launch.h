// layer_launch.h -- host-side launchers of the kernels between the linears of
// a layer: the norm that feeds them, the paged 4-bit cache and its attention.
// Arguments are already validated by layer_api.hip.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace rad {

hipError_t launch_norm_quant(const void *x, const void *res, void *res_out, const float *gamma, float eps,
                             int8_t *q, float *scale, int64_t M, int K, int dtype, int rotate, hipStream_t st);

// The paged cache and the ragged batch (include/rad.h), with the page size as a shift.
struct Kv4Cache {
    uint8_t *k_codes, *v_codes;
    uint16_t *k_scale, *v_scale;
    int pages, heads, page_shift, D;
};
struct KvBatch {
    const int32_t *block_table, *seq_len, *q_start;
    int B, max_pages, rows, max_q, page_shift;
};
// With cache and batch 192 bytes, three lines of the memory that a kernel's arguments are fetched from.
struct Kv4New {
    const void *q, *k, *v;
    int64_t ldq, ldk, ldv;
    int q_heads, rope_rows;
    void *q_out;
    const float *rope;
    int rope_dim, rope_style, rotate;
    const int32_t *position;     // angles of each row, or null: by its place in the cache
};

hipError_t launch_kv4_append(const Kv4Cache &c, const KvBatch &b, const Kv4New &n, int dtype, hipStream_t st);
hipError_t launch_kv4_read(const Kv4Cache &c, const KvBatch &b, uint16_t *k, uint16_t *v, hipStream_t st);

// With the other arguments of its kernels 192 bytes, three lines of the memory that they are fetched from: a fourth
// cost a decoded token's call 0.16 us of 9.7.
struct Kv4Attn {
    const void *q;
    void *o;
    int q_heads;
    float sm_scale;
    int causal, window;      // causal: of trees the words of a row's mask; window 0: none
    union {
        float2 *stats;           // [rows][q_heads]: reference exponent, 1 / normaliser (0: sees nothing); or null
        const uint64_t *mask;    // trees: [rows][words]
    };
    __host__ __device__ int words() const { return causal; }
};
bool kv4_attn_fits(const Kv4Cache &c, const KvBatch &b, int q_heads);     // one launch holds the call
int64_t kv4_attn_workspace(const Kv4Cache &c, const KvBatch &b, int q_heads, int dtype);
hipError_t launch_kv4_attn(const Kv4Cache &c, const KvBatch &b, const Kv4Attn &a, void *workspace, int dtype, hipStream_t st);
hipError_t launch_kv4_attn_tree(const Kv4Cache &c, const KvBatch &b, const Kv4Attn &a, void *workspace, int dtype, hipStream_t st);

// Attention weights of the cached tokens, from the rows' statistics (Kv4Attn::stats).
struct Kv4Weights {
    float *weight;
    int64_t ldw;
    int observe;             // last rows that count; 0: all
    float factor;
    void *pairs;             // queries made ready, where a call has many (kv4_weights_workspace)
};
int64_t kv4_weights_workspace(const Kv4Cache &c, const KvBatch &b, int q_heads, int dtype);
hipError_t launch_kv4_weights(const Kv4Cache &c, const KvBatch &b, const Kv4Attn &a, const Kv4Weights &w, int dtype, hipStream_t st);

struct Kv4Select {
    const float *weight;
    int64_t ldw;
    const int32_t *seq_len;
    int B, heads, max_tokens, budget, first, recent;
    int32_t *kept, *count;
    float *kept_weight;
    int64_t ld_kept;
};
int64_t kv4_select_workspace(int64_t B, int64_t heads, int64_t max_tokens);
hipError_t launch_kv4_select(const Kv4Select &s, void *workspace, hipStream_t st);

struct Kv4Move {
    const int32_t *from, *count, *to_table, *to_start;
    int lists, entries, to_pages;      // to_table null: in place
};
hipError_t launch_kv4_move(const Kv4Cache &c, const KvBatch &b, const Kv4Cache &to, const Kv4Move &m, hipStream_t st);

// Linear attention (include/rad.h, rad_linear).
struct Linear {
    const void *q, *k, *v;
    int64_t ldq, ldk, ldv;
    const float *log_decay;
    const int32_t *q_start;
    int B, rows, max_q, qk_heads, heads, D;
    const float *state;
    float *state_out;
    float scale;
    void *o;
};
bool linear_fits(const Linear &l, int dtype);      // one launch holds the call
int64_t linear_workspace(const Linear &l, int dtype);
hipError_t launch_linear(const Linear &l, int dtype, void *workspace, hipStream_t st);

}  // namespace rad
