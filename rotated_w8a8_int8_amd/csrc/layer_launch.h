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
struct Kv4New {
    const void *q, *k, *v;
    int64_t ldq, ldk, ldv;
    int q_heads;
    void *q_out;
    const float *rope;
    int64_t rope_rows;
    int rope_dim, rope_style, rotate;
};

hipError_t launch_kv4_append(const Kv4Cache &c, const KvBatch &b, const Kv4New &n, int dtype, hipStream_t st);
hipError_t launch_kv4_read(const Kv4Cache &c, const KvBatch &b, uint16_t *k, uint16_t *v, hipStream_t st);

struct Kv4Attn {
    const void *q;
    void *o;
    int q_heads;
    float sm_scale;
    int causal, window;      // window 0: none
    void *workspace;
};
bool kv4_attn_fits(const Kv4Cache &c, const KvBatch &b, int q_heads);     // one launch holds the call
int64_t kv4_attn_workspace(const Kv4Cache &c, const KvBatch &b, int q_heads, int dtype);
hipError_t launch_kv4_attn(const Kv4Cache &c, const KvBatch &b, const Kv4Attn &a, int dtype, hipStream_t st);

}  // namespace rad
