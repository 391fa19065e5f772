// layer_api.hip -- the C ABI of the calls between a layer's linears (declared
// in include/rad.h).  As in rad_api.hip every argument is checked on the host
// before any HIP call: types -> shapes -> ranges -> (empty: done) -> pointers
// -> alignment -> aliasing.
#include "layer_launch.h"
#include "rad_check.h"

namespace {

int dtype_bytes(int32_t dtype) {
    if (dtype == RAD_DT_F32) return 4;
    if (dtype == RAD_DT_BF16 || dtype == RAD_DT_F16) return 2;
    return 0;
}

constexpr int64_t kMaxRows = int64_t(1) << 22, kMaxTokens = int64_t(1) << 30;
// A launch holds fewer than 2^32 threads: one for every eight values read back, and of the norm up to 256 a
// token for K <= 2048, 64 for every 1024 values (1024 at most) for longer ones (norm_quant.hip, many tokens).
constexpr int64_t kMaxNormRows = int64_t(1) << 24, kMaxRead = (int64_t(1) << 35) - 2048, kMaxThreads = int64_t(1) << 32;
int64_t norm_threads(int64_t K) { return K <= 2048 ? 256 : K <= 16384 ? 64 * ((K + 1023) / 1024) : 1024; }

// Shape and range of a cache descriptor (no pointers).
int check_cache(const rad_kv4_cache *c) {
    if (!c) return RAD_E_NULL;
    if (c->D != 64 && c->D != 128 && c->D != 256) return RAD_E_SHAPE;
    if (c->page_size != 32 && c->page_size != 64 && c->page_size != 128 && c->page_size != 256) return RAD_E_SHAPE;
    if (c->pages < 1 || c->heads < 1) return RAD_E_SHAPE;
    if (c->pages > kI32Max || c->heads > 1024) return RAD_E_RANGE;
    return RAD_OK;
}

// Shape and range of a batch; 1 when it is empty.
int check_batch(const rad_kv4_cache *c, const rad_kv_batch *b) {
    if (!b) return RAD_E_NULL;
    if (b->B < 0 || b->rows < 0 || b->max_pages < 0 || b->max_q < 0) return RAD_E_SHAPE;
    if (b->B >= kMaxRows || b->rows >= kMaxRows || b->max_pages > kI32Max ||
        b->max_pages * c->page_size >= kMaxTokens)
        return RAD_E_RANGE;
    if (b->B == 0 || b->rows == 0) return 1;
    if (!b->q_start && b->rows != b->B) return RAD_E_SHAPE;
    return RAD_OK;
}

int64_t code_bytes4(const rad_kv4_cache *c) { return c->pages * c->heads * c->page_size * (c->D / 2); }
int64_t scale_bytes4(const rad_kv4_cache *c) { return c->pages * c->heads * c->page_size * 2; }

int check_pointers(const rad_kv4_cache *c, const rad_kv_batch *b) {
    if (!c->k_codes || !c->k_scale || !c->v_codes || !c->v_scale || !b->seq_len) return RAD_E_NULL;
    if (b->max_pages > 0 && !b->block_table) return RAD_E_NULL;
    if (!aligned(c->k_codes, 16) || !aligned(c->k_scale, 16) || !aligned(c->v_codes, 16) || !aligned(c->v_scale, 16) ||
        !aligned(b->block_table, 4) || !aligned(b->seq_len, 4) || !aligned(b->q_start, 4))
        return RAD_E_ALIGN;
    return RAD_OK;
}

// The cache's four arrays and the batch's three.
struct Spans {
    Span cache[4], batch[3];
    Spans(const rad_kv4_cache *c, const rad_kv_batch *b)
        : cache{span(c->k_codes, code_bytes4(c)), span(c->k_scale, scale_bytes4(c)), span(c->v_codes, code_bytes4(c)),
                span(c->v_scale, scale_bytes4(c))},
          batch{span(b->block_table, b->B * b->max_pages * 4), span(b->seq_len, b->B * 4),
                b->q_start ? span(b->q_start, (b->B + 1) * 4) : Span{0, 0}} {}
    bool meets_cache(Span s) const {
        for (const Span &x : cache)
            if (overlap(x, s)) return true;
        return false;
    }
    bool meets(Span s) const {
        for (const Span &x : batch)
            if (overlap(x, s)) return true;
        return meets_cache(s);
    }
};

int page_shift(const rad_kv4_cache *c) { return __builtin_ctzll(static_cast<uint64_t>(c->page_size)); }
rad::Kv4Cache cache_args(const rad_kv4_cache *c) {
    return rad::Kv4Cache{c->k_codes, c->v_codes, c->k_scale, c->v_scale, static_cast<int>(c->pages),
                         static_cast<int>(c->heads), page_shift(c), static_cast<int>(c->D)};
}
rad::KvBatch batch_args(const rad_kv4_cache *c, const rad_kv_batch *b) {
    const int64_t most = b->q_start ? (b->max_q < b->rows ? b->max_q : b->rows) : 1;
    return rad::KvBatch{b->block_table, b->seq_len, b->q_start, static_cast<int>(b->B),
                        static_cast<int>(b->max_pages), static_cast<int>(b->rows), static_cast<int>(most), page_shift(c)};
}

}  // namespace

extern "C" {

int rad_add_rmsnorm_quant_i8(const void *x, const void *residual, void *residual_out, const float *gamma, float eps,
                             int8_t *q, float *scale, int64_t M, int64_t K, int32_t dtype, int rotate,
                             rad_stream_t stream) {
    const int e = dtype_bytes(dtype);
    if (e == 0) return RAD_E_FMT;
    if (M < 0 || K <= 0 || K % 128 != 0) return RAD_E_SHAPE;
    if (K > RAD_QUANT_MAX_K || M >= kMaxNormRows || M * norm_threads(K) >= kMaxThreads || (rotate != 0 && rotate != 1)) return RAD_E_RANGE;
    if (!(eps >= 0.0f) || eps > 3.0e38f) return RAD_E_RANGE;
    if ((residual == nullptr) != (residual_out == nullptr)) return RAD_E_NULL;
    if (M == 0) return RAD_OK;
    if (!x || !gamma || !q || !scale) return RAD_E_NULL;
    if (!aligned(x, 16) || !aligned(residual, 16) || !aligned(residual_out, 16) || !aligned(gamma, 16) ||
        !aligned(q, 16) || !aligned(scale, 4))
        return RAD_E_ALIGN;
    const int64_t n = M * K;
    const Span none{0, 0}, in[] = {span(x, n * e), span(gamma, K * 4), residual ? span(residual, n * e) : none};
    const Span out[] = {residual_out && residual_out != residual ? span(residual_out, n * e) : none, span(q, n),
                        span(scale, M * 4)};
    for (const Span &o : out)
        for (const Span &i : in)
            if (overlap(o, i)) return RAD_E_ALIAS;
    if (overlap(out[0], out[1]) || overlap(out[0], out[2]) || overlap(out[1], out[2])) return RAD_E_ALIAS;
    // in place: the residual may meet neither x nor gamma
    if (residual && (overlap(in[0], in[2]) || overlap(in[1], in[2])) && residual_out == residual) return RAD_E_ALIAS;
    return hip_status(rad::launch_norm_quant(x, residual, residual_out, gamma, eps, q, scale, M,
                                             static_cast<int>(K), dtype, rotate, static_cast<hipStream_t>(stream)));
}

int rad_kv4_append(const rad_kv4_cache *cache, const rad_kv_batch *batch, const void *k, int64_t ldk, const void *v,
                   int64_t ldv, const void *q, int64_t ldq, int64_t q_heads, void *q_out, const rad_rope *rope,
                   int rotate, int32_t dtype, rad_stream_t stream) {
    const int e = dtype_bytes(dtype);
    if (e == 0) return RAD_E_FMT;
    int rc = check_cache(cache);
    if (rc != RAD_OK) return rc;
    const int empty = check_batch(cache, batch);
    if (empty < 0) return empty;
    const int64_t D = cache->D, H = cache->heads;
    if (rotate != 0 && rotate != 1) return RAD_E_RANGE;
    if (rotate && D % 128 != 0) return RAD_E_SHAPE;
    if (ldk < H * D || ldv < H * D || q_heads < 0 || ldq < q_heads * D) return RAD_E_SHAPE;
    if (q_heads > 16384 || ldk > kI32Max || ldv > kI32Max || ldq > kI32Max) return RAD_E_RANGE;
    if (rope) {
        if (rope->dim < 8 || rope->dim > D || rope->dim % 8 != 0 || rope->rows < 0) return RAD_E_SHAPE;
        if ((rope->style != 0 && rope->style != 1) || rope->rows > kI32Max) return RAD_E_RANGE;
    }
    if (empty) return RAD_OK;
    if ((q_heads > 0) != (q != nullptr) || (q != nullptr) != (q_out != nullptr)) return RAD_E_NULL;
    rc = check_pointers(cache, batch);
    if (rc != RAD_OK) return rc;
    if (!k || !v || (rope && !rope->table)) return RAD_E_NULL;
    if (!aligned(k, 16) || !aligned(v, 16) || !aligned(q, 16) || !aligned(q_out, 16) || (ldk * e) % 16 != 0 ||
        (ldv * e) % 16 != 0 || (ldq * e) % 16 != 0 || (rope && !aligned(rope->table, 16)))
        return RAD_E_ALIGN;
    const int64_t T = batch->rows, n = H * D;
    const Span none{0, 0}, in[] = {span(k, ((T - 1) * ldk + n) * e), span(v, ((T - 1) * ldv + n) * e),
                                   q ? span(q, ((T - 1) * ldq + q_heads * D) * e) : none,
                                   rope ? span(rope->table, rope->rows * rope->dim * 4) : none};
    const Span qo = q ? span(q_out, T * q_heads * D * e) : none;
    const Spans sp(cache, batch);
    for (const Span &i : in)
        if (overlap(qo, i) || sp.meets_cache(i)) return RAD_E_ALIAS;
    for (const Span &i : sp.batch)
        if (sp.meets_cache(i)) return RAD_E_ALIAS;
    for (int i = 0; i < 4; ++i)
        for (int j = 0; j < i; ++j)
            if (overlap(sp.cache[i], sp.cache[j])) return RAD_E_ALIAS;
    if (sp.meets(qo)) return RAD_E_ALIAS;
    const rad::Kv4New nw{q, k, v, ldq, ldk, ldv, static_cast<int>(q_heads), q_out,
                         rope ? rope->table : nullptr, rope ? rope->rows : 0, rope ? rope->dim : 0,
                         rope ? rope->style : 0, rotate};
    return hip_status(rad::launch_kv4_append(cache_args(cache), batch_args(cache, batch), nw, dtype,
                                             static_cast<hipStream_t>(stream)));
}

int rad_kv4_read(const rad_kv4_cache *cache, const rad_kv_batch *batch, uint16_t *k_out, uint16_t *v_out,
                 rad_stream_t stream) {
    int rc = check_cache(cache);
    if (rc != RAD_OK) return rc;
    const int empty = check_batch(cache, batch);
    if (empty < 0) return empty;
    if (batch->rows * cache->heads * cache->D > kMaxRead) return RAD_E_RANGE;
    if (empty) return RAD_OK;
    rc = check_pointers(cache, batch);
    if (rc != RAD_OK) return rc;
    if (!k_out || !v_out) return RAD_E_NULL;
    if (!aligned(k_out, 16) || !aligned(v_out, 16)) return RAD_E_ALIGN;
    const int64_t bytes = batch->rows * cache->heads * cache->D * 2;
    const Span ks = span(k_out, bytes), vs = span(v_out, bytes);
    const Spans sp(cache, batch);
    if (overlap(ks, vs) || sp.meets(ks) || sp.meets(vs)) return RAD_E_ALIAS;
    return hip_status(rad::launch_kv4_read(cache_args(cache), batch_args(cache, batch), k_out, v_out,
                                           static_cast<hipStream_t>(stream)));
}

}  // extern "C"

namespace {
// Sizes that the attention call and its workspace call share; 1 when there is no row to attend for.
int check_attn(const rad_kv4_cache *c, const rad_kv_batch *b, int64_t q_heads, int32_t dtype) {
    if (dtype_bytes(dtype) == 0) return RAD_E_FMT;
    const int rc = check_cache(c);
    if (rc != RAD_OK) return rc;
    const int empty = check_batch(c, b);
    if (empty < 0) return empty;
    if (q_heads < 1 || q_heads % c->heads != 0) return RAD_E_SHAPE;
    if (q_heads > 16384 || b->rows * q_heads >= (int64_t(1) << 29)) return RAD_E_RANGE;
    if (empty || (b->q_start && b->max_q == 0)) return 1;
    return rad::kv4_attn_fits(cache_args(c), batch_args(c, b), static_cast<int>(q_heads)) ? RAD_OK : RAD_E_RANGE;
}
}  // namespace

extern "C" {

int rad_attn_kv4_workspace(const rad_kv4_cache *cache, const rad_kv_batch *batch, int64_t q_heads, int32_t dtype,
                           int64_t *bytes) {
    const int rc = check_attn(cache, batch, q_heads, dtype);
    if (rc < 0) return rc;
    if (!bytes) return RAD_E_NULL;
    *bytes = rc ? 0
                : rad::kv4_attn_workspace(cache_args(cache), batch_args(cache, batch), static_cast<int>(q_heads), dtype);
    return RAD_OK;
}

int rad_attn_kv4(const rad_kv4_cache *cache, const rad_kv_batch *batch, const void *q, int64_t q_heads, float sm_scale,
                 int causal, int64_t window, void *o, void *workspace, int64_t workspace_bytes, int32_t dtype,
                 rad_stream_t stream) {
    int rc = check_attn(cache, batch, q_heads, dtype);
    if (rc < 0) return rc;
    const bool empty = rc > 0;
    if (!(sm_scale > 0.0f) || sm_scale > 0x1p126f || (causal != 0 && causal != 1)) return RAD_E_RANGE;
    if (window < 0) return RAD_E_SHAPE;
    if (empty) return RAD_OK;
    const rad::Kv4Cache ca = cache_args(cache);
    const rad::KvBatch ba = batch_args(cache, batch);
    const int64_t need = rad::kv4_attn_workspace(ca, ba, static_cast<int>(q_heads), dtype);
    if (workspace_bytes < need) return RAD_E_RANGE;
    rc = check_pointers(cache, batch);
    if (rc != RAD_OK) return rc;
    if (!q || !o || (need > 0 && !workspace)) return RAD_E_NULL;
    if (!aligned(q, 16) || !aligned(o, 16) || !aligned(workspace, 16)) return RAD_E_ALIGN;
    const int64_t bytes = batch->rows * q_heads * cache->D * dtype_bytes(dtype);
    const Span qs = span(q, bytes), os = span(o, bytes), ws = need > 0 ? span(workspace, need) : Span{0, 0};
    const Spans sp(cache, batch);
    if (overlap(os, qs) || overlap(ws, qs) || overlap(ws, os) || sp.meets(os) || sp.meets(ws)) return RAD_E_ALIAS;
    const int win = window > 0 && window < kMaxTokens ? static_cast<int>(window) : 0;
    const rad::Kv4Attn at{q, o, static_cast<int>(q_heads), sm_scale, causal, win, workspace};
    return hip_status(rad::launch_kv4_attn(ca, ba, at, dtype, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
