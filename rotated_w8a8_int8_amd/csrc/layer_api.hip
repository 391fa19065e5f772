// layer_api.hip -- the C ABI of the calls between a layer's linears (declared
// in include/rad.h).  As in rad_api.hip every argument is checked on the host
// before any HIP call: types -> shapes -> ranges -> (empty: done) -> pointers
// -> alignment -> aliasing.
#include <math.h>

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

int append(const rad_kv4_cache *cache, const rad_kv_batch *batch, const void *k, int64_t ldk, const void *v, int64_t ldv,
           const void *q, int64_t ldq, int64_t q_heads, void *q_out, const rad_rope *rope, const int32_t *position,
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
        (ldv * e) % 16 != 0 || (ldq * e) % 16 != 0 || (rope && !aligned(rope->table, 16)) || !aligned(position, 4))
        return RAD_E_ALIGN;
    const int64_t T = batch->rows, n = H * D;
    const Span none{0, 0}, in[] = {span(k, ((T - 1) * ldk + n) * e), span(v, ((T - 1) * ldv + n) * e),
                                   q ? span(q, ((T - 1) * ldq + q_heads * D) * e) : none,
                                   rope ? span(rope->table, rope->rows * rope->dim * 4) : none,
                                   position ? span(position, T * 4) : none};
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
    const rad::Kv4New nw{q, k, v, ldq, ldk, ldv, static_cast<int>(q_heads), rope ? static_cast<int>(rope->rows) : 0, q_out,
                         rope ? rope->table : nullptr, rope ? rope->dim : 0, rope ? rope->style : 0, rotate, position};
    return hip_status(rad::launch_kv4_append(cache_args(cache), batch_args(cache, batch), nw, dtype,
                                             static_cast<hipStream_t>(stream)));
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
    return append(cache, batch, k, ldk, v, ldv, q, ldq, q_heads, q_out, rope, nullptr, rotate, dtype, stream);
}

int rad_kv4_append_at(const rad_kv4_cache *cache, const rad_kv_batch *batch, const void *k, int64_t ldk, const void *v,
                      int64_t ldv, const void *q, int64_t ldq, int64_t q_heads, void *q_out, const rad_rope *rope,
                      const int32_t *position, int rotate, int32_t dtype, rad_stream_t stream) {
    return append(cache, batch, k, ldk, v, ldv, q, ldq, q_heads, q_out, rope, position, rotate, dtype, stream);
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

// What an attention call asks for beside the outputs: a tree's masks, or the tokens' weights.
struct Extra {
    bool tree, weights;
    const uint64_t *mask;
    int64_t words;
    float *weight;
    int64_t ldw, observe;
    float factor;
};

// The rows' statistics lie behind the attention's own workspace (whose sizes are multiples of 4).
int64_t stats_at(const rad_kv4_cache *c, const rad_kv_batch *b, int64_t q_heads, int32_t dtype) {
    return (rad::kv4_attn_workspace(cache_args(c), batch_args(c, b), static_cast<int>(q_heads), dtype) + 15) / 16 * 16;
}
// Behind them what the second pass makes ready.
int64_t pairs_at(const rad_kv4_cache *c, const rad_kv_batch *b, int64_t q_heads, int32_t dtype) {
    return stats_at(c, b, q_heads, dtype) + (b->rows * q_heads * 8 + 15) / 16 * 16;
}
int64_t weights_workspace(const rad_kv4_cache *c, const rad_kv_batch *b, int64_t q_heads, int32_t dtype) {
    return pairs_at(c, b, q_heads, dtype) + rad::kv4_weights_workspace(cache_args(c), batch_args(c, b), static_cast<int>(q_heads), dtype);
}

int attend(const rad_kv4_cache *cache, const rad_kv_batch *batch, const void *q, int64_t q_heads, float sm_scale, int causal,
           int64_t window, void *o, const Extra &x, void *workspace, int64_t workspace_bytes, int32_t dtype, rad_stream_t stream) {
    int rc = check_attn(cache, batch, q_heads, dtype);
    if (rc < 0) return rc;
    const bool empty = rc > 0;
    if (!(sm_scale > 0.0f) || sm_scale > 0x1p126f || (causal != 0 && causal != 1)) return RAD_E_RANGE;
    if (window < 0) return RAD_E_SHAPE;
    if (x.tree && (x.words < 1 || x.words > RAD_TREE_MAX_WORDS)) return RAD_E_RANGE;
    if (x.weights) {
        if (x.observe < 0 || x.ldw % 4 != 0 || x.ldw < batch->max_pages * cache->page_size) return RAD_E_SHAPE;
        if (!(x.factor >= 0.0f) || x.factor > 3.0e38f || x.ldw > kI32Max) return RAD_E_RANGE;
    }
    if (empty) return RAD_OK;
    const rad::Kv4Cache ca = cache_args(cache);
    const rad::KvBatch ba = batch_args(cache, batch);
    const int64_t need = x.weights ? weights_workspace(cache, batch, q_heads, dtype)
                                   : rad::kv4_attn_workspace(ca, ba, static_cast<int>(q_heads), dtype);
    if (workspace_bytes < need) return RAD_E_RANGE;
    rc = check_pointers(cache, batch);
    if (rc != RAD_OK) return rc;
    if (!q || !o || (need > 0 && !workspace) || (x.tree && !x.mask) || (x.weights && !x.weight)) return RAD_E_NULL;
    if (!aligned(q, 16) || !aligned(o, 16) || !aligned(workspace, 16) || !aligned(x.mask, 8) || !aligned(x.weight, 16)) return RAD_E_ALIGN;
    const int64_t bytes = batch->rows * q_heads * cache->D * dtype_bytes(dtype);
    const Span none{0, 0}, qs = span(q, bytes), os = span(o, bytes), ws = need > 0 ? span(workspace, need) : none;
    const Span ms = x.tree ? span(x.mask, batch->rows * x.words * 8) : none;
    const Span wt = x.weights ? span(x.weight, batch->B * cache->heads * x.ldw * 4) : none;
    const Spans sp(cache, batch);
    if (overlap(os, qs) || overlap(ws, qs) || overlap(ws, os) || sp.meets(os) || sp.meets(ws)) return RAD_E_ALIAS;
    if (overlap(ms, os) || overlap(ms, ws) || overlap(wt, qs) || overlap(wt, os) || overlap(wt, ws) || sp.meets(wt)) return RAD_E_ALIAS;
    const int win = window > 0 && window < kMaxTokens ? static_cast<int>(window) : 0;
    rad::Kv4Attn at{q, o, static_cast<int>(q_heads), sm_scale, x.tree ? static_cast<int>(x.words) : causal, win, {nullptr}};
    if (x.weights) at.stats = reinterpret_cast<float2 *>(static_cast<char *>(workspace) + stats_at(cache, batch, q_heads, dtype));
    if (x.tree) at.mask = x.mask;
    hipStream_t st = static_cast<hipStream_t>(stream);
    if (x.tree) return hip_status(rad::launch_kv4_attn_tree(ca, ba, at, workspace, dtype, st));
    const hipError_t err = rad::launch_kv4_attn(ca, ba, at, workspace, dtype, st);
    if (err != hipSuccess || !x.weights) return hip_status(err);
    const int observe = x.observe < batch->rows ? static_cast<int>(x.observe) : 0;
    void *pairs = static_cast<char *>(workspace) + pairs_at(cache, batch, q_heads, dtype);
    return hip_status(rad::launch_kv4_weights(ca, ba, at, rad::Kv4Weights{x.weight, x.ldw, observe, x.factor, pairs}, dtype, st));
}

// Sizes of the selection; 1 when there is nothing to select.
int check_select(int64_t B, int64_t heads, int64_t max_tokens) {
    if (B < 0 || heads < 0 || max_tokens < 0) return RAD_E_SHAPE;
    if (B >= kMaxRows || heads > 1024 || max_tokens >= kMaxTokens || B * heads >= kMaxRows) return RAD_E_RANGE;
    return B == 0 || heads == 0 ? 1 : RAD_OK;
}

rad::Linear linear_args(const rad_linear *in, const float *state, float *state_out, float scale, void *o) {
    const int64_t most = in->q_start ? (in->max_q < in->rows ? in->max_q : in->rows) : 1;
    return rad::Linear{in->q, in->k, in->v, in->ldq, in->ldk, in->ldv, in->log_decay, in->q_start, static_cast<int>(in->B),
                       static_cast<int>(in->rows), static_cast<int>(most), static_cast<int>(in->qk_heads),
                       static_cast<int>(in->heads), static_cast<int>(in->D), state, state_out, scale, o};
}

// Sizes of linear attention; 1 when there is neither a row nor a state to hand on.
int check_linear(const rad_linear *in) {
    if (!in) return RAD_E_NULL;
    if (dtype_bytes(in->dtype) == 0) return RAD_E_FMT;
    if (in->D != 64 && in->D != 128 && in->D != 256) return RAD_E_SHAPE;
    if (in->B < 0 || in->rows < 0 || in->max_q < 0 || in->heads < 1 || in->qk_heads < 1 || in->heads % in->qk_heads != 0) return RAD_E_SHAPE;
    if (in->B >= kMaxRows || in->rows >= kMaxRows || in->heads > 1024 || in->B * in->heads >= kMaxRows) return RAD_E_RANGE;
    const int64_t nk = in->qk_heads * in->D;
    if (in->ldq < nk || in->ldk < nk || in->ldv < in->heads * in->D) return RAD_E_SHAPE;
    if (in->ldq > kI32Max || in->ldk > kI32Max || in->ldv > kI32Max) return RAD_E_RANGE;
    if (!in->q_start && in->rows != in->B) return RAD_E_SHAPE;
    if (in->B == 0) return 1;
    return rad::linear_fits(linear_args(in, nullptr, nullptr, 1.0f, nullptr), in->dtype) ? RAD_OK : RAD_E_RANGE;
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
    return attend(cache, batch, q, q_heads, sm_scale, causal, window, o, Extra{}, workspace, workspace_bytes, dtype, stream);
}

int rad_attn_kv4_tree(const rad_kv4_cache *cache, const rad_kv_batch *batch, const void *q, int64_t q_heads,
                      float sm_scale, const uint64_t *mask, int64_t words, int64_t window, void *o, void *workspace,
                      int64_t workspace_bytes, int32_t dtype, rad_stream_t stream) {
    Extra x{};
    x.tree = true;
    x.mask = mask;
    x.words = words;
    return attend(cache, batch, q, q_heads, sm_scale, 1, window, o, x, workspace, workspace_bytes, dtype, stream);
}

int rad_attn_kv4_weights_workspace(const rad_kv4_cache *cache, const rad_kv_batch *batch, int64_t q_heads, int32_t dtype,
                                   int64_t *bytes) {
    const int rc = check_attn(cache, batch, q_heads, dtype);
    if (rc < 0) return rc;
    if (!bytes) return RAD_E_NULL;
    *bytes = rc ? 0 : weights_workspace(cache, batch, q_heads, dtype);
    return RAD_OK;
}

int rad_attn_kv4_weights(const rad_kv4_cache *cache, const rad_kv_batch *batch, const void *q, int64_t q_heads,
                         float sm_scale, int causal, int64_t window, void *o, float *weight, int64_t ldw,
                         int64_t observe, float factor, void *workspace, int64_t workspace_bytes, int32_t dtype,
                         rad_stream_t stream) {
    Extra x{};
    x.weights = true;
    x.weight = weight;
    x.ldw = ldw;
    x.observe = observe;
    x.factor = factor;
    return attend(cache, batch, q, q_heads, sm_scale, causal, window, o, x, workspace, workspace_bytes, dtype, stream);
}

int rad_kv4_select_workspace(int64_t B, int64_t heads, int64_t max_tokens, int64_t *bytes) {
    const int rc = check_select(B, heads, max_tokens);
    if (rc < 0) return rc;
    if (!bytes) return RAD_E_NULL;
    *bytes = rc ? 0 : rad::kv4_select_workspace(B, heads, max_tokens);
    return RAD_OK;
}

int rad_kv4_select(const float *weight, int64_t ldw, const int32_t *seq_len, int64_t B, int64_t heads, int64_t max_tokens,
                   int64_t budget, int64_t first, int64_t recent, int32_t *kept, int32_t *count, float *kept_weight,
                   int64_t ld_kept, void *workspace, int64_t workspace_bytes, rad_stream_t stream) {
    const int rc = check_select(B, heads, max_tokens);
    if (rc < 0) return rc;
    if (budget < 1 || first < 0 || recent < 0 || ldw < max_tokens || ldw % 4 != 0) return RAD_E_SHAPE;
    if (kept_weight && ld_kept < budget) return RAD_E_SHAPE;
    if (budget >= kMaxTokens || first > budget || recent > budget - first || ldw > kI32Max || ld_kept > kI32Max) return RAD_E_RANGE;
    if (rc) return RAD_OK;
    const int64_t need = rad::kv4_select_workspace(B, heads, max_tokens);
    if (workspace_bytes < need) return RAD_E_RANGE;
    if ((max_tokens > 0 && !weight) || !seq_len || !kept || !count || (need > 0 && !workspace)) return RAD_E_NULL;
    if (!aligned(weight, 16) || !aligned(seq_len, 4) || !aligned(kept, 4) || !aligned(count, 4) ||
        !aligned(kept_weight, 4) || !aligned(workspace, 16))
        return RAD_E_ALIGN;
    const int64_t pairs = B * heads;
    const Span in[] = {span(weight, pairs * ldw * 4), span(seq_len, B * 4)};
    const Span out[] = {span(kept, pairs * budget * 4), span(count, B * 4),
                        kept_weight ? span(kept_weight, pairs * ld_kept * 4) : Span{0, 0},
                        need > 0 ? span(workspace, need) : Span{0, 0}};
    for (int i = 0; i < 4; ++i) {
        for (const Span &x : in)
            if (overlap(out[i], x)) return RAD_E_ALIAS;
        for (int j = 0; j < i; ++j)
            if (overlap(out[i], out[j])) return RAD_E_ALIAS;
    }
    const rad::Kv4Select sel{weight, ldw, seq_len, static_cast<int>(B), static_cast<int>(heads), static_cast<int>(max_tokens),
                             static_cast<int>(budget), static_cast<int>(first), static_cast<int>(recent), kept, count,
                             kept_weight, ld_kept};
    return hip_status(rad::launch_kv4_select(sel, workspace, static_cast<hipStream_t>(stream)));
}

int rad_kv4_move(const rad_kv4_cache *cache, const rad_kv_batch *batch, const int32_t *from, int64_t lists,
                 int64_t entries, const int32_t *count, const rad_kv4_cache *to, const int32_t *to_table, int64_t to_pages,
                 const int32_t *to_start, rad_stream_t stream) {
    int rc = check_cache(cache);
    if (rc != RAD_OK) return rc;
    if (!batch) return RAD_E_NULL;
    const int64_t B = batch->B, heads = cache->heads;
    if (B < 0 || batch->max_pages < 0 || entries < 0 || to_pages < 0) return RAD_E_SHAPE;
    if (lists != 1 && lists != heads) return RAD_E_SHAPE;
    if (B * heads >= kMaxRows || B >= kMaxRows || batch->max_pages > kI32Max || batch->max_pages * cache->page_size >= kMaxTokens ||
        entries >= kMaxTokens || to_pages > kI32Max)
        return RAD_E_RANGE;
    if (to) {
        rc = check_cache(to);
        if (rc != RAD_OK) return rc;
        if (to->heads != heads || to->D != cache->D) return RAD_E_SHAPE;
    } else {
        to = cache;
    }
    if (to_pages * to->page_size >= kMaxTokens) return RAD_E_RANGE;
    const bool in_place = to_pages == 0 && !to_table;
    if (in_place && to != cache) return RAD_E_NULL;
    if (in_place && entries > RAD_KV4_MOVE_MAX) return RAD_E_RANGE;
    if (B == 0 || entries == 0 || (!in_place && to_pages == 0)) return RAD_OK;
    rc = check_pointers(cache, batch);
    if (rc != RAD_OK) return rc;
    if (!from || !count || (!in_place && !to_table) || !to->k_codes || !to->k_scale || !to->v_codes || !to->v_scale) return RAD_E_NULL;
    if (!aligned(from, 4) || !aligned(count, 4) || !aligned(to_table, 4) || !aligned(to_start, 4) || !aligned(to->k_codes, 16) ||
        !aligned(to->k_scale, 16) || !aligned(to->v_codes, 16) || !aligned(to->v_scale, 16))
        return RAD_E_ALIGN;
    // the arrays written: the target cache's, which the call reads only where the two are one
    rad_kv_batch lists_only = *batch;
    lists_only.q_start = nullptr;
    const Spans from_sp(cache, &lists_only), to_sp(to, &lists_only);
    const Span lists_in[] = {span(from, B * lists * entries * 4), span(count, B * 4), to_start ? span(to_start, B * 4) : Span{0, 0},
                             in_place ? Span{0, 0} : span(to_table, B * to_pages * 4)};
    for (const Span &x : lists_in)
        if (to_sp.meets_cache(x)) return RAD_E_ALIAS;
    for (const Span &x : to_sp.batch)
        if (to_sp.meets_cache(x)) return RAD_E_ALIAS;
    for (int i = 0; i < 4; ++i) {
        for (int j = 0; j < i; ++j)
            if (overlap(to_sp.cache[i], to_sp.cache[j])) return RAD_E_ALIAS;
        // another cache's arrays: none of them may meet these, but each may be its own counterpart
        for (int j = 0; j < 4; ++j)
            if (overlap(to_sp.cache[i], from_sp.cache[j]) && (i != j || to_sp.cache[i].lo != from_sp.cache[j].lo || to->page_size != cache->page_size)) return RAD_E_ALIAS;
    }
    const rad::Kv4Move m{from, count, in_place ? nullptr : to_table, to_start, static_cast<int>(lists), static_cast<int>(entries),
                         static_cast<int>(to_pages)};
    const rad::KvBatch b{batch->block_table, batch->seq_len, nullptr, static_cast<int>(B), static_cast<int>(batch->max_pages), 0, 0,
                         page_shift(cache)};
    return hip_status(rad::launch_kv4_move(cache_args(cache), b, cache_args(to), m, static_cast<hipStream_t>(stream)));
}

int rad_linear_attn_workspace(const rad_linear *in, int64_t *bytes) {
    const int rc = check_linear(in);
    if (rc < 0) return rc;
    if (!bytes) return RAD_E_NULL;
    *bytes = rc ? 0 : rad::linear_workspace(linear_args(in, nullptr, nullptr, 1.0f, nullptr), in->dtype);
    return RAD_OK;
}

int rad_linear_attn(const rad_linear *in, const float *state, float *state_out, float scale, void *o, void *workspace,
                    int64_t workspace_bytes, rad_stream_t stream) {
    const int rc = check_linear(in);
    if (rc < 0) return rc;
    if (!(fabsf(scale) <= 3.4028234663852886e38f)) return RAD_E_RANGE;
    if (rc) return RAD_OK;
    const int e = dtype_bytes(in->dtype);
    const rad::Linear l = linear_args(in, state, state_out, scale, o);
    const int64_t need = rad::linear_workspace(l, in->dtype);
    if (workspace_bytes < need) return RAD_E_RANGE;
    const int64_t T = in->rows, n = in->heads * in->D, nk = in->qk_heads * in->D;
    if (!in->log_decay || (need > 0 && !workspace) || (T > 0 && (!in->q || !in->k || !in->v || !o))) return RAD_E_NULL;
    if (!aligned(in->q, 16) || !aligned(in->k, 16) || !aligned(in->v, 16) || !aligned(o, 16) || !aligned(in->log_decay, 4) ||
        !aligned(in->q_start, 4) || !aligned(state, 16) || !aligned(state_out, 16) || !aligned(workspace, 16) ||
        (in->ldq * e) % 16 != 0 || (in->ldk * e) % 16 != 0 || (in->ldv * e) % 16 != 0)
        return RAD_E_ALIGN;
    const Span none{0, 0};
    const int64_t sb = in->B * in->heads * in->D * in->D * 4;
    const Span is[] = {T > 0 ? span(in->q, ((T - 1) * in->ldq + nk) * e) : none, T > 0 ? span(in->k, ((T - 1) * in->ldk + nk) * e) : none,
                       T > 0 ? span(in->v, ((T - 1) * in->ldv + n) * e) : none, span(in->log_decay, in->heads * 4),
                       in->q_start ? span(in->q_start, (in->B + 1) * 4) : none,
                       state && state != state_out ? span(state, sb) : none};
    const Span os[] = {T > 0 ? span(o, T * n * e) : none, state_out ? span(state_out, sb) : none, need > 0 ? span(workspace, need) : none};
    for (int i = 0; i < 3; ++i) {
        for (const Span &x : is)
            if (overlap(os[i], x)) return RAD_E_ALIAS;
        for (int j = 0; j < i; ++j)
            if (overlap(os[i], os[j])) return RAD_E_ALIAS;
    }
    return hip_status(rad::launch_linear(l, in->dtype, workspace, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
