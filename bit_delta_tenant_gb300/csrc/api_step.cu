// api_step.cu -- the extern "C" boundary of the decode-step operators around
// the linears (declared in include/bitdelta.h): norm, key-value cache,
// attention, sampling.  Arguments are checked before anything is launched.
#include "bd_internal.h"
#include "bitdelta.h"

#define BD_API extern "C" __attribute__((visibility("default")))

namespace {

bool aligned(const void *p, uintptr_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) == 0; }

// A page table without entries (nothing cached yet) has no address.
bool no_table(const int32_t *page_table, int32_t n_seqs, int32_t max_pages) {
    return !page_table && n_seqs > 0 && max_pages > 0;
}

int32_t status_of(cudaError_t e) { return e == cudaSuccess ? BD_OK : BD_ERR_CUDA; }

int32_t check_cache(const bd_kv_cache *c) {
    if (!c || !c->k || !c->v) return BD_ERR_INVALID_ARG;
    if (c->kv_type != BD_KV_BF16 && c->kv_type != BD_KV_E4M3 && c->kv_type != BD_KV_E2M1) return BD_ERR_INVALID_ARG;
    const bool scaled = c->kv_type != BD_KV_BF16;
    if (scaled != (c->k_scale != nullptr) || scaled != (c->v_scale != nullptr)) return BD_ERR_INVALID_ARG;
    if (c->n_pages < 1 || c->kv_heads < 1 || c->page_size < 1) return BD_ERR_INVALID_ARG;
    if (c->head_dim != 64 && c->head_dim != 128) return BD_ERR_UNSUPPORTED_SHAPE;
    if (c->page_size % 16 != 0 || c->page_size > 1024) return BD_ERR_UNSUPPORTED_SHAPE;
    if (c->kv_heads > BD_KV_MAX_HEADS || c->n_pages >= BD_MAX_DIM) return BD_ERR_UNSUPPORTED_SHAPE;
    if (!aligned(c->k, 16) || !aligned(c->v, 16) || !aligned(c->k_scale, 16) || !aligned(c->v_scale, 16))
        return BD_ERR_MISALIGNED;
    return BD_OK;
}

}  // namespace

BD_API int32_t bd_rmsnorm(const void *x, const void *residual, const void *weight, const int32_t *weight_ids,
                          int32_t n_weights, int64_t m, int64_t n, float eps, void *y, int32_t y_type, float *y_scale,
                          int32_t scale_cols, void *residual_out, void *stream) {
    if (m < 0 || n < 1 || n_weights < 1 || !weight) return BD_ERR_INVALID_ARG;
    if (m > 0 && (!x || !y)) return BD_ERR_INVALID_ARG;
    if (!(eps >= 0.f)) return BD_ERR_INVALID_ARG;
    if (y_type != BD_Y_BF16 && y_type != BD_Y_E4M3) return BD_ERR_INVALID_ARG;
    if (y_type == BD_Y_BF16 && y_scale) return BD_ERR_INVALID_ARG;
    if (n % 8 != 0 || n > BD_NORM_MAX_N || m >= BD_MAX_DIM) return BD_ERR_UNSUPPORTED_SHAPE;
    if (y_type == BD_Y_E4M3) {
        if (m > 0 && !y_scale) return BD_ERR_INVALID_ARG;
        if (scale_cols != n && (scale_cols != 128 || n % 128 != 0)) return BD_ERR_UNSUPPORTED_SHAPE;
    }
    for (const void *p : {x, residual, weight, static_cast<const void *>(y), static_cast<const void *>(residual_out)})
        if (!aligned(p, 16)) return BD_ERR_MISALIGNED;
    if (!aligned(weight_ids, 4) || !aligned(y_scale, 4)) return BD_ERR_MISALIGNED;
    if (m == 0) return BD_OK;
    bd::DevCtx ctx;
    const int32_t rc = bd::make_dev_ctx(&ctx);
    if (rc != BD_OK) return rc;
    bd::NormProblem q;
    q.x = x, q.residual = residual, q.weight = weight, q.ids = weight_ids, q.y = y, q.residual_out = residual_out;
    q.y_scale = y_scale, q.m = m, q.n = n, q.n_weights = n_weights, q.y_type = y_type, q.scale_cols = scale_cols;
    q.eps = eps;
    return status_of(bd::launch_rmsnorm(q, ctx, static_cast<cudaStream_t>(stream)));
}

BD_API int32_t bd_kv_append_rotary(const bd_kv_cache *cache, const void *q, int32_t q_heads, const void *k, const void *v,
                                   int64_t n_tokens, const int32_t *seq_ids, const int32_t *positions,
                                   const int32_t *page_table, int32_t n_seqs, int32_t max_pages, const float *rope,
                                   int64_t rope_len, int32_t rope_dim, int32_t rope_layout, void *q_out, void *stream) {
    const int32_t c = check_cache(cache);
    if (c != BD_OK) return c;
    if (n_tokens < 0 || n_seqs < 0 || max_pages < 0 || q_heads < 0 || rope_len < 0) return BD_ERR_INVALID_ARG;
    if ((q != nullptr) != (q_out != nullptr) && n_tokens > 0) return BD_ERR_INVALID_ARG;
    if (q && (!rope || q_heads < 1)) return BD_ERR_INVALID_ARG;
    if (rope && rope_layout != BD_ROTARY_HALF && rope_layout != BD_ROTARY_INTERLEAVED) return BD_ERR_INVALID_ARG;
    if (n_tokens > 0 && (!k || !v || !positions || no_table(page_table, n_seqs, max_pages))) return BD_ERR_INVALID_ARG;
    if (n_tokens >= BD_MAX_DIM || q_heads > BD_KV_MAX_HEADS * 16) return BD_ERR_UNSUPPORTED_SHAPE;
    if (rope && (rope_dim < 16 || rope_dim > cache->head_dim || rope_dim % 16 != 0)) return BD_ERR_UNSUPPORTED_SHAPE;
    if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(rope, 16) || !aligned(q_out, 16))
        return BD_ERR_MISALIGNED;
    if (!aligned(seq_ids, 4) || !aligned(positions, 4) || !aligned(page_table, 4)) return BD_ERR_MISALIGNED;
    if (n_tokens == 0) return BD_OK;
    bd::DevCtx ctx;
    const int32_t rc = bd::make_dev_ctx(&ctx);
    if (rc != BD_OK) return rc;
    return status_of(bd::launch_kv_append(*cache, q, q_heads, k, v, n_tokens, seq_ids, positions, page_table, n_seqs,
                                          max_pages, rope, rope_len, rope_dim, rope_layout == BD_ROTARY_INTERLEAVED,
                                          q_out, ctx, static_cast<cudaStream_t>(stream)));
}

BD_API int32_t bd_kv_append(const bd_kv_cache *cache, const void *q, int32_t q_heads, const void *k, const void *v,
                            int64_t n_tokens, const int32_t *seq_ids, const int32_t *positions,
                            const int32_t *page_table, int32_t n_seqs, int32_t max_pages, const float *rope,
                            int64_t rope_len, void *q_out, void *stream) {
    return bd_kv_append_rotary(cache, q, q_heads, k, v, n_tokens, seq_ids, positions, page_table, n_seqs, max_pages,
                               rope, rope_len, cache ? cache->head_dim : 0, BD_ROTARY_HALF, q_out, stream);
}

BD_API int32_t bd_rotary_table(float *table, int64_t positions, int32_t dim, double base, double factor, double original,
                               double low, double high, double amplitude, void *stream) {
    if (positions < 0 || dim < 1 || (positions > 0 && !table)) return BD_ERR_INVALID_ARG;
    for (const double v : {base, factor, original, low, high, static_cast<double>(static_cast<float>(amplitude))})
        if (!(v - v == 0)) return BD_ERR_INVALID_ARG;
    if (!(base > 0) || !(factor > 0) || !(original >= 0) || !(high > low)) return BD_ERR_INVALID_ARG;
    if (dim % 2 != 0 || dim > BD_ROTARY_MAX_DIM || positions >= BD_MAX_DIM) return BD_ERR_UNSUPPORTED_SHAPE;
    if (!aligned(table, 16)) return BD_ERR_MISALIGNED;
    uint64_t step[BD_ROTARY_MAX_DIM / 2];
    if (!bd::rotary_steps(step, dim, base, factor, original, low, high)) return BD_ERR_INVALID_ARG;
    if (positions == 0) return BD_OK;
    bd::DevCtx ctx;
    const int32_t rc = bd::make_dev_ctx(&ctx);
    if (rc != BD_OK) return rc;
    return status_of(bd::launch_rotary_table(table, positions, dim, step, static_cast<float>(amplitude), ctx,
                                             static_cast<cudaStream_t>(stream)));
}

BD_API int32_t bd_kv_read(const bd_kv_cache *cache, const int32_t *page_table, int32_t n_seqs, int32_t max_pages,
                          const int32_t *offsets, int64_t total, void *k_out, void *v_out, void *stream) {
    const int32_t c = check_cache(cache);
    if (c != BD_OK) return c;
    if (total < 0 || n_seqs < 0 || max_pages < 0) return BD_ERR_INVALID_ARG;
    if (total > 0 && n_seqs > 0 && (no_table(page_table, n_seqs, max_pages) || !offsets || !k_out || !v_out))
        return BD_ERR_INVALID_ARG;
    if (total >= BD_MAX_DIM) return BD_ERR_UNSUPPORTED_SHAPE;
    if (!aligned(k_out, 16) || !aligned(v_out, 16) || !aligned(page_table, 4) || !aligned(offsets, 4))
        return BD_ERR_MISALIGNED;
    if (total == 0 || n_seqs == 0) return BD_OK;
    bd::DevCtx ctx;
    const int32_t rc = bd::make_dev_ctx(&ctx);
    if (rc != BD_OK) return rc;
    return status_of(bd::launch_kv_read(*cache, page_table, n_seqs, max_pages, offsets, total, k_out, v_out, ctx,
                                        static_cast<cudaStream_t>(stream)));
}

namespace {

bool bad_rule(const bd_score_rule *r) {
    if (!r || r->window < 0 || !(r->scale - r->scale == 0.f) || r->reserved != 0) return true;
    return !(r->cap == 0.f || (r->cap >= 0x1p-100f && r->cap <= 0x1p100f));  // 1 / cap and cap in base 2 stay finite
}

int32_t check_heads(const bd_kv_cache *c, int32_t n_seqs, int32_t q_heads) {
    const int32_t rc = check_cache(c);
    if (rc != BD_OK) return rc;
    if (n_seqs < 0 || q_heads < 1) return BD_ERR_INVALID_ARG;
    if (q_heads % c->kv_heads != 0 || q_heads > BD_KV_MAX_HEADS * 16) return BD_ERR_UNSUPPORTED_SHAPE;
    return BD_OK;
}

}  // namespace

BD_API size_t bd_attention_workspace_size(const bd_kv_cache *cache, int32_t n_seqs, int32_t q_heads) {
    bd::DevCtx ctx;
    if (check_heads(cache, n_seqs, q_heads) != BD_OK || bd::make_dev_ctx(&ctx) != BD_OK) return 0;
    return bd::attention_workspace_size(ctx.num_sms);
}

BD_API int32_t bd_attention_decode_scored(const bd_kv_cache *cache, const void *q, int32_t q_heads,
                                          const int32_t *page_table, const int32_t *lengths, int32_t n_seqs,
                                          int32_t max_pages, const bd_score_rule *rule, void *out, float *lse,
                                          void *workspace, size_t workspace_bytes, void *stream) {
    const int32_t c = check_heads(cache, n_seqs, q_heads);
    if (c != BD_OK) return c;
    if (max_pages < 0 || bad_rule(rule)) return BD_ERR_INVALID_ARG;
    if (n_seqs > 0 && (!q || no_table(page_table, n_seqs, max_pages) || !lengths || !out)) return BD_ERR_INVALID_ARG;
    if (!aligned(q, 16) || !aligned(out, 16) || !aligned(page_table, 4) || !aligned(lengths, 4) || !aligned(lse, 4))
        return BD_ERR_MISALIGNED;
    if (!aligned(rule->slopes, 4) || !aligned(rule->first, 4) || !aligned(rule->prefix, 4)) return BD_ERR_MISALIGNED;
    if (n_seqs == 0) return BD_OK;
    if (!workspace || !aligned(workspace, 256)) return BD_ERR_WORKSPACE;
    bd::DevCtx ctx;
    const int32_t rc = bd::make_dev_ctx(&ctx);
    if (rc != BD_OK) return rc;
    if (workspace_bytes < bd::attention_workspace_size(ctx.num_sms)) return BD_ERR_WORKSPACE;
    return status_of(bd::launch_attention(*cache, q, q_heads, page_table, lengths, n_seqs, max_pages, *rule, out, lse,
                                          workspace, ctx, static_cast<cudaStream_t>(stream)));
}

BD_API int32_t bd_attention_decode(const bd_kv_cache *cache, const void *q, int32_t q_heads, const int32_t *page_table,
                                   const int32_t *lengths, int32_t n_seqs, int32_t max_pages, float scale,
                                   int32_t window, void *out, float *lse, void *workspace, size_t workspace_bytes,
                                   void *stream) {
    bd_score_rule rule = {};
    rule.scale = scale;
    rule.window = window;
    return bd_attention_decode_scored(cache, q, q_heads, page_table, lengths, n_seqs, max_pages, &rule, out, lse, workspace,
                                      workspace_bytes, stream);
}

BD_API size_t bd_attention_prompt_workspace_size(const bd_kv_cache *cache, int32_t q_heads) {
    bd::DevCtx ctx;
    if (check_heads(cache, 0, q_heads) != BD_OK || bd::make_dev_ctx(&ctx) != BD_OK) return 0;
    return bd::prompt_workspace_size(ctx.num_sms, cache->head_dim);
}

BD_API int32_t bd_attention_prompt(const bd_kv_cache *cache, const void *q, int32_t q_heads, const int32_t *offsets,
                                   int64_t total, const int32_t *page_table, const int32_t *lengths, int32_t n_seqs,
                                   int32_t max_pages, const bd_score_rule *rule, void *out, float *lse, void *workspace,
                                   size_t workspace_bytes, void *stream) {
    const int32_t c = check_heads(cache, n_seqs, q_heads);
    if (c != BD_OK) return c;
    if (max_pages < 0 || total < 0 || bad_rule(rule)) return BD_ERR_INVALID_ARG;
    if (n_seqs > 0 && total > 0 && (!q || !offsets || no_table(page_table, n_seqs, max_pages) || !lengths || !out))
        return BD_ERR_INVALID_ARG;
    if (total >= BD_MAX_DIM) return BD_ERR_UNSUPPORTED_SHAPE;
    if (!aligned(q, 16) || !aligned(out, 16) || !aligned(page_table, 4) || !aligned(lengths, 4) || !aligned(offsets, 4) ||
        !aligned(lse, 4) || !aligned(rule->slopes, 4) || !aligned(rule->first, 4) || !aligned(rule->prefix, 4))
        return BD_ERR_MISALIGNED;
    if (n_seqs == 0 || total == 0) return BD_OK;
    if (!workspace || !aligned(workspace, 256)) return BD_ERR_WORKSPACE;
    bd::DevCtx ctx;
    const int32_t rc = bd::make_dev_ctx(&ctx);
    if (rc != BD_OK) return rc;
    if (workspace_bytes < bd::prompt_workspace_size(ctx.num_sms, cache->head_dim)) return BD_ERR_WORKSPACE;
    return status_of(bd::launch_prompt(*cache, q, q_heads, offsets, total, page_table, lengths, n_seqs, max_pages, *rule,
                                       out, lse, workspace, ctx, static_cast<cudaStream_t>(stream)));
}

BD_API int32_t bd_sample(const void *logits, int32_t logits_type, int64_t m, int64_t vocab, const float *temperature,
                         const int32_t *top_k, const float *top_p, const float *min_p, const float *noise,
                         int32_t *ids, float *logprob, void *stream) {
    if (m < 0 || vocab < 1) return BD_ERR_INVALID_ARG;
    if (logits_type != BD_LOGITS_BF16 && logits_type != BD_LOGITS_F32) return BD_ERR_INVALID_ARG;
    if (m > 0 && (!logits || !noise || !ids)) return BD_ERR_INVALID_ARG;
    if (vocab > BD_SAMPLE_MAX_VOCAB || m >= BD_MAX_DIM / 8) return BD_ERR_UNSUPPORTED_SHAPE;
    if (!aligned(logits, 16) || !aligned(noise, 16)) return BD_ERR_MISALIGNED;
    for (const void *p : {static_cast<const void *>(temperature), static_cast<const void *>(top_k),
                          static_cast<const void *>(top_p), static_cast<const void *>(min_p),
                          static_cast<const void *>(ids), static_cast<const void *>(logprob)})
        if (!aligned(p, 4)) return BD_ERR_MISALIGNED;
    if (m == 0) return BD_OK;
    bd::DevCtx ctx;
    const int32_t rc = bd::make_dev_ctx(&ctx);
    if (rc != BD_OK) return rc;
    return status_of(bd::launch_sample(logits, logits_type, m, vocab, temperature, top_k, top_p, min_p, noise, ids,
                                       logprob, ctx, static_cast<cudaStream_t>(stream)));
}
