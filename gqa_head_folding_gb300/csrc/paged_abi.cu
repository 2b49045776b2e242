// paged_abi.cu -- the extern "C" entry points of the paged cache declared in
// include/gqaq.h: host-side argument validation, then one launch each.
#include <math.h>

#include "internal.h"

using namespace gqaq;

namespace {

constexpr int kMaxTokens = 1 << 22;
constexpr int64_t kMaxHeads = 1 << 20;  // q, k and v heads of a token: the append's grid and the bytes of its ring are 32-bit numbers

bool page_size_ok(int s) { return s == 8 || s == 16 || s == 32 || s == 64 || s == 128; }

// Shape checks of the tables (heads: also of the rows and the pools).
int check_paged(const gqaq_paged_dims *d, bool heads) {
    if (d == nullptr) return GQAQ_ERR_INVALID_ARG;
    if (d->batch < 1 || d->page_size < 1 || d->num_pages < 1 || d->max_pages < 1 || d->max_tokens < 1 ||
        d->max_len < 0)
        return GQAQ_ERR_INVALID_ARG;
    if (!page_size_ok(d->page_size) || d->batch > kPagedMaxBatch || d->max_tokens > kMaxTokens) return GQAQ_ERR_UNSUPPORTED;
    // positions, slots and their tiles' ends are 32-bit numbers
    if ((int64_t)d->max_pages * d->page_size > INT32_MAX - 1024 || (int64_t)d->num_pages * d->page_size > INT32_MAX - 1024 ||
        (int64_t)d->batch * d->max_pages > INT32_MAX)
        return GQAQ_ERR_UNSUPPORTED;
    if (!heads) return GQAQ_OK;
    if (d->num_q_heads < 1 || d->num_kv_heads < 1 || d->head_dim < 1) return GQAQ_ERR_INVALID_ARG;
    if (d->num_q_heads % d->num_kv_heads != 0) return GQAQ_ERR_INVALID_ARG;
    if (d->dtype != GQAQ_F16 && d->dtype != GQAQ_BF16) return GQAQ_ERR_UNSUPPORTED;
    if ((int64_t)d->num_q_heads + 2 * (int64_t)d->num_kv_heads > kMaxHeads) return GQAQ_ERR_UNSUPPORTED;
    const int G = d->num_q_heads / d->num_kv_heads;
    if (G != 1 && G != 2 && G != 4 && G != 8) return GQAQ_ERR_UNSUPPORTED;
    if (d->head_dim != 64 && d->head_dim != 128) return GQAQ_ERR_UNSUPPORTED;
    if ((int64_t)d->num_pages * d->num_kv_heads * d->page_size > (int64_t)INT32_MAX - 1024) return GQAQ_ERR_UNSUPPORTED;
    if ((int64_t)d->max_tokens * d->num_q_heads > INT32_MAX / 2) return GQAQ_ERR_UNSUPPORTED;
    return GQAQ_OK;
}

bool aligned4(const void *p) { return p != nullptr && (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

}  // namespace

extern "C" {

int paged_build_tables(const gqaq_paged_dims *dims, const int32_t *cache_len, const int32_t *new_len,
                       const int32_t *free_pages, const int32_t *free_count, int32_t *block_table, int32_t *kv_len,
                       int32_t *cu_q, int32_t *positions, int32_t *slots, int32_t *free_count_out, void *stream) {
    int rc = check_paged(dims, false);
    if (rc != GQAQ_OK) return rc;
    if (!aligned4(cache_len) || !aligned4(new_len) || !aligned4(free_pages) || !aligned4(free_count) ||
        !aligned4(block_table) || !aligned4(kv_len) || !aligned4(cu_q) || !aligned4(positions) || !aligned4(slots) ||
        !aligned4(free_count_out))
        return GQAQ_ERR_INVALID_ARG;
    if (kv_len == cache_len || kv_len == new_len) return GQAQ_ERR_INVALID_ARG;  // read while it is written
    LaunchCtx ctx;
    rc = make_ctx(&ctx, stream);
    if (rc != GQAQ_OK) return rc;
    PagedTablesArgs a = {dims, cache_len, new_len, free_pages, free_count, block_table, kv_len, cu_q, positions, slots,
                         free_count_out};
    return launch_paged_tables(a, ctx);
}

int paged_release_pages(const gqaq_paged_dims *dims, const int32_t *kv_len, const int32_t *keep_len,
                        const int32_t *block_table, int32_t *free_pages, const int32_t *free_count,
                        int32_t *free_count_out, void *stream) {
    int rc = check_paged(dims, false);
    if (rc != GQAQ_OK) return rc;
    if (!aligned4(kv_len) || !aligned4(keep_len) || !aligned4(block_table) || !aligned4(free_pages) ||
        !aligned4(free_count) || !aligned4(free_count_out))
        return GQAQ_ERR_INVALID_ARG;
    if (free_pages == block_table) return GQAQ_ERR_INVALID_ARG;  // read while it is written
    LaunchCtx ctx;
    rc = make_ctx(&ctx, stream);
    if (rc != GQAQ_OK) return rc;
    PagedReleaseArgs a = {dims, kv_len, keep_len, block_table, free_count, free_pages, free_count_out};
    return launch_paged_release(a, ctx);
}

int paged_norm_rope_append(const gqaq_paged_dims *dims, const gqaq_half *q, int64_t q_stride, const gqaq_half *k,
                           int64_t k_stride, const gqaq_half *v, int64_t v_stride, const int32_t *positions,
                           const int32_t *slots, const gqaq_half *q_weight, const gqaq_half *k_weight, float eps,
                           const float *cos_sin, int rope_dim, int max_position, int interleaved, gqaq_half *q_out,
                           gqaq_half *k_pages, gqaq_half *v_pages, void *stream) {
    int rc = check_paged(dims, true);
    if (rc != GQAQ_OK) return rc;
    if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(q_out) || !aligned16(k_pages) ||
        !aligned16(v_pages) || !aligned4(positions) || !aligned4(slots))
        return GQAQ_ERR_INVALID_ARG;
    if ((q_weight != nullptr && !aligned16(q_weight)) || (k_weight != nullptr && !aligned16(k_weight)))
        return GQAQ_ERR_INVALID_ARG;
    const int64_t qrow = (int64_t)dims->num_q_heads * dims->head_dim, krow = (int64_t)dims->num_kv_heads * dims->head_dim;
    if (q_stride < qrow || k_stride < krow || v_stride < krow) return GQAQ_ERR_INVALID_ARG;
    if ((q_stride | k_stride | v_stride) % 8 != 0) return GQAQ_ERR_INVALID_ARG;  // rows are read 16 bytes at a time
    if (q_out == q && q_stride != qrow) return GQAQ_ERR_INVALID_ARG;             // in place: the rows must coincide
    if (rope_dim < 0 || rope_dim > dims->head_dim || rope_dim % 16 != 0) return GQAQ_ERR_INVALID_ARG;
    if (rope_dim > 0 && (!aligned16(cos_sin) || max_position < 1)) return GQAQ_ERR_INVALID_ARG;
    if (!isfinite(eps) || eps < 0.f) return GQAQ_ERR_INVALID_ARG;
    LaunchCtx ctx;
    rc = make_ctx(&ctx, stream);
    if (rc != GQAQ_OK) return rc;
    PagedAppendArgs a = {dims, q, k, v, q_stride, k_stride, v_stride, positions, slots, q_weight, k_weight, eps, cos_sin,
                         rope_dim, max_position, interleaved, q_out, k_pages, v_pages};
    return launch_paged_append(a, ctx);
}

size_t gqaq_paged_workspace_bytes(const gqaq_paged_dims *dims) {
    if (check_paged(dims, true) != GQAQ_OK) return 0;
    LaunchCtx ctx;
    if (make_ctx(&ctx, nullptr) != GQAQ_OK) return 0;
    return paged_attn_workspace_bytes(dims, ctx);
}

int gqa_paged_attn(const gqaq_paged_dims *dims, int max_q_len, const gqaq_half *q, const gqaq_half *k_pages,
                   const gqaq_half *v_pages, const int32_t *block_table, const int32_t *cu_q, const int32_t *kv_len,
                   float scale, gqaq_half *out, void *workspace, size_t workspace_bytes, void *stream) {
    int rc = check_paged(dims, true);
    if (rc != GQAQ_OK) return rc;
    if (max_q_len < 1) return GQAQ_ERR_INVALID_ARG;
    if (!aligned16(q) || !aligned16(k_pages) || !aligned16(v_pages) || !aligned16(out) || !aligned4(block_table) ||
        !aligned4(cu_q) || !aligned4(kv_len))
        return GQAQ_ERR_INVALID_ARG;
    if (!isfinite(scale)) return GQAQ_ERR_INVALID_ARG;
    if (workspace == nullptr || !aligned16(workspace)) return GQAQ_ERR_WORKSPACE;
    LaunchCtx ctx;
    rc = make_ctx(&ctx, stream);
    if (rc != GQAQ_OK) return rc;
    PagedAttnArgs a = {dims, max_q_len, q, k_pages, v_pages, block_table, cu_q, kv_len, scale, out, workspace,
                       workspace_bytes};
    return launch_paged_attn(a, ctx);
}

}  // extern "C"
