// C ABI of the serving step's operators: argument checks on the host, then
// the launches of each call on the caller's stream.  Nothing here allocates,
// frees or synchronizes.
#include <algorithm>
#include <cstdarg>
#include <cstdio>

#include "csgmv_internal.h"
#include "serving.h"

namespace {

int fail(int code, const char *fmt, ...) {
    char buf[512];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(buf, sizeof buf, fmt, ap);
    va_end(ap);
    return csgmv::set_error(code, buf);
}

int launched(cudaError_t e, const char *what) {
    if (e == cudaSuccess) return CSGMV_OK;
    return fail(CSGMV_ERR_CUDA, "%s launch: %s (%s)", what, cudaGetErrorName(e), cudaGetErrorString(e));
}

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool aligned4(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

bool overlaps(const void *a, size_t abytes, const void *b, size_t bbytes) {
    if (!a || !b || !abytes || !bbytes) return false;
    const uintptr_t a0 = reinterpret_cast<uintptr_t>(a), b0 = reinterpret_cast<uintptr_t>(b);
    return a0 < b0 + bbytes && b0 < a0 + abytes;
}

struct Dim {
    int64_t extent, stride;
};
// Whether no two elements of an array of dense rows of `row` share a place:
// each dimension steps over all that those of shorter strides reach.
template <int N>
bool apart(int64_t row, Dim (&&dims)[N]) {
    std::sort(dims, dims + N, [](const Dim &a, const Dim &b) { return a.stride < b.stride; });
    int64_t span = row;
    for (const Dim &d : dims) {
        if (d.extent <= 1) continue;
        if (d.stride < span || d.stride > (INT64_MAX - span) / (d.extent - 1)) return false;
        span += (d.extent - 1) * d.stride;
    }
    return true;
}

// The cache's bookkeeping steers every kernel's addresses: nothing a call
// writes may overlap it.
bool overlaps_meta(const csgmv_kv_cache *kv, const void *p, size_t bytes) {
    return overlaps(p, bytes, kv->page_table, 4 * (size_t)kv->max_seqs * kv->max_pages_per_seq) ||
           overlaps(p, bytes, kv->seq_lens, 4 * (size_t)kv->max_seqs) ||
           overlaps(p, bytes, kv->page_refs, 4 * (size_t)kv->num_pages) || overlaps(p, bytes, kv->status, 4);
}

// A plan and the move behind it both read a call's lists; the plan checks them,
// and writes the bookkeeping and scratch: no list may lie there.
bool overlaps_plan(const csgmv_kv_cache *kv, const int32_t *list, size_t n) {
    return overlaps_meta(kv, list, 4 * n) ||
           overlaps(list, 4 * n, kv->scratch, 4 * (size_t)csgmv::kv_scratch_ints(kv->num_pages, kv->max_seqs));
}

int check_kv(const csgmv_kv_cache *kv) {
    if (!kv) return fail(CSGMV_ERR_INVALID_ARG, "kv cache is NULL");
    if (!kv->k_pages || !kv->v_pages || !kv->page_table || !kv->seq_lens || !kv->page_refs || !kv->scratch || !kv->status)
        return fail(CSGMV_ERR_INVALID_ARG, "kv cache has a NULL device buffer");
    if (!aligned16(kv->k_pages) || !aligned16(kv->v_pages))
        return fail(CSGMV_ERR_INVALID_ARG, "k_pages / v_pages must be 16-byte aligned");
    if (!aligned4(kv->page_table) || !aligned4(kv->seq_lens) || !aligned4(kv->page_refs) || !aligned4(kv->scratch) ||
        !aligned4(kv->status))
        return fail(CSGMV_ERR_INVALID_ARG, "kv cache buffers must be 4-byte aligned");
    if (kv->dtype != CSGMV_DTYPE_BF16 && kv->dtype != CSGMV_DTYPE_F16)
        return fail(CSGMV_ERR_INVALID_ARG, "kv cache dtype %d must be bf16 or f16", kv->dtype);
    if (kv->num_layers > 16384) return fail(CSGMV_ERR_UNSUPPORTED, "at most 16384 layers");
    if (kv->num_layers <= 0 || kv->num_pages <= 0 || kv->num_kv_heads <= 0 || kv->max_seqs <= 0 ||
        kv->max_pages_per_seq <= 0)
        return fail(CSGMV_ERR_INVALID_ARG, "kv cache sizes must be positive");
    if (kv->page_size < 8 || kv->page_size > 4096 || (kv->page_size & (kv->page_size - 1)))
        return fail(CSGMV_ERR_UNSUPPORTED, "page_size %d must be a power of two in 8..4096", kv->page_size);
    if (kv->num_pages > (1 << 24) || kv->max_seqs > (1 << 20))
        return fail(CSGMV_ERR_UNSUPPORTED, "at most 2^24 pages and 2^20 sequences");
    if ((int64_t)kv->max_pages_per_seq * kv->page_size > INT32_MAX / 2)
        return fail(CSGMV_ERR_UNSUPPORTED, "max_pages_per_seq * page_size exceeds 2^30 tokens");
    if (kv->head_dim <= 0 || kv->head_dim % 8 || kv->head_dim > 1024)
        return fail(CSGMV_ERR_UNSUPPORTED, "head_dim %d must be a multiple of 8, at most 1024", kv->head_dim);
    if (kv->num_kv_heads > 1024) return fail(CSGMV_ERR_UNSUPPORTED, "at most 1024 kv heads");
    if (kv->layer_stride % 8 || kv->page_stride % 8 || kv->head_stride % 8 || kv->token_stride % 8 ||
        kv->layer_stride < 0 || kv->page_stride <= 0 || kv->head_stride <= 0 || kv->token_stride <= 0)
        return fail(CSGMV_ERR_INVALID_ARG, "kv cache strides must be positive multiples of 8");
    if (kv->page_stride > INT32_MAX) return fail(CSGMV_ERR_UNSUPPORTED, "page_stride exceeds 2^31 - 1 elements");
    // a head's rows, a page and a layer each keep to themselves: pages with
    // heads outside or inside the token axis, whatever the padding
    const int64_t D = kv->head_dim, H = kv->num_kv_heads, P = kv->page_size;
    const bool heads_out = kv->token_stride >= D && kv->head_stride >= P * kv->token_stride - (kv->token_stride - D) &&
                           kv->page_stride >= (H - 1) * kv->head_stride + (P - 1) * kv->token_stride + D;
    const bool heads_in = kv->head_stride >= D && kv->token_stride >= (H - 1) * kv->head_stride + D &&
                          kv->page_stride >= (P - 1) * kv->token_stride + (H - 1) * kv->head_stride + D;
    if ((!heads_out && !heads_in) || !apart(D, {{kv->num_layers, kv->layer_stride},
                                                {kv->num_pages, kv->page_stride},
                                                {H, kv->head_stride},
                                                {P, kv->token_stride}}))
        return fail(CSGMV_ERR_INVALID_ARG, "kv cache strides overlap");
    return CSGMV_OK;
}

int check_new(const void *k, const void *v, int64_t ts, int64_t hs) {
    if (!k || !v) return fail(CSGMV_ERR_INVALID_ARG, "k_new / v_new is NULL");
    if (!aligned16(k) || !aligned16(v)) return fail(CSGMV_ERR_INVALID_ARG, "k_new / v_new must be 16-byte aligned");
    if (ts % 8 || hs % 8 || ts <= 0 || hs <= 0)
        return fail(CSGMV_ERR_INVALID_ARG, "k_new / v_new strides must be positive multiples of 8");
    return CSGMV_OK;
}

cudaStream_t st(csgmv_stream_t s) { return reinterpret_cast<cudaStream_t>(s); }

}  // namespace

extern "C" {

int64_t csgmv_kv_scratch_ints(int num_pages, int max_seqs) {
    if (num_pages < 0 || max_seqs < 0) return 0;
    return csgmv::kv_scratch_ints(num_pages, max_seqs);
}

int csgmv_kv_commit(const csgmv_kv_cache *kv, const void *k_new, const void *v_new, int64_t new_layer_stride,
                    int64_t new_token_stride, int64_t new_head_stride, int64_t num_tokens, const int32_t *accept_index,
                    int accept_width, const int32_t *accept_len, const int32_t *tree_indptr, const int32_t *seq_slots,
                    int bs, csgmv_stream_t stream) {
    int rc = check_kv(kv);
    if (rc) return rc;
    if (bs < 0 || num_tokens < 0) return fail(CSGMV_ERR_INVALID_ARG, "negative bs / num_tokens");
    if (bs > kv->max_seqs) return fail(CSGMV_ERR_CAPACITY, "bs %d exceeds max_seqs %d", bs, kv->max_seqs);
    if (num_tokens > INT32_MAX) return fail(CSGMV_ERR_UNSUPPORTED, "num_tokens exceeds int32");
    if (bs == 0) return CSGMV_OK;
    if (!accept_len || !tree_indptr) return fail(CSGMV_ERR_INVALID_ARG, "accept_len / tree_indptr is NULL");
    if (accept_index && accept_width <= 0) return fail(CSGMV_ERR_INVALID_ARG, "accept_width must be positive");
    if (num_tokens == 0) return CSGMV_OK;
    if ((rc = check_new(k_new, v_new, new_token_stride, new_head_stride))) return rc;
    if (new_layer_stride % 8 || new_layer_stride < 0)
        return fail(CSGMV_ERR_INVALID_ARG, "new_layer_stride must be a non-negative multiple of 8");
    if (overlaps_plan(kv, accept_index, (size_t)bs * accept_width) || overlaps_plan(kv, accept_len, bs) ||
        overlaps_plan(kv, tree_indptr, (size_t)bs + 1) || overlaps_plan(kv, seq_slots, bs))
        return fail(CSGMV_ERR_INVALID_ARG, "a list of the call overlaps the cache's bookkeeping or scratch");
    csgmv::CommitParams p;
    p.k_new = static_cast<const uint16_t *>(k_new);
    p.v_new = static_cast<const uint16_t *>(v_new);
    p.layer_stride = new_layer_stride;
    p.token_stride = new_token_stride;
    p.head_stride = new_head_stride;
    p.num_tokens = num_tokens;
    p.accept_index = accept_index;
    p.accept_width = accept_width;
    p.accept_len = accept_len;
    p.tree_indptr = tree_indptr;
    p.seq_slots = seq_slots;
    p.bs = bs;
    return launched(csgmv::launch_kv_commit(*kv, p, st(stream)), "csgmv_kv_commit");
}

int csgmv_kv_fork(const csgmv_kv_cache *kv, const int32_t *parents, const int32_t *children, int n,
                  csgmv_stream_t stream) {
    int rc = check_kv(kv);
    if (rc) return rc;
    if (n < 0) return fail(CSGMV_ERR_INVALID_ARG, "negative n");
    if (n > kv->max_seqs) return fail(CSGMV_ERR_CAPACITY, "n %d exceeds max_seqs %d", n, kv->max_seqs);
    if (n == 0) return CSGMV_OK;
    if (!parents || !children) return fail(CSGMV_ERR_INVALID_ARG, "parents / children is NULL");
    if (overlaps_plan(kv, parents, n) || overlaps_plan(kv, children, n))
        return fail(CSGMV_ERR_INVALID_ARG, "a list of the call overlaps the cache's bookkeeping or scratch");
    return launched(csgmv::launch_kv_fork(*kv, parents, children, n, st(stream)), "csgmv_kv_fork");
}

int csgmv_kv_free(const csgmv_kv_cache *kv, const int32_t *seqs, const int32_t *keep_lens, int n,
                  csgmv_stream_t stream) {
    int rc = check_kv(kv);
    if (rc) return rc;
    if (n < 0) return fail(CSGMV_ERR_INVALID_ARG, "negative n");
    if (n > kv->max_seqs) return fail(CSGMV_ERR_CAPACITY, "n %d exceeds max_seqs %d", n, kv->max_seqs);
    if (n == 0) return CSGMV_OK;
    if (!seqs) return fail(CSGMV_ERR_INVALID_ARG, "seqs is NULL");
    return launched(csgmv::launch_kv_free(*kv, seqs, keep_lens, n, st(stream)), "csgmv_kv_free");
}

int csgmv_kv_compact(const csgmv_kv_cache *kv, csgmv_stream_t stream) {
    int rc = check_kv(kv);
    if (rc) return rc;
    return launched(csgmv::launch_kv_compact(*kv, st(stream)), "csgmv_kv_compact");
}

int csgmv_kv_copy_pages(const csgmv_kv_cache *kv, const int32_t *src, const int32_t *dst, int n,
                        csgmv_stream_t stream) {
    int rc = check_kv(kv);
    if (rc) return rc;
    if (n < 0) return fail(CSGMV_ERR_INVALID_ARG, "negative n");
    if (n == 0) return CSGMV_OK;
    if (!src || !dst) return fail(CSGMV_ERR_INVALID_ARG, "src / dst is NULL");
    return launched(csgmv::launch_kv_copy(*kv, src, dst, n, st(stream)), "csgmv_kv_copy_pages");
}

size_t csgmv_tree_attention_workspace_bytes(const csgmv_kv_cache *kv, int num_q_heads) {
    if (!kv || num_q_heads <= 0) return 0;
    return csgmv::attn_workspace_bytes(kv->head_dim);
}

int csgmv_tree_attention(const void *q, int64_t q_token_stride, int64_t q_head_stride, int num_q_heads,
                         const void *k_new, const void *v_new, int64_t new_token_stride, int64_t new_head_stride,
                         const csgmv_kv_cache *kv, int layer, const int32_t *tree_indptr, const int32_t *seq_slots,
                         int bs, int64_t num_tokens, const int32_t *mask, int mask_words, float scale, void *out,
                         int64_t out_token_stride, int64_t out_head_stride, float *lse, void *workspace,
                         size_t workspace_bytes, csgmv_stream_t stream) {
    int rc = check_kv(kv);
    if (rc) return rc;
    if (kv->head_dim != 64 && kv->head_dim != 128)
        return fail(CSGMV_ERR_UNSUPPORTED, "head_dim %d must be 64 or 128", kv->head_dim);
    if (num_q_heads <= 0 || num_q_heads % kv->num_kv_heads)
        return fail(CSGMV_ERR_INVALID_ARG, "num_q_heads %d must be a positive multiple of num_kv_heads %d", num_q_heads,
                    kv->num_kv_heads);
    if (num_q_heads / kv->num_kv_heads > 128)
        return fail(CSGMV_ERR_UNSUPPORTED, "more than 128 query heads for each kv head");
    if (layer < 0 || layer >= kv->num_layers)
        return fail(CSGMV_ERR_INVALID_ARG, "layer %d outside [0, %d)", layer, kv->num_layers);
    if (bs < 0 || num_tokens < 0) return fail(CSGMV_ERR_INVALID_ARG, "negative bs / num_tokens");
    if (num_tokens > INT32_MAX / 128) return fail(CSGMV_ERR_UNSUPPORTED, "num_tokens exceeds 2^24");
    if (num_tokens * (num_q_heads / kv->num_kv_heads) > (1 << 30))
        return fail(CSGMV_ERR_UNSUPPORTED, "num_tokens times the query heads of a kv head exceeds 2^30");
    if (bs > csgmv::attn_max_requests())
        return fail(CSGMV_ERR_UNSUPPORTED, "bs %d exceeds %d", bs, csgmv::attn_max_requests());
    if (bs == 0 || num_tokens == 0) return CSGMV_OK;
    if (!q || !out || !tree_indptr) return fail(CSGMV_ERR_INVALID_ARG, "NULL tensor");
    if (!aligned16(q) || !aligned16(out)) return fail(CSGMV_ERR_INVALID_ARG, "q / out must be 16-byte aligned");
    if (q_token_stride % 8 || q_head_stride % 8 || out_token_stride % 8 || out_head_stride % 8 || q_token_stride < 0 ||
        q_head_stride < 0 || out_token_stride < 0 || out_head_stride < 0)
        return fail(CSGMV_ERR_INVALID_ARG, "q / out strides must be non-negative multiples of 8");
    if ((rc = check_new(k_new, v_new, new_token_stride, new_head_stride))) return rc;
    if (mask && mask_words <= 0) return fail(CSGMV_ERR_INVALID_ARG, "mask_words must be positive");
    if (lse && !aligned4(lse)) return fail(CSGMV_ERR_INVALID_ARG, "lse must be 4-byte aligned");
    if (!(scale > 0.0f) || scale > 1e30f) return fail(CSGMV_ERR_INVALID_ARG, "scale must be positive and finite");
    const size_t need = csgmv::attn_workspace_bytes(kv->head_dim);
    if (need && (!workspace || !aligned16(workspace)))
        return fail(CSGMV_ERR_INVALID_ARG, "workspace is NULL or not 16-byte aligned");
    if (!apart(kv->head_dim, {{num_tokens, out_token_stride}, {num_q_heads, out_head_stride}}))
        return fail(CSGMV_ERR_INVALID_ARG, "out strides overlap");
    // what steers the kernels' addresses and barriers, and what they write
    const size_t lse_bytes = 4 * (size_t)num_tokens * num_q_heads, ptr_bytes = 4 * (size_t)(bs + 1), slot_bytes = 4 * (size_t)bs;
    const size_t out_bytes =
        2 * ((size_t)(num_tokens - 1) * out_token_stride + (size_t)(num_q_heads - 1) * out_head_stride + kv->head_dim);
    const struct { const void *at; size_t bytes; } written[] = {{out, out_bytes}, {lse, lse_bytes}, {workspace, need}};
    bool over = overlaps(out, out_bytes, lse, lse_bytes) || overlaps(out, out_bytes, workspace, need) ||
                overlaps(lse, lse_bytes, workspace, need);
    for (const auto &w : written)
        over = over || overlaps_meta(kv, w.at, w.bytes) || overlaps(tree_indptr, ptr_bytes, w.at, w.bytes) ||
               overlaps(seq_slots, slot_bytes, w.at, w.bytes);
    if (over)
        return fail(CSGMV_ERR_INVALID_ARG,
                    "out / lse / workspace overlaps the cache's bookkeeping, tree_indptr, seq_slots or each other");
    if (workspace_bytes < need)
        return fail(CSGMV_ERR_CAPACITY, "workspace of %zu bytes, %zu needed", workspace_bytes, need);
    csgmv::AttnParams p = {};
    p.q = static_cast<const uint16_t *>(q);
    p.k_new = static_cast<const uint16_t *>(k_new);
    p.v_new = static_cast<const uint16_t *>(v_new);
    p.out = static_cast<uint16_t *>(out);
    p.lse = lse;
    p.q_ts = q_token_stride;
    p.q_hs = q_head_stride;
    p.n_ts = new_token_stride;
    p.n_hs = new_head_stride;
    p.o_ts = out_token_stride;
    p.o_hs = out_head_stride;
    p.k_pages = static_cast<const uint16_t *>(kv->k_pages) + (int64_t)layer * kv->layer_stride;
    p.v_pages = static_cast<const uint16_t *>(kv->v_pages) + (int64_t)layer * kv->layer_stride;
    p.page_stride = kv->page_stride;
    p.head_stride = kv->head_stride;
    p.token_stride = kv->token_stride;
    p.page_table = kv->page_table;
    p.seq_lens = kv->seq_lens;
    p.indptr = tree_indptr;
    p.slots = seq_slots;
    p.mask = mask;
    p.status = kv->status;
    p.scale = scale;
    p.num_tokens = (int)num_tokens;
    p.bs = bs;
    p.hq = num_q_heads;
    p.hkv = kv->num_kv_heads;
    p.group = num_q_heads / kv->num_kv_heads;
    p.d = kv->head_dim;
    p.page_size = kv->page_size;
    p.num_pages = kv->num_pages;
    p.max_seqs = kv->max_seqs;
    p.max_pages = kv->max_pages_per_seq;
    p.mask_words = mask ? mask_words : 0;
    p.f16 = kv->dtype == CSGMV_DTYPE_F16;
    return launched(csgmv::launch_tree_attention(p, workspace, st(stream)), "csgmv_tree_attention");
}

int csgmv_build_draft_tree(const int32_t *parents, const int32_t *tree_indptr, int bs, int64_t num_nodes,
                           int mask_words, int32_t *mask, int32_t *depth, int32_t *first_child, int32_t *next_sibling,
                           int32_t *status, csgmv_stream_t stream) {
    if (bs < 0 || num_nodes < 0) return fail(CSGMV_ERR_INVALID_ARG, "negative bs / num_nodes");
    if (mask_words < 1 || mask_words > csgmv::kTreeMaxWords)
        return fail(CSGMV_ERR_UNSUPPORTED, "mask_words %d outside 1..%d", mask_words, csgmv::kTreeMaxWords);
    if (num_nodes > INT32_MAX) return fail(CSGMV_ERR_UNSUPPORTED, "num_nodes exceeds int32");
    if (bs == 0 || num_nodes == 0) return CSGMV_OK;
    if (!parents || !tree_indptr || !mask || !depth || !first_child || !next_sibling || !status)
        return fail(CSGMV_ERR_INVALID_ARG, "NULL buffer");
    csgmv::TreeParams p = {parents, tree_indptr, bs, mask_words, num_nodes, mask, depth, first_child, next_sibling,
                           status};
    return launched(csgmv::launch_build_tree(p, st(stream)), "csgmv_build_draft_tree");
}

int csgmv_verify_drafts(const float *target_probs, int64_t target_stride, const float *draft_probs,
                        int64_t draft_stride, const int32_t *draft_tokens, const int32_t *tree_indptr,
                        const int32_t *first_child, const int32_t *next_sibling, const float *accept_uniforms,
                        const float *sample_uniforms, int bs, int64_t num_nodes, int vocab_size, int32_t *accept_index,
                        int accept_width, int32_t *accept_len, int32_t *next_token, int32_t *status,
                        csgmv_stream_t stream) {
    if (bs < 0 || num_nodes < 0) return fail(CSGMV_ERR_INVALID_ARG, "negative bs / num_nodes");
    if (num_nodes > INT32_MAX) return fail(CSGMV_ERR_UNSUPPORTED, "num_nodes exceeds int32");
    if (vocab_size < 1 || vocab_size > (1 << 18))
        return fail(CSGMV_ERR_UNSUPPORTED, "vocab_size %d outside 1..2^18", vocab_size);
    if (accept_width < 1) return fail(CSGMV_ERR_INVALID_ARG, "accept_width must be positive");
    if (bs == 0) return CSGMV_OK;
    if (!tree_indptr || !sample_uniforms || !accept_index || !accept_len || !next_token || !status)
        return fail(CSGMV_ERR_INVALID_ARG, "NULL buffer");
    if (num_nodes > 0 && (!target_probs || !draft_tokens || !first_child || !next_sibling || !accept_uniforms))
        return fail(CSGMV_ERR_INVALID_ARG, "NULL buffer");
    if (!aligned4(target_probs) || !aligned4(draft_probs))
        return fail(CSGMV_ERR_INVALID_ARG, "target_probs / draft_probs must be 4-byte aligned");
    if (target_stride < vocab_size || (draft_probs && draft_stride < vocab_size))
        return fail(CSGMV_ERR_INVALID_ARG, "target_stride / draft_stride below vocab_size");
    // a request's CTAs walk its tree each by itself and meet at cluster barriers: what they read must not change
    const size_t n4 = 4 * (size_t)num_nodes, b4 = 4 * (size_t)bs;
    auto rows = [&](int64_t stride) { return num_nodes ? 4 * ((size_t)(num_nodes - 1) * stride + vocab_size) : 0; };
    const struct { const void *at; size_t bytes; } read[] = {
        {target_probs, rows(target_stride)}, {draft_probs, rows(draft_stride)}, {draft_tokens, n4}, {tree_indptr, b4 + 4},
        {first_child, n4}, {next_sibling, n4}, {accept_uniforms, n4}, {sample_uniforms, b4}},
        written[] = {{accept_index, b4 * accept_width}, {accept_len, b4}, {next_token, b4}, {status, 4}};
    for (const auto &r : read)
        for (const auto &w : written)
            if (overlaps(r.at, r.bytes, w.at, w.bytes))
                return fail(CSGMV_ERR_INVALID_ARG, "an output overlaps an input");
    csgmv::VerifyParams p = {target_probs, draft_probs,  target_stride, draft_stride,    num_nodes,       draft_tokens,
                             tree_indptr,  first_child,  next_sibling,  accept_uniforms, sample_uniforms, bs,
                             vocab_size,   accept_width, accept_index,  accept_len,      next_token,      status};
    return launched(csgmv::launch_verify(p, st(stream)), "csgmv_verify_drafts");
}

}  // extern "C"
