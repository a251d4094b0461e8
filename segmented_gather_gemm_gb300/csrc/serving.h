// Internal interface of the serving step's operators (paged K/V cache,
// attention of draft trees, draft verification) between the C-ABI layer
// (serving_api.cu) and the kernels.
#pragma once
#include <cuda_runtime.h>
#include <cstdint>

#include "../../include/csgmv.h"

namespace csgmv {

constexpr int kTreeMaxWords = 8;           // mask words of csgmv_build_draft_tree

// csgmv_kv_cache.scratch, in ints: a header of counters, then arrays over
// pages and over sequences (see kv_cache.cu).
constexpr int kKvHeader = 64;
inline int64_t kv_scratch_ints(int64_t num_pages, int64_t max_seqs) { return kKvHeader + 4 * num_pages + 8 * max_seqs + 8; }

struct CommitParams {
    const uint16_t *k_new, *v_new;
    int64_t layer_stride, token_stride, head_stride, num_tokens;
    const int32_t *accept_index;  // NULL: 0, 1, 2, ...
    int accept_width;
    const int32_t *accept_len, *tree_indptr, *seq_slots;
    int bs;
};
cudaError_t launch_kv_commit(const csgmv_kv_cache &kv, const CommitParams &p, cudaStream_t stream);
struct ExtendParams {
    CommitParams plan;  // num_tokens, accept_len (NULL: all rows), tree_indptr, seq_slots, bs
    int64_t *slots;
    int32_t *positions, *lens_before;
};
cudaError_t launch_kv_extend(const csgmv_kv_cache &kv, const ExtendParams &p, cudaStream_t stream);
cudaError_t launch_kv_fork(const csgmv_kv_cache &kv, const int32_t *parents, const int32_t *children, int n,
                           cudaStream_t stream);
cudaError_t launch_kv_free(const csgmv_kv_cache &kv, const int32_t *seqs, const int32_t *keep, int n,
                           cudaStream_t stream);
cudaError_t launch_kv_compact(const csgmv_kv_cache &kv, cudaStream_t stream);
cudaError_t launch_kv_copy(const csgmv_kv_cache &kv, const int32_t *src, const int32_t *dst, int n,
                           cudaStream_t stream);

struct AttnParams {
    const uint16_t *q, *k_new, *v_new;
    uint16_t *out;
    float *lse;  // or NULL
    int64_t q_ts, q_hs, n_ts, n_hs, o_ts, o_hs;
    const uint16_t *k_pages, *v_pages;  // of the layer
    int64_t page_stride, head_stride, token_stride;
    const int32_t *page_table, *seq_lens, *indptr, *slots;
    const int32_t *mask;  // or NULL: causal
    int32_t *status;
    float scale;
    int num_tokens, bs, hq, hkv, group, d, page_size, num_pages, max_seqs, max_pages, mask_words;
    int f16;  // 1: IEEE half, 0: bfloat16
};
size_t attn_workspace_bytes(int head_dim);
int attn_max_requests();
cudaError_t launch_tree_attention(const AttnParams &p, void *workspace, cudaStream_t stream);

struct TreeParams {
    const int32_t *parents, *indptr;
    int bs, words;
    int64_t num_nodes;
    int32_t *mask, *depth, *first_child, *next_sibling, *status;
};
cudaError_t launch_build_tree(const TreeParams &p, cudaStream_t stream);

struct VerifyParams {
    const float *target, *draft;  // draft or NULL
    int64_t target_stride, draft_stride, num_nodes;
    const int32_t *tokens, *indptr, *first_child, *next_sibling;
    const float *accept_u, *sample_u;
    int bs, vocab, width;
    int32_t *accept_index, *accept_len, *next_token, *status;
};
cudaError_t launch_verify(const VerifyParams &p, cudaStream_t stream);

}  // namespace csgmv
