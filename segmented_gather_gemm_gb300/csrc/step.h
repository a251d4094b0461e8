// Internal interface of what a decoder does between the projections, the
// attention and the verification (residual and norms, rotary positions,
// appending to the cache, logits to probabilities) between the C-ABI layer
// (step_api.cu) and the kernels.
#pragma once
#include <cuda_runtime.h>
#include <cstdint>

#include "../../include/csgmv.h"

namespace csgmv {

constexpr int kNormMaxHidden = 16384;

struct NormSide {
    const void *w, *b;  // or NULL
    float eps;
    int kind;
};
struct AddNormParams {
    const void *x, *r, *gate;  // r, gate: or NULL
    void *r_out, *out;         // or NULL
    int64_t x_s, r_s, g_s, ro_s, o_s;  // elements from row to row
    NormSide post, pre;
    float scale;
    int n, hidden;
    int dtype, r_dtype;
};
cudaError_t launch_add_norm(const AddNormParams &p, cudaStream_t stream);

// Heads of one tensor: element (t, h, d) at at + t * ts + h * hs + d.
struct Heads {
    const void *in;
    void *out;  // or NULL
    int64_t ts, hs, o_ts, o_hs;
    int n;
};
struct RotaryParams {
    const uint64_t *turns;  // [rot / 2]
    const int32_t *positions;
    float scale, sign;      // sign -1: by the negative angles
    int rot, interleaved, d, dtype;
    int rest;               // of a head's elements, those that are moved without turning
    int64_t num_tokens;
    Heads q, k;
    // appending to a layer of the cache (v, slots); slots NULL: only turning
    Heads v;
    const int64_t *slots;
    void *k_pages, *v_pages;  // of the layer
    int64_t page_stride, head_stride, token_stride, num_slots;
    int page_shift;
    int32_t *status;
};
cudaError_t launch_rotary(const RotaryParams &p, cudaStream_t stream);

struct LogitParams {
    const void *logits;
    float *out;
    int64_t logits_s, out_s, num_tokens, bias_total;
    const int32_t *indptr, *slots;
    const int32_t *counts, *seen, *num_seen;  // or NULL
    const float *repetition, *frequency, *presence, *temperature;
    const int32_t *bias_indptr, *bias_tokens;
    const float *bias_values;
    const int32_t *allow, *allow_index;
    const int32_t *drafts, *mask;  // both or neither
    int32_t *status;
    int bs, vocab, max_seqs, num_allow, allow_words, mask_words, softmax, dtype;
    int chunk;  // of a row, to a CTA
};
cudaError_t launch_process_logits(const LogitParams &p, cudaStream_t stream);

struct CountParams {
    int32_t *counts, *seen, *num_seen, *status;
    int max_seqs, vocab, prompt, accept_width;
    int64_t num_tokens;
    const int32_t *tokens, *indptr, *accept_index, *accept_len, *slots;
};
cudaError_t launch_count_tokens(const CountParams &p, int bs, cudaStream_t stream);
cudaError_t launch_count_reset(const CountParams &p, int n, cudaStream_t stream);
cudaError_t launch_count_fork(const CountParams &p, const int32_t *parents, const int32_t *children, int n, cudaStream_t stream);

}  // namespace csgmv
