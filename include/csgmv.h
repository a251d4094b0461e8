/*
 * csgmv.h — C ABI of libcsgmv.so, the GB300 (sm_103a) chunked segmented-gather
 * matrix-vector (csgmv) multi-adapter LoRA delta path.
 *
 * The operations follow sglang's LoRA backend interface as printed in
 *   python/sglang/srt/lora/backend/base_backend.py   (class BaseLoRABackend)
 *   python/sglang/srt/lora/backend/chunked_backend.py (class ChunkedSgmvLoRABackend)
 *   python/sglang/srt/lora/lora_manager.py            (LoRAManager.prepare_lora_batch)
 *
 * Conventions for every call:
 *  - Pointers are DEVICE pointers owned by the caller unless marked "host".
 *    The library allocates nothing, frees nothing and never synchronizes; all
 *    work is enqueued on the given stream (NULL = legacy default stream), so
 *    every call can be captured in a CUDA graph.
 *  - bf16 tensors are passed as void* holding IEEE bfloat16 values; all
 *    tensors are dense row-major with the stated shapes; every device pointer
 *    must be 16-byte aligned.
 *  - Return value: CSGMV_OK (0) or a negative CSGMV_ERR_* code; then nothing
 *    was enqueued (except CSGMV_ERR_CUDA, when a launch itself failed).
 *    csgmv_last_error() gives a message for the calling thread.
 *  - Problems only the device can see (a slot index out of range, a rank
 *    above the buffer rank, a token id outside the vocabulary, a permutation
 *    entry out of range, a segment-capacity overflow, inconsistent request
 *    lengths) are OR-ed as CSGMV_STATUS_* bits into the batch info's device
 *    status word; the offending work item is skipped, nothing traps.
 */
#ifndef CSGMV_H
#define CSGMV_H

#include <stddef.h>
#include <stdint.h>

#if defined(__GNUC__)
#define CSGMV_API __attribute__((visibility("default")))
#else
#define CSGMV_API
#endif

#ifdef __cplusplus
extern "C" {
#endif

/* A cudaStream_t. */
typedef struct CUstream_st *csgmv_stream_t;

enum {
    CSGMV_OK = 0,
    CSGMV_ERR_INVALID_ARG = -1, /* bad pointer, size, dtype or offsets (host check) */
    CSGMV_ERR_CAPACITY = -2,    /* batch exceeds the batch-info buffers (host check) */
    CSGMV_ERR_CUDA = -3,        /* a CUDA runtime call or launch failed */
    CSGMV_ERR_TIMEOUT = -4,     /* reserved: no call here waits on another agent */
    CSGMV_ERR_DEVICE = -5,      /* reserved for callers that map the status word */
    CSGMV_ERR_UNSUPPORTED = -6  /* shape outside this build's limits (e.g. rank > 64) */
};

enum { CSGMV_DTYPE_BF16 = 0, CSGMV_DTYPE_F32 = 1 };

/* Bits of the device status word (csgmv_batch_info.status). */
enum {
    CSGMV_STATUS_BAD_ADAPTER = 1,     /* slot index outside [0, num_loras) */
    CSGMV_STATUS_BAD_RANK = 2,        /* slot rank outside [0, max_rank] */
    CSGMV_STATUS_BAD_TOKEN_ID = 4,    /* embedding id outside [0, vocab_size) */
    CSGMV_STATUS_BAD_PERMUTATION = 8, /* permutation entry outside [0, num_tokens) */
    CSGMV_STATUS_CAPACITY = 16,       /* segments exceed max_segments */
    CSGMV_STATUS_BAD_LENS = 32        /* negative length or lengths not summing to num_tokens */
};

/*
 * Batch info shared by every layer of one forward batch (sglang LoRABatchInfo;
 * chunked_backend.py init_cuda_graph_batch_info / prepare_lora_batch).
 * The caller allocates every device buffer once at the capacities below
 * (csgmv_batch_info_capacity gives the CUDA-graph capacities) and fills the
 * capacity fields; csgmv_build_batch_info fills the buffers and the host
 * mirror fields in place, so graphs captured over these pointers stay valid
 * across batches.
 *
 * Meaning (chunked_backend.py _get_permutation / _get_segments_info):
 *   permutation[p]     original token index at adapter-sorted position p
 *                      (stable: ties keep token order)
 *   seg_indptr[k]      first sorted position of segment k; segment k holds
 *                      positions [seg_indptr[k], seg_indptr[k+1]) that all use
 *                      slot weight_indices[k], at most chunk_size of them
 *   lora_ranks[a], scalings[a]   rank r_a and scaling of slot a (0 = no adapter)
 */
typedef struct csgmv_batch_info {
    int32_t *seg_indptr;         /* [max_segments + 1] */
    int32_t *weight_indices;     /* [max_segments] */
    int32_t *permutation;        /* [max_tokens] */
    int32_t *lora_ranks;         /* [max_loras] */
    float *scalings;             /* [max_loras] */
    int32_t *num_segments_dev;   /* [1] segments of the current batch */
    int32_t *max_len_dev;        /* [1] chunk size of the current batch */
    int32_t *req_seg_indptr;     /* [max_bs + 1] per-request token indptr, or NULL */
    int32_t *req_weight_indices; /* [max_bs] per-request slot, or NULL */
    int32_t *status;             /* [1] CSGMV_STATUS_* bits; reset by each build */
    /* capacities (set by the caller) */
    int32_t max_segments, max_tokens, max_loras, max_bs, max_rank;
    /* host mirror of the current batch (set by csgmv_build_batch_info) */
    int32_t num_tokens, chunk_size, bs, num_loras, use_cuda_graph;
    /* Optional (NULL for none): the token tiles of the current batch, for the
     * decode kernels of csgmv_qkv, so that no CTA rebuilds them from the
     * segments.  csgmv_build_batch_info writes [0] = tile count and [1..3] =
     * 0, then per tile {slot, first sorted position, tokens, 0}: every slot
     * run (a maximal stretch of segments on one slot) cut into
     * ceil(n / 64) tiles of balanced size, in segment order;
     * csgmv_build_lm_head_batch_info writes [0] = -1 (no tiles: the kernels
     * derive them from the segments).  csgmv_tile_table_ints() gives its
     * int32 length. */
    int32_t *tile_table;
} csgmv_batch_info;

/* int32 entries of csgmv_batch_info.tile_table for these capacities:
 * 4 * (max_loras + max_tokens / 64 + 2).  Host only; 0 for negative sizes. */
CSGMV_API int64_t csgmv_tile_table_ints(int max_loras, int max_tokens);

/* Message of the last failed call on this thread ("" if none). */
CSGMV_API const char *csgmv_last_error(void);

/* Library version string. */
CSGMV_API const char *csgmv_version(void);

/*
 * Chunk size for a batch of num_tokens tokens (chunked_backend.py
 * MIN_CHUNK_SIZE = 16 and _determine_chunk_size_for_tokens): 16 when
 * max_chunk_size <= 16; else min(max_chunk_size, 128 if num_tokens >= 256,
 * 32 if num_tokens >= 64, else 16).  Host only; never fails.
 */
CSGMV_API int csgmv_chunk_size(int num_tokens, int max_chunk_size);

/*
 * CUDA-graph capacities (chunked_backend.py init_cuda_graph_batch_info):
 * *max_segments = ceil(num_tokens_per_bs / 16) * max_bs and
 * *max_tokens = max_bs * num_tokens_per_bs (host pointers).  Returns
 * CSGMV_ERR_INVALID_ARG for negative sizes or int32 overflow.
 */
CSGMV_API int csgmv_batch_info_capacity(int max_bs, int num_tokens_per_bs, int32_t *max_segments,
                              int32_t *max_tokens);

/*
 * Build the batch info of one forward batch on the device (chunked_backend.py
 * prepare_lora_batch with _get_permutation and _get_segments_info;
 * lora_manager.py prepare_lora_batch for the slot ranks and scalings).
 *   req_lens[bs], req_adapter[bs]   device; tokens and slot of each request in
 *                                   token order (a decode request has 1 token)
 *   num_tokens                      host; sum of req_lens (checked on device)
 *   lora_ranks[num_loras], scalings[num_loras]  device; copied into the batch
 *                                   info (slots [num_loras, max_loras) get 0)
 *   max_chunk_size, chunk_size_override   chunk = override if > 0, else
 *                                   csgmv_chunk_size(num_tokens, max_chunk_size)
 *   use_cuda_graph                  1: pad weight_indices[n:max_segments] = 0 and
 *                                   seg_indptr[n+1:max_segments+1] = num_tokens
 * One single-CTA kernel; resets bi->status.  Host errors: bs > max_bs,
 * num_tokens > max_tokens, num_loras > max_loras, negative sizes, NULL buffers,
 * or a batch too large for one CTA's shared memory (CSGMV_ERR_UNSUPPORTED).
 * On a device-side error (status bits BAD_ADAPTER / BAD_LENS / BAD_RANK /
 * CAPACITY) the batch is left with zero segments, so later calls do nothing.
 */
CSGMV_API int csgmv_build_batch_info(csgmv_batch_info *bi, const int32_t *req_lens, const int32_t *req_adapter,
                           int bs, int num_tokens, const int32_t *lora_ranks, const float *scalings,
                           int num_loras, int max_chunk_size, int chunk_size_override,
                           int use_cuda_graph, csgmv_stream_t stream);

/*
 * Batch info of a pruned lm_head pass (chunked_backend.py
 * _prepare_lm_head_batch_info and _build_lm_head_batch_info): only
 * pruned_lens[i] tokens of request i go through lm_head, and they stay in
 * their original order, so the permutation is the identity.  Segments come
 * from merge_and_chunk_segments(weight_indices, pruned_lens, chunk), whose
 * body is not on the pages; read from its call sites: consecutive requests on
 * the same slot form one run (requests without pruned tokens are skipped, so
 * runs merge across them), and every run is cut into pieces of chunk tokens,
 * the last one shorter.  chunk = chunk_size_override if > 0, else
 * csgmv_chunk_size(num_tokens, max_chunk_size).
 *   pruned_lens[bs], req_adapter[bs]   device; pruned tokens and slot of each
 *                                      request, in request order
 *   num_tokens                         host; sum of pruned_lens
 *   lora_ranks, scalings, num_loras, use_cuda_graph   as csgmv_build_batch_info
 * The result drives csgmv_shrink / csgmv_expand / csgmv_qkv over the pruned
 * rows (x and base_output with num_tokens rows).  Runs here follow request
 * order, not slot order, so the batch info needs max_segments of up to
 * ceil(num_tokens / chunk) plus the number of requests with pruned tokens
 * (CSGMV_STATUS_CAPACITY otherwise).  req_seg_indptr and
 * req_weight_indices are not written.  One single-CTA kernel; errors as
 * csgmv_build_batch_info.
 */
CSGMV_API int csgmv_build_lm_head_batch_info(csgmv_batch_info *bi, const int32_t *pruned_lens,
                                   const int32_t *req_adapter, int bs, int num_tokens,
                                   const int32_t *lora_ranks, const float *scalings, int num_loras,
                                   int max_chunk_size, int chunk_size_override, int use_cuda_graph,
                                   csgmv_stream_t stream);

/*
 * Shrink (base_backend.py run_lora_a_sgemm; chunked_backend.py
 * run_lora_a_sgemm with num_slices): for token t on slot w with rank r,
 *     h[t][j*r + k] = sum_i x[t][i] * A[w][j*r + k][i]     (j < c, k < r)
 * and h[t][n] = 0 for c*r <= n < c*R (also for rank-0 tokens).
 *   x  bf16 (s, K), s = bi->num_tokens;  A  bf16 (max_loras, c*R, K), R = bi->max_rank
 *   h  (s, ldh) of h_dtype (CSGMV_DTYPE_BF16 rounds to nearest even,
 *      CSGMV_DTYPE_F32 keeps fp32), ldh >= c*R; only columns [0, c*R) are written
 *   num_slices c in {1, 2, 3}; K a multiple of 8; R in {8, 16, 32, 64}.
 * fp32 accumulation on the tensor cores.
 */
CSGMV_API int csgmv_shrink(const void *x, int64_t s, int64_t K, const void *A, int num_slices, void *h,
                 int h_dtype, int64_t ldh, const csgmv_batch_info *bi, csgmv_stream_t stream);

/*
 * Expand (base_backend.py run_lora_b_sgemm; chunked_backend.py
 * run_lora_b_sgemm / run_qkv_lora with slice_offsets, max_slice_size and
 * base_output): for token t on slot w with rank r and scaling sigma, slice j
 * and column n in [off[j], off[j+1]),
 *     out[t][n] = (accumulate ? out[t][n] : 0) + sigma * sum_{k<r} h[t][j*r+k] * B[w][n][k]
 * rounded once to bf16.  Columns outside [off[0], off[c]) are not touched;
 * with accumulate = 1 rows of rank-0 tokens are not touched either, with
 * accumulate = 0 they are set to 0 in the covered columns.
 *   h   (s, ldh) of h_dtype, as produced by csgmv_shrink
 *   B   bf16 (max_loras, N, R);  out  bf16 (s, N), in place when accumulate = 1
 *   slice_offsets  HOST int32[c+1], non-decreasing, multiples of 8, off[c] <= N
 *   max_slice_size >= the widest slice (sglang passes it to size the launch)
 * The fp32 h is applied as a bf16 hi + lo pair, so the product keeps ~16 bits.
 */
CSGMV_API int csgmv_expand(const void *h, int h_dtype, int64_t ldh, const void *B, int64_t N,
                 const int32_t *slice_offsets, int num_slices, int max_slice_size, void *out,
                 int accumulate, const csgmv_batch_info *bi, csgmv_stream_t stream);

/*
 * Fused shrink -> expand (chunked_backend.py run_qkv_lora and
 * run_gate_up_lora; c = 1 is the single-projection pair run_lora_a_sgemm +
 * run_lora_b_sgemm):
 *     base_output[t][n] += sigma_w * sum_k (sum_i x[t][i] A[w][j*r+k][i]) B[w][n][k]
 * for n in slice j = [off[j], off[j+1]).  h stays fp32, so the only rounding
 * to bf16 is the final store.  Shapes and limits as csgmv_shrink and
 * csgmv_expand; base_output is bf16 (s, N), updated in place.
 *   workspace, workspace_bytes   optional device scratch for h (NULL / 0 for
 *       none).  Without it h never leaves the chip (reduced across a
 *       thread-block cluster in distributed shared memory).  With room for
 *       a 256-byte header and one plane of fp32 h (num_tokens * num_slices *
 *       max_rank * 4 bytes; csgmv_qkv_workspace_bytes() covers every batch
 *       and the widest split of K), two kinds of call instead run the shrink and the expand
 *       as two kernels with h in the workspace, which is faster there:
 *       batches of long per-slot runs (128-token tiles, max_rank >= 16),
 *       decode batches (short per-slot runs onto fewer than 32768 columns,
 *       at most 2048 tokens, max_segments <= 512 and max_loras <= 256), and
 *       short per-slot runs with at least 32768 output columns (a
 *       vocabulary-wide lm_head).  The shrink may cut K into parts, one plane
 *       of partial sums each, that the expand adds in part order, so results
 *       do not depend on timing.  csgmv_qkv_path() tells which path a call
 *       takes.  Its contents on entry do
 *       not matter; on return they are unspecified.  It must be 16-byte
 *       aligned and must not overlap any other argument.
 */
CSGMV_API int csgmv_qkv(const void *x, int64_t K, const void *A, const void *B, int64_t N,
              const int32_t *slice_offsets, int num_slices, int max_slice_size, void *base_output,
              void *workspace, size_t workspace_bytes, const csgmv_batch_info *bi, csgmv_stream_t stream);

/*
 * Tuple-form B (base_backend.py run_qkv_lora: qkv_lora_b as a tuple of a q
 * buffer (1, num_lora, output_dim_q, r) and a combined kv buffer
 * (2, num_lora, output_dim_kv, r); run_gate_up_lora: gate_up_lora_b as a tuple
 * of two (num_lora, output_dim, r) buffers).  These are csgmv_expand and
 * csgmv_qkv with B given per slice instead of as one tensor:
 *   B_slices  HOST array of num_slices device pointers; B_slices[j] is bf16
 *             (max_loras, off[j+1] - off[j], R), row 0 being output column
 *             off[j].  For the qkv tuple: {q, kv, kv + max_loras * N_kv * R}.
 * Every slice offset must be a multiple of 64 (CSGMV_ERR_UNSUPPORTED
 * otherwise); everything else, results included, is as the single-tensor call.
 */
CSGMV_API int csgmv_expand_sliced(const void *h, int h_dtype, int64_t ldh, const void *const *B_slices, int64_t N,
                                  const int32_t *slice_offsets, int num_slices, int max_slice_size, void *out,
                                  int accumulate, const csgmv_batch_info *bi, csgmv_stream_t stream);
CSGMV_API int csgmv_qkv_sliced(const void *x, int64_t K, const void *A, const void *const *B_slices, int64_t N,
                               const int32_t *slice_offsets, int num_slices, int max_slice_size, void *base_output,
                               void *workspace, size_t workspace_bytes, const csgmv_batch_info *bi,
                               csgmv_stream_t stream);

/* Kernel paths of csgmv_qkv (csgmv_qkv_path). */
enum {
    CSGMV_PATH_FUSED = 0,       /* one kernel: h reduced across a thread-block cluster, never in memory */
    CSGMV_PATH_DECODE = 1,      /* decode batches: split-K shrink into fp32 planes, then the expand */
    CSGMV_PATH_SMALL_SPLIT = 2, /* short runs onto vocabulary-wide outputs: small-tile shrink, then expand */
    CSGMV_PATH_STREAM = 3       /* 128-token tiles: streaming tcgen05 shrink, then streaming expand */
};

/*
 * The path csgmv_qkv takes for the batch last built into bi, with these
 * shapes (as csgmv_qkv's K, N, slice_offsets, num_slices) and a workspace of
 * workspace_bytes (0 for none).  Host only: reads the capacity and host
 * mirror fields of bi, launches nothing, needs no GPU.  Returns a
 * CSGMV_PATH_* value (CSGMV_PATH_FUSED for an empty batch), or
 * CSGMV_ERR_INVALID_ARG / CSGMV_ERR_UNSUPPORTED as csgmv_qkv would for the
 * same shapes.  Paths other than CSGMV_PATH_FUSED launch two kernels.
 */
CSGMV_API int csgmv_qkv_path(const csgmv_batch_info *bi, int64_t K, int64_t N, const int32_t *slice_offsets,
                             int num_slices, size_t workspace_bytes);

/* Workspace bytes that let csgmv_qkv use its two-kernel paths for any batch
 * of this batch info, with h (fp32) held as partial sums over parts of K
 * (planes of max_tokens * num_slices * max_rank floats) after a 256-byte
 * header: 256 + P * max_tokens * num_slices * max_rank * 4 with P = 4, or
 * P = 32 * min(max_tokens, 2048) / max_tokens when that is more (room for the
 * decode kernels' 32 parts).  A smaller workspace of at least 256 +
 * num_tokens * num_slices * max_rank * 4 bytes also takes the paths, with
 * fewer parts. */
CSGMV_API size_t csgmv_qkv_workspace_bytes(const csgmv_batch_info *bi, int num_slices);

/*
 * csgmv_qkv for callers that cannot allocate device memory when they call it
 * (no counterpart on the pages: an addition of this library).  Some callers
 * cannot call cudaMalloc or a caching allocator at that point (for instance
 * code whose device memory is planned up front by an engine that owns every
 * buffer), so they cannot provide csgmv_qkv's workspace.  This entry point
 * takes the same arguments without one and uses a fixed 32 MiB array in the
 * library's own device memory as the h workspace; the library allocates
 * nothing and frees nothing here either.
 *   - Limit: when csgmv_qkv would take a two-kernel path, the batch's h,
 *     num_tokens * num_slices * max_rank * 4 bytes, and a 256-byte header
 *     must fit in 32 MiB, else CSGMV_ERR_CAPACITY (nothing is launched).  A
 *     batch whose h does not fit but which csgmv_qkv runs as one kernel
 *     (csgmv_qkv_path gives CSGMV_PATH_FUSED even with an unbounded
 *     workspace) runs that way, with no workspace.
 *   - Every GPU that loads the library holds the 32 MiB until the process
 *     exits.
 *   - The first call on each device looks up the array's device address
 *     (cudaGetSymbolAddress, with that device current); make that first call
 *     before capturing the stream.
 *   - All calls share the one array: two calls that may run at the same time
 *     on the GPU (different streams, or unordered graph branches) race on it.
 *     Nothing in it has to start at zero; the shrink writes every h row the
 *     expand reads.
 */
CSGMV_API int csgmv_qkv_static_scratch(const void *x, int64_t K, const void *A, const void *B, int64_t N,
                             const int32_t *slice_offsets, int num_slices, int max_slice_size,
                             void *base_output, const csgmv_batch_info *bi, csgmv_stream_t stream);

/*
 * Embedding LoRA-A gather (base_backend.py run_lora_a_embedding;
 * chunked_backend.py run_lora_a_embedding, which takes no extra-token
 * embeddings): for token t on slot w with rank r,
 *     out[t][k] = A_emb[w][k][input_ids[t]]  for k < r,  0 for r <= k < rank.
 *   input_ids int32 (s,), s = bi->num_tokens;  A_emb bf16 (max_loras, rank, vocab_size)
 *   out bf16 (s, rank);  1 <= rank <= 1024.
 * An id outside [0, vocab_size) sets CSGMV_STATUS_BAD_TOKEN_ID and leaves
 * that row 0.  Bit-exact copy; no arithmetic.
 */
CSGMV_API int embedding_lora_a(const int32_t *input_ids, const void *A_emb, int64_t vocab_size, int rank,
                     void *out, const csgmv_batch_info *bi, csgmv_stream_t stream);

/*
 * Embedding LoRA-A gather with extra tokens (base_backend.py
 * run_lora_a_embedding with extra_embeddings: tokens with ids >= vocab_size
 * are extra tokens the adapter adds beyond the base vocabulary).  For token t
 * on slot w with rank r:
 *     out[t][k] = A_emb[w][k][id]                    0 <= id < vocab_size
 *     out[t][k] = extra_embeddings[w][id - vocab_size][k]
 *                                 vocab_size <= id < vocab_size + num_extra_tokens
 * for k < r, and 0 for r <= k < rank.
 *   extra_embeddings  bf16 (max_loras, num_extra_tokens, rank); may be NULL
 *                     when num_extra_tokens = 0 (then this is embedding_lora_a)
 *   other arguments as embedding_lora_a; out must be 16-byte aligned when rank
 *   is a multiple of 8.
 * An id outside [0, vocab_size + num_extra_tokens) sets
 * CSGMV_STATUS_BAD_TOKEN_ID and leaves that row 0.  Bit-exact copy.
 */
CSGMV_API int embedding_lora_a_extra(const int32_t *input_ids, const void *A_emb, int64_t vocab_size, int rank,
                                     const void *extra_embeddings, int64_t num_extra_tokens, void *out,
                                     const csgmv_batch_info *bi, csgmv_stream_t stream);

/*
 * embedding_lora_a_extra with A_emb stored transposed: A_emb_t bf16
 * (max_loras, vocab_size, rank), A_emb_t[w][id][k] = A_emb[w][k][id].  The
 * (max_loras, rank, vocab_size) layout of the pages puts each of a token's
 * rank values in its own 32-byte memory sector; here they are one
 * contiguous row, so the gather reads rank * 2 bytes per token instead of
 * rank sectors.  A caller transposes each adapter once when it loads it
 * (csgmv_transpose_embedding).  Results are identical to
 * embedding_lora_a_extra on the untransposed table.  An addition of this
 * library (the load-time layout is not on the pages).
 */
CSGMV_API int embedding_lora_a_transposed(const int32_t *input_ids, const void *A_emb_t, int64_t vocab_size,
                                          int rank, const void *extra_embeddings, int64_t num_extra_tokens,
                                          void *out, const csgmv_batch_info *bi, csgmv_stream_t stream);

/*
 * A_emb_t[w][v][k] = A_emb[w][k][v] for w < num_loras (both bf16, device):
 * the load-time layout of embedding_lora_a_transposed.  Asynchronous on
 * stream; the two buffers must not overlap.  1 <= rank <= 1024.
 */
CSGMV_API int csgmv_transpose_embedding(const void *A_emb, int64_t num_loras, int rank, int64_t vocab_size,
                                        void *A_emb_t, csgmv_stream_t stream);

/*
 * Extra-token embedding (base_backend.py run_extra_token_embedding): in the
 * (s, embed_dim) output of the base embedding, the row of every token t on
 * slot w with vocab_size <= id < vocab_size + num_extra_tokens becomes
 *     output[t][:] = extra_embeddings[w][id - vocab_size][:]
 * (the base vocabulary has no row for it); rows of ids below vocab_size are
 * not touched.
 *   input_ids         int32 (s,), s = bi->num_tokens (tokens mapped to slots
 *                     by the batch info)
 *   output            bf16 (s, embed_dim), updated in place
 *   extra_embeddings  bf16 (max_loras, num_extra_tokens, embed_dim)
 * Both bf16 tensors must be 16-byte aligned when embed_dim is a multiple of
 * 8.  An id outside [0, vocab_size + num_extra_tokens) sets
 * CSGMV_STATUS_BAD_TOKEN_ID and leaves the row untouched; num_extra_tokens = 0
 * does nothing.  Bit-exact copy.
 */
CSGMV_API int extra_token_embedding(const int32_t *input_ids, void *output, int64_t embed_dim,
                                    const void *extra_embeddings, int64_t num_extra_tokens, int64_t vocab_size,
                                    const csgmv_batch_info *bi, csgmv_stream_t stream);

/* ------------------------------------------------------------------------
 * The serving step around the adapters: a paged K/V cache, attention of a
 * tree of drafted tokens over it, verification of the drafts, and the cache's
 * page bookkeeping (additions of this library; the pages stop at the
 * projections).  The conventions above hold: device pointers, the given
 * stream, nothing allocated, nothing synchronized.
 * ------------------------------------------------------------------------ */

/* csgmv_kv_cache.dtype also takes IEEE half. */
enum { CSGMV_DTYPE_F16 = 2 };

/* Bits of csgmv_kv_cache.status and of the status words below.  Device-side
 * problems are OR-ed in and the offending request is left out; a status word
 * is never reset by the library. */
enum {
    CSGMV_KV_STATUS_BAD_SEQ = 1,   /* sequence slot out of range, used twice, or (fork) not empty */
    CSGMV_KV_STATUS_BAD_PAGE = 2,  /* page number out of range, or a reference count that would go below zero */
    CSGMV_KV_STATUS_CAPACITY = 4,  /* no free pages left, or a row of the page table is full */
    CSGMV_KV_STATUS_BAD_LENS = 8,  /* negative or inconsistent lengths */
    CSGMV_KV_STATUS_BAD_TREE = 16, /* a parent that does not come before its child, a bad node number, or a node
                                      under two parents */
    CSGMV_KV_STATUS_BAD_TOKEN = 32, /* a token outside the vocabulary, or a distribution without mass */
    CSGMV_KV_STATUS_BAD_VALUE = 64, /* csgmv_process_logits: a request's factor, list of biases or mask that is not one */
    CSGMV_KV_STATUS_TIMEOUT = 1 << 30 /* csgmv_tree_attention: a bounded wait inside the kernel ran out, the call's
                                         results are meaningless; while the bit is set its calls give no output */
};

/*
 * A paged K/V cache: num_pages pages of page_size tokens for every layer,
 * handed out to at most max_seqs sequences.  Element (layer l, page p, head
 * h, token slot t, d) of k_pages and of v_pages is at
 *     l * layer_stride + p * page_stride + h * head_stride + t * token_stride + d
 * (strides in elements, multiples of 8; no two elements share a place).  Token i
 * of sequence s is in slot i % page_size of page
 * page_table[s * max_pages_per_seq + i / page_size].
 * page_refs[p] counts the sequences that hold page p; a page is free when it
 * is 0, and pages are given out lowest first.  The caller allocates every
 * buffer; an empty cache has seq_lens = 0, page_refs = 0 and page_table = -1.
 */
typedef struct csgmv_kv_cache {
    void *k_pages, *v_pages;
    int32_t *page_table; /* [max_seqs][max_pages_per_seq]; -1 past a sequence's pages */
    int32_t *seq_lens;   /* [max_seqs] tokens held */
    int32_t *page_refs;  /* [num_pages] */
    int32_t *scratch;    /* [csgmv_kv_scratch_ints()]; contents do not matter between calls */
    int32_t *status;     /* [1] CSGMV_KV_STATUS_* bits */
    int64_t layer_stride, page_stride, head_stride, token_stride;
    int32_t dtype;       /* CSGMV_DTYPE_BF16 or CSGMV_DTYPE_F16 */
    int32_t num_layers, num_pages, page_size, num_kv_heads, head_dim, max_seqs, max_pages_per_seq;
} csgmv_kv_cache;

/* int32 entries of csgmv_kv_cache.scratch.  Host only; 0 for negative sizes. */
CSGMV_API int64_t csgmv_kv_scratch_ints(int num_pages, int max_seqs);

/*
 * Appends tokens to sequences, in every layer.  Request b appends
 * accept_len[b] tokens to sequence seq_slots[b] (b itself when seq_slots is
 * NULL): its j-th is row tree_indptr[b] + accept_index[b * accept_width + j]
 * of k_new and v_new.  Pages are taken as needed; a partly filled last page
 * that another sequence holds too is first replaced by a copy of its own.
 *   k_new, v_new   dtype of the cache; element (layer l, row t, head h, d) at
 *                  l * new_layer_stride + t * new_token_stride + h * new_head_stride + d
 *                  (strides in elements, multiples of 8); num_tokens rows
 *   accept_index   [bs][accept_width]; node numbers inside the request, each
 *                  in [0, tree_indptr[b+1] - tree_indptr[b]); NULL for 0, 1, 2, ...
 *                  (accept_width is then ignored)
 *   accept_len     [bs]
 * A request with a bad slot, length or node number, or without room in its
 * row of the page table, is left out; when the free pages do not suffice for
 * the whole batch nothing is appended at all (CSGMV_KV_STATUS_CAPACITY).
 * A sequence may appear once in a batch.  bs <= max_seqs, accept_width <= 2^30.  The lists may not lie
 * in the cache's bookkeeping or scratch (nor csgmv_kv_fork's).
 */
CSGMV_API int csgmv_kv_commit(const csgmv_kv_cache *kv, const void *k_new, const void *v_new, int64_t new_layer_stride,
                              int64_t new_token_stride, int64_t new_head_stride, int64_t num_tokens,
                              const int32_t *accept_index, int accept_width, const int32_t *accept_len,
                              const int32_t *tree_indptr, const int32_t *seq_slots, int bs, csgmv_stream_t stream);

/*
 * children[i] becomes a copy of sequence parents[i], for i < n: whole pages
 * are shared (their count goes up), a partly filled last page is copied into
 * a fresh one in every layer.  A child must be empty, may appear once, and
 * may not be a parent in the same call; an entry that breaks this is left out
 * (CSGMV_KV_STATUS_BAD_SEQ).  Without enough free pages nothing is forked.
 * n <= max_seqs.
 */
CSGMV_API int csgmv_kv_fork(const csgmv_kv_cache *kv, const int32_t *parents, const int32_t *children, int n,
                            csgmv_stream_t stream);

/*
 * Cuts sequence seqs[i] back to keep_lens[i] tokens (to none when keep_lens
 * is NULL) and gives up its pages past them: their counts go down, their
 * page-table entries become -1.  A sequence no longer than that is left as it
 * is.  A page that stays partly used by it may then be shared; appending to the
 * sequence copies such a page first (csgmv_kv_commit).  A sequence listed
 * twice is cut to the smaller length.  n <= max_seqs.
 */
CSGMV_API int csgmv_kv_free(const csgmv_kv_cache *kv, const int32_t *seqs, const int32_t *keep_lens, int n,
                            csgmv_stream_t stream);

/*
 * Moves every live page whose number is at least the count of live pages into
 * a hole below it (k-th such page into the k-th hole), in every layer, and
 * rewrites page_refs and the page tables: afterwards the live pages are
 * 0 .. live - 1.
 */
CSGMV_API int csgmv_kv_compact(const csgmv_kv_cache *kv, csgmv_stream_t stream);

/*
 * Copies the contents of page src[i] to page dst[i] in every layer, i < n.
 * No page may be both a source and a destination or a destination twice;
 * pairs with a page out of range are left out (CSGMV_KV_STATUS_BAD_PAGE).
 */
CSGMV_API int csgmv_kv_copy_pages(const csgmv_kv_cache *kv, const int32_t *src, const int32_t *dst, int n,
                                  csgmv_stream_t stream);

/*
 * Attention of the drafted tokens of each request over its sequence and its
 * own tree.  Request b owns rows [tree_indptr[b], tree_indptr[b+1]) of q,
 * k_new, v_new and out, and sequence s = seq_slots[b] (b when NULL) of the
 * cache.  For row t of the request, query head h and kv head
 * g = h / (num_q_heads / num_kv_heads),
 *     a_i = scale * q[t][h] . K_i,   out[t][h] = sum_i softmax(a)_i V_i,
 *     lse[t][h] = log sum_i exp(a_i)
 * over the tokens i of sequence s in layer `layer` of the cache, and over the
 * request's own rows j whose bit is set in row t of `mask`.  A row that sees
 * no token gives out = 0 and lse = -inf.  What is masked has no influence,
 * whatever it holds (infinities and NaN too, and slots past a sequence's end);
 * an infinity in a V that a row does see gives an infinity or NaN.
 *   q, out         dtype of the cache; element (t, h, d) at t * q_token_stride
 *                  + h * q_head_stride + d (out_* for out; multiples of 8)
 *   k_new, v_new   element (t, g, d) at t * new_token_stride + g * new_head_stride + d
 *   lse            f32 [num_tokens][num_q_heads], or NULL
 *   mask           int32 [num_tokens][mask_words]: bit j % 32 of word j / 32 of
 *                  row t lets t see row j of its request; a request has at most
 *                  32 * mask_words rows.  NULL: row t sees rows 0 .. t (any
 *                  number of rows: plain decoding and prompts)
 * head_dim 64 or 128; num_q_heads a multiple of num_kv_heads, at most 128
 * times it; page_size a power of two >= 8.  One row for each request is plain
 * decoding.  Sums are fp32; before they meet V the softmax weights are
 * rounded: bfloat16's to a pair of 16 bits, half's to one half of 11 bits, as
 * many as out has.  (The rows of a request and kv head, tokens times query heads,
 * are taken 128 at a time: where that leaves 16 or fewer, plain decoding for
 * instance, half's weights are a pair of 22 bits.)  Results do not depend on
 * timing.  A page number out of range sets CSGMV_KV_STATUS_BAD_PAGE and makes
 * its request's rows meaningless; other bad requests are left out (their rows
 * of out and lse stay as they are).  bs <= 16000;
 * num_tokens times the query heads of a kv head <= 2^30.  A batch of more than
 * some four minutes of work on the whole GPU (2^40 units of 64 clocks of an SM,
 * of which 128 rows against 128 tokens take 16 to 45, so at least 4 * 10^14
 * pairs of a row and a token) sets CSGMV_KV_STATUS_CAPACITY and gives no output.
 *   workspace      csgmv_tree_attention_workspace_bytes(); contents do not matter
 * out, lse and workspace may not overlap one another, tree_indptr, seq_slots or
 * the cache's bookkeeping, nor rows of out each other.
 */
CSGMV_API int csgmv_tree_attention(const void *q, int64_t q_token_stride, int64_t q_head_stride, int num_q_heads,
                                   const void *k_new, const void *v_new, int64_t new_token_stride,
                                   int64_t new_head_stride, const csgmv_kv_cache *kv, int layer,
                                   const int32_t *tree_indptr, const int32_t *seq_slots, int bs, int64_t num_tokens,
                                   const int32_t *mask, int mask_words, float scale, void *out,
                                   int64_t out_token_stride, int64_t out_head_stride, float *lse, void *workspace,
                                   size_t workspace_bytes, csgmv_stream_t stream);

/* Workspace bytes of csgmv_tree_attention: independent of the batch. */
CSGMV_API size_t csgmv_tree_attention_workspace_bytes(const csgmv_kv_cache *kv, int num_q_heads);

/*
 * Derived fields of a batch of draft trees.  Node i of request b is row
 * tree_indptr[b] + i; parents[row] is its parent's number inside the request,
 * smaller than i, and -1 for node 0 (the root: the last accepted token) only.
 *   mask          [num_nodes][mask_words]: the node itself and its ancestors
 *                 (csgmv_tree_attention's mask)
 *   depth         [num_nodes]: 0 at the root (a token's position is its
 *                 sequence's length plus its depth)
 *   first_child, next_sibling   [num_nodes]: node numbers in increasing order
 *                 of siblings, -1 for none
 * A request with a bad parent or more than 32 * mask_words nodes gets an empty
 * mask, depth 0 and no children (CSGMV_KV_STATUS_BAD_TREE).  mask_words <= 8.
 */
CSGMV_API int csgmv_build_draft_tree(const int32_t *parents, const int32_t *tree_indptr, int bs, int64_t num_nodes,
                                     int mask_words, int32_t *mask, int32_t *depth, int32_t *first_child,
                                     int32_t *next_sibling, int32_t *status, csgmv_stream_t stream);

/*
 * Verification of drafted tokens: a walk from the root of each tree that
 * keeps a prefix of accepted tokens and draws one more, so that every token is
 * distributed as the target says.  At node c with target distribution
 * p = target_probs[c] and children x_1, x_2, ... in order:
 *   - with draft_probs (children drawn independently from q = draft_probs[c]):
 *     r = p, z = 1; child k is accepted if (u_k * q(x_k)) * z < r(x_k), with
 *     u_k = accept_uniforms of the child; otherwise r = max(r - z * q, 0),
 *     z = sum r, and the next child is tried while z > 0;
 *   - without (children chosen by the drafter, distinct tokens): child k is
 *     accepted if u < p(x_1) + ... + p(x_k), with u = accept_uniforms of c;
 *     otherwise r = p without the children's tokens (a token that an earlier
 *     sibling has already is passed over).
 * The walk goes on at an accepted child.  When no child is accepted, next_token
 * is the first token whose running sum of r exceeds sample_uniforms[b] times
 * the total (of p where r is empty).
 * Sums and the comparisons of sums are exact: a probability, clamped to
 * [0, 1], counts in whole steps of 2^-44 (rounded down), a uniform number in
 * steps of 2^-44 against a sum of p and of 2^-31 for the draw; r, u * q * z
 * are fp32, each operation rounded.  So results do not depend on the order of
 * summation.
 *   target_probs, draft_probs   f32, row of a node at target_stride / draft_stride
 *                  elements; draft_probs may be NULL
 *   draft_tokens   [num_nodes] (the root's is not used)
 *   first_child, next_sibling   from csgmv_build_draft_tree (a number that is
 *                  not above its node's own, or past the request, ends a list)
 *   accept_uniforms [num_nodes], sample_uniforms [bs]   in [0, 1)
 *   accept_index   [bs][accept_width]: node numbers of the accepted path, the
 *                  root first, then -1
 *   accept_len     [bs]: nodes on the path (1 when no draft was accepted)
 *   next_token     [bs]
 * A request without nodes, with a node in two nodes' lists (BAD_TREE), or whose
 * path is longer than accept_width (CSGMV_KV_STATUS_CAPACITY), gets accept_len
 * = 0 and next_token = -1; one whose last distribution has no mass (BAD_TOKEN)
 * next_token = -1 only.
 * 1 <= vocab_size <= 2^18, accept_width <= 2^30.  No output may overlap an input.
 */
CSGMV_API int csgmv_verify_drafts(const float *target_probs, int64_t target_stride, const float *draft_probs,
                                  int64_t draft_stride, const int32_t *draft_tokens, const int32_t *tree_indptr,
                                  const int32_t *first_child, const int32_t *next_sibling,
                                  const float *accept_uniforms, const float *sample_uniforms, int bs,
                                  int64_t num_nodes, int vocab_size, int32_t *accept_index, int accept_width,
                                  int32_t *accept_len, int32_t *next_token, int32_t *status, csgmv_stream_t stream);

/* ------------------------------------------------------------------------
 * What a decoder does between the projections, the attention and the
 * verification (additions of this library as well): residual and norms,
 * rotary positions, appending to the cache layer by layer, logits to
 * probabilities.  The conventions above hold, except that pointers need only
 * their elements' alignment (16 bytes are faster).
 * ------------------------------------------------------------------------ */

/* Kinds of norm: none, root mean square, and centred ("layer"). */
enum { CSGMV_NORM_NONE = 0, CSGMV_NORM_RMS = 1, CSGMV_NORM_LAYER = 2 };

/* A norm over a row v of `hidden` elements:
 *     RMS    v * rsqrt(mean(v^2) + eps) * weight + bias
 *     LAYER  (v - mean(v)) * rsqrt(mean((v - mean(v))^2) + eps) * weight + bias
 * weight and bias have the row's type (dtype of the call); NULL: 1 and 0. */
typedef struct csgmv_norm {
    const void *weight, *bias;
    float eps;
    int32_t kind; /* CSGMV_NORM_* */
} csgmv_norm;

/*
 * Adds a block's output x to the residual stream and norms the sum for the
 * next block: for every row t,
 *     r'[t] = residual_scale * r[t] + gate[t] * post(x[t]),   out[t] = pre(r'[t]).
 *   x, out, gate   dtype (CSGMV_DTYPE_BF16, _F16 or _F32); rows of `hidden`
 *                  dense elements, *_stride elements apart
 *   gate           NULL: 1; gate_stride 0: one row for all
 *   residual, residual_out   dtype or f32 (residual_dtype); residual NULL: r = 0;
 *                  residual_out NULL: r' is not written
 *   pre            NULL or kind NONE with out NULL: only r' is made
 *   post           NULL: x as it is
 * r' enters pre with 32 bits, not as it is rounded for residual_out.  Sums are
 * f32.  out and residual_out may each be x, residual or gate (same address and
 * stride, types of one size); otherwise no output overlaps an input or the other
 * output.
 * 1 <= hidden <= 16384.
 */
CSGMV_API int csgmv_add_norm(const void *x, int64_t x_stride, int dtype, const void *residual, int64_t residual_stride,
                             int residual_dtype, const void *gate, int64_t gate_stride, const csgmv_norm *post,
                             const csgmv_norm *pre, float residual_scale, int64_t num_tokens, int hidden,
                             void *residual_out, int64_t residual_out_stride, void *out, int64_t out_stride,
                             csgmv_stream_t stream);

/*
 * Rotary positions.  Elements u, v of pair i (0 <= i < rotary_dim / 2) of a head
 * at position p become
 *     scale * (u cos a - v sin a),  scale * (u sin a + v cos a),  a = p * f_i
 * (f_i radians a position); the other elements of the head stay as they are.
 *   interleaved  1: pair i is elements 2 i and 2 i + 1; 0: elements i and
 *                i + rotary_dim / 2
 *   turns        device, [rotary_dim / 2]: f_i in units of 2^-64 turns, from
 *                csgmv_rope_turns().  p * turns[i] in 64 bits wraps at whole turns, so
 *                angles of far positions keep all their bits.
 */
typedef struct csgmv_rope {
    const uint64_t *turns;
    float scale;
    int32_t rotary_dim; /* even, at most head_dim */
    int32_t interleaved;
} csgmv_rope;

/* turns[i] = round(2^64 * freq[i] / (2 pi)) modulo 2^64 (freq in radians a
 * position, finite), rounded once; 2 pi is the double next to it, which is off by
 * 2^-54 of it, less than a double's own rounding.  -freq gives -turns.  Host only. */
CSGMV_API int csgmv_rope_turns(const double *freq, int n, uint64_t *turns);

/*
 * Turns the heads of queries and keys by the positions of their tokens.
 *   dtype       CSGMV_DTYPE_BF16, _F16 or _F32
 *   q, k        element (t, h, d) at t * token_stride + h * head_stride + d; k (with
 *               num_k_heads 0) or q (with num_q_heads 0) may be NULL
 *   positions   [num_tokens], any int32
 *   q_out, k_out  may be q and k (same address and strides); otherwise no
 *               output overlaps an input, nor the other output
 *   inverse     1: by the negative angles, times scale: the gradient of the
 *               inputs from that of the outputs
 * Products are f32, rounded once.  1 <= head_dim <= 1024; at most 4096 heads of each;
 * strides of at most 2^40 elements (as in the calls below and above).
 */
CSGMV_API int csgmv_rotary(const csgmv_rope *rope, int dtype, int head_dim, const int32_t *positions,
                           int64_t num_tokens, const void *q, int64_t q_token_stride, int64_t q_head_stride,
                           int num_q_heads, const void *k, int64_t k_token_stride, int64_t k_head_stride,
                           int num_k_heads, void *q_out, int64_t qo_token_stride, int64_t qo_head_stride, void *k_out,
                           int64_t ko_token_stride, int64_t ko_head_stride, int inverse, csgmv_stream_t stream);

/*
 * Makes room for add_lens[b] more tokens (all of its rows when add_lens is
 * NULL) in sequence seq_slots[b] (b when NULL) of the cache: takes pages, copies
 * a partly filled last page that another sequence holds too, raises seq_lens.
 * What csgmv_kv_commit does but for the contents, which csgmv_kv_append brings
 * layer by layer.  Request b owns rows [tree_indptr[b], tree_indptr[b+1]); its
 * first add_lens[b] rows are the tokens, in order.
 *   slots        int64 [num_tokens]: page * page_size + slot of a row's token; -1
 *                for a row that is not appended
 *   positions    [num_tokens]: the token's index in its sequence; 0 where slots is -1
 *   lens_before  [max_seqs] or NULL: seq_lens as they were.  With them in place of
 *                seq_lens, csgmv_tree_attention sees the cache without the new
 *                tokens, which it takes from k_new and v_new (prompts).  With
 *                seq_lens and a mask of zeros, a single new token is seen from the
 *                cache (plain decoding).
 * Requests are left out as by csgmv_kv_commit.  A tree_indptr that decreases or
 * leaves [0, num_tokens] (CSGMV_KV_STATUS_BAD_LENS), or too few free pages
 * (CSGMV_KV_STATUS_CAPACITY): nothing is extended, all slots are -1.  bs <=
 * max_seqs.  slots holds until a page is moved, shared or given up
 * (csgmv_kv_compact, _fork, _free of the sequence): bring the contents before.
 * The call's buffers overlap neither one another nor the cache's.
 */
CSGMV_API int csgmv_kv_extend(const csgmv_kv_cache *kv, const int32_t *add_lens, const int32_t *tree_indptr,
                              const int32_t *seq_slots, int bs, int64_t num_tokens, int64_t *slots, int32_t *positions,
                              int32_t *lens_before, csgmv_stream_t stream);

/*
 * Writes the rows of k and v into their slots of one layer of the cache, k
 * turned by its positions on the way, and turns q beside them.
 *   rope        NULL: nothing is turned (positions may then be NULL)
 *   q, k, v     dtype of the cache, strided as in csgmv_rotary; k and v have
 *               the cache's heads and head_dim; q may be NULL (num_q_heads 0)
 *   slots       [num_tokens], from csgmv_kv_extend; rows of a slot outside
 *               [0, num_pages * page_size) are left out (-1 without a word, others with
 *               CSGMV_KV_STATUS_BAD_PAGE): nothing is written for them
 *   q_out       the turned queries; may be q
 *   k_out       the turned keys, or NULL; may be k
 * A slot that is listed twice holds one of its rows' elements, which is not said.
 * No output overlaps an input (but q_out and k_out as said), another output, the
 * cache's pages or its bookkeeping.
 */
CSGMV_API int csgmv_kv_append(const csgmv_kv_cache *kv, int layer, const csgmv_rope *rope, const int32_t *positions,
                              const int64_t *slots, int64_t num_tokens, const void *q, int64_t q_token_stride,
                              int64_t q_head_stride, int num_q_heads, const void *k, int64_t k_token_stride,
                              int64_t k_head_stride, const void *v, int64_t v_token_stride, int64_t v_head_stride,
                              void *q_out, int64_t qo_token_stride, int64_t qo_head_stride, void *k_out,
                              int64_t ko_token_stride, int64_t ko_head_stride, csgmv_stream_t stream);

/*
 * How often each sequence holds each token.  counts[s * vocab_size + v] is the
 * number of times that sequence s gave token v, plus 2^30 if its prompt has it;
 * seen[s * vocab_size + i], i < num_seen[s], lists the tokens whose count is not
 * zero, each once, in no certain order.  The caller allocates the buffers; all
 * zero (seen: anything) is empty.
 */
typedef struct csgmv_token_counts {
    int32_t *counts, *seen; /* [max_seqs][vocab_size] */
    int32_t *num_seen;      /* [max_seqs] */
    int32_t *status;        /* [1] CSGMV_KV_STATUS_* bits */
    int32_t max_seqs, vocab_size;
} csgmv_token_counts;

/*
 * Counts tokens of request b for sequence seq_slots[b] (b when NULL): the first
 * accept_len[b] (NULL: all) of rows tree_indptr[b] + accept_index[b * accept_width
 * + j] (NULL: j) of tokens: what csgmv_kv_commit appends for the same lists.
 * prompt 1: they are the sequence's prompt.  A sequence may come several times,
 * and so may a token.  A request with a bad sequence, length or node is left out;
 * a token outside the vocabulary is (CSGMV_KV_STATUS_BAD_TOKEN).  A sequence may
 * give a token at most 2^30 - 1 times.  accept_width <= 2^30.
 */
CSGMV_API int csgmv_count_tokens(const csgmv_token_counts *counts, const int32_t *tokens, int64_t num_tokens,
                                 const int32_t *tree_indptr, const int32_t *accept_index, int accept_width,
                                 const int32_t *accept_len, const int32_t *seq_slots, int bs, int prompt,
                                 csgmv_stream_t stream);

/* Empties the sequences seqs[i], i < n. */
CSGMV_API int csgmv_count_reset(const csgmv_token_counts *counts, const int32_t *seqs, int n, csgmv_stream_t stream);

/* children[i] becomes a copy of parents[i], i < n.  A child must be empty, may
 * appear once, and may not be a parent in the same call; an entry that breaks
 * this is left out (CSGMV_KV_STATUS_BAD_SEQ).  n <= max_seqs. */
CSGMV_API int csgmv_count_fork(const csgmv_token_counts *counts, const int32_t *parents, const int32_t *children,
                               int n, csgmv_stream_t stream);

/*
 * What csgmv_process_logits does to a row of request b.  Any pointer may be
 * NULL: then that step is left out.
 *   repetition, frequency, presence, temperature   [bs]; repetition > 0 and
 *                 temperature >= 0, both finite, none NaN
 *   bias_tokens, bias_values   entries [bias_indptr[b], bias_indptr[b+1]) are
 *                 request b's, in increasing order of their tokens (a token may
 *                 come again: the values are added in turn); bias_total entries in all, at
 *                 most 2^30
 *   allow         [num_allow][allow_words]: bit v % 32 of word v / 32 lets token v
 *                 through; allow_words >= vocab_size / 32, rounded up
 *   allow_index   [num_tokens]: the row of allow for each row of logits, or -1
 *                 for none
 */
typedef struct csgmv_logit_rules {
    const csgmv_token_counts *counts; /* host pointer; NULL: only a row's own branch counts */
    const float *repetition, *frequency, *presence, *temperature;
    const int32_t *bias_indptr, *bias_tokens;
    const float *bias_values;
    const int32_t *allow, *allow_index;
    int64_t bias_total;
    int32_t num_allow, allow_words;
    int32_t *status; /* [1] CSGMV_KV_STATUS_* bits */
} csgmv_logit_rules;

/*
 * Logits of drafted tokens to what csgmv_verify_drafts takes.  Request b owns
 * rows [tree_indptr[b], tree_indptr[b+1]) and sequence seq_slots[b] (b when
 * NULL) of the counts.  With c_v the number of times that the sequence gave v
 * (counts), plus those that the row's own branch has it (rows j of the request
 * whose bit is set in the row's mask: draft_tokens), for every token v of row t
 *     z = logits[t][v]
 *     z = z > 0 ? z / repetition : z * repetition   if c_v > 0 or v is in the prompt
 *     z = z - frequency * c_v - presence * [c_v > 0]
 *     z = z + biases of v
 *     z = -infinity                                 if v is not allowed
 * and, with softmax, out[t] = exp((z - max z) / temperature) / sum of these; where
 * the temperature is 0, 1 at the lowest v with the largest z and 0 elsewhere.
 * Each step of z is rounded to f32.  A row with nothing but -infinity gives zeros
 * (verification draws nothing from it); one with a NaN, or whose largest z is
 * infinite (but at temperature 0), NaN everywhere.  What is not allowed has no
 * influence, whatever it holds.
 *   logits      dtype (CSGMV_DTYPE_BF16, _F16 or _F32); rows of vocab_size, logits_stride
 *               elements apart
 *   out         f32, rows out_stride elements apart; may be logits when those are f32
 *               (same address and stride), else it overlaps no input
 *   mask        [num_tokens][mask_words] as csgmv_build_draft_tree writes it; NULL,
 *               like draft_tokens NULL: no branch
 * A request with a bad sequence, length, factor or list of biases, and a row
 * with a bad allow_index, is left out: its rows of out stay as they are, and so do
 * those of no request.  A drafted token or a bias outside the vocabulary counts
 * for nothing (CSGMV_KV_STATUS_BAD_TOKEN).
 * 1 <= vocab_size <= 2^18, mask_words <= 8, num_tokens < 2^24, bs <= 2^30.
 */
CSGMV_API int csgmv_process_logits(const void *logits, int dtype, int64_t logits_stride, const int32_t *tree_indptr,
                                   const int32_t *seq_slots, int bs, int64_t num_tokens, int vocab_size,
                                   const csgmv_logit_rules *rules, const int32_t *draft_tokens, const int32_t *mask,
                                   int mask_words, int softmax, float *out, int64_t out_stride, csgmv_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* CSGMV_H */
