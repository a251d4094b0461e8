// Host-side argument checks of the C ABI's serving calls: what serving_api.cu
// and step_api.cu share.
#pragma once
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

// The longest list that a kernel's 32-bit index walks by steps of a CTA's threads.
[[maybe_unused]] constexpr int kMaxList = 1 << 30;

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
[[maybe_unused]] bool overlaps_plan(const csgmv_kv_cache *kv, const int32_t *list, size_t n) {
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

[[maybe_unused]] int check_new(const void *k, const void *v, int64_t ts, int64_t hs) {
    if (!k || !v) return fail(CSGMV_ERR_INVALID_ARG, "k_new / v_new is NULL");
    if (!aligned16(k) || !aligned16(v)) return fail(CSGMV_ERR_INVALID_ARG, "k_new / v_new must be 16-byte aligned");
    if (ts % 8 || hs % 8 || ts <= 0 || hs <= 0)
        return fail(CSGMV_ERR_INVALID_ARG, "k_new / v_new strides must be positive multiples of 8");
    return CSGMV_OK;
}

cudaStream_t st(csgmv_stream_t s) { return reinterpret_cast<cudaStream_t>(s); }

}  // namespace
