// C ABI of what a decoder does between the projections, the attention and the
// verification: argument checks on the host, then the launches of each call
// on the caller's stream.  Nothing here allocates, frees or synchronizes.
#include <cmath>

#include "serving_checks.h"
#include "elements.cuh"
#include "step.h"

namespace {

bool known_type(int dtype) { return dtype == CSGMV_DTYPE_BF16 || dtype == CSGMV_DTYPE_F16 || dtype == CSGMV_DTYPE_F32; }
bool aligned_to(const void *p, int bytes) { return reinterpret_cast<uintptr_t>(p) % bytes == 0; }

// A tensor of rows (t, h), `row` dense elements each, as the overlap checks see
// it.  Strides and sizes in bytes.
struct Rows {
    const void *at;
    int64_t n, ts, heads, hs, row;
};
Rows rows_of(const void *at, int bytes, int64_t n, int64_t ts, int64_t heads, int64_t hs, int64_t row) {
    if (!at || n <= 0 || heads <= 0) return {nullptr, 0, 0, 0, 0, 0};
    return {at, n, ts * bytes, heads, hs * bytes, row * bytes};
}
Rows plain(const void *at, size_t bytes) { return {bytes ? at : nullptr, 1, 0, 1, 0, (int64_t)std::min<size_t>(bytes, INT64_MAX)}; }

bool same(const Rows &a, const Rows &b) {
    return a.at == b.at && a.n == b.n && a.heads == b.heads && a.row == b.row && (a.n == 1 || a.ts == b.ts) &&
           (a.heads == 1 || a.hs == b.hs);
}

// Whether two tensors may share bytes: their ranges meet, and they are not
// slices side by side of rows at one stride (as q and k are of a projection's
// output).
bool meet(const Rows &a, const Rows &b) {
    if (!a.at || !b.at) return false;
    using Wide = unsigned __int128;
    struct Flat {
        Wide lo, span, inner;
        int64_t outer;
    };
    auto flat = [](const Rows &r) {
        const int64_t ts = r.n > 1 ? r.ts : 0, hs = r.heads > 1 ? r.hs : 0;
        const bool tokens = ts >= hs;  // the longer stride is the outer one
        const Wide inner = (Wide)(tokens ? r.heads - 1 : r.n - 1) * (tokens ? hs : ts) + r.row;
        const Wide span = (Wide)(tokens ? r.n - 1 : r.heads - 1) * (tokens ? ts : hs) + inner;
        return Flat{reinterpret_cast<uintptr_t>(r.at), span, inner, tokens ? ts : hs};
    };
    const Flat x = flat(a), y = flat(b);
    if (x.lo + x.span <= y.lo || y.lo + y.span <= x.lo) return false;
    if (x.outer > 0 && x.outer == y.outer && x.inner <= (Wide)x.outer && y.inner <= (Wide)x.outer) {
        const Wide S = x.outer, d = y.lo >= x.lo ? (y.lo - x.lo) % S : (S - (x.lo - y.lo) % S) % S;
        return !(d >= x.inner && d + y.inner <= S);
    }
    return true;
}

// An output may be the input of the same place, element by element, or apart from it.
bool in_place_or_apart(const Rows &out, const Rows &in) { return same(out, in) || !meet(out, in); }

// turns and the rest of a rope for heads of head_dim elements; 0 or an error.
int check_rope(const csgmv_rope *rope, int head_dim) {
    if (rope->rotary_dim < 0 || rope->rotary_dim % 2 || rope->rotary_dim > head_dim)
        return fail(CSGMV_ERR_INVALID_ARG, "rotary_dim %d must be even and at most head_dim %d", rope->rotary_dim, head_dim);
    if (rope->rotary_dim && (!rope->turns || !aligned_to(rope->turns, 8)))
        return fail(CSGMV_ERR_INVALID_ARG, "turns is NULL or not 8-byte aligned");
    if (rope->interleaved != 0 && rope->interleaved != 1)
        return fail(CSGMV_ERR_INVALID_ARG, "interleaved must be 0 or 1");
    if (!(rope->scale - rope->scale == 0.0f)) return fail(CSGMV_ERR_INVALID_ARG, "a rope's scale must be finite");
    return CSGMV_OK;
}

constexpr int64_t kMaxStride = (int64_t)1 << 40;  // elements; a row's offset stays within 64 bits
bool stride_ok(int64_t s) { return s >= 0 && s <= kMaxStride; }

// From the first element of k_pages or v_pages to the last, all layers.
size_t kv_pool_bytes(const csgmv_kv_cache *kv) {
    return 2 * ((size_t)(kv->num_layers - 1) * kv->layer_stride + (size_t)(kv->num_pages - 1) * kv->page_stride +
                (size_t)(kv->num_kv_heads - 1) * kv->head_stride + (size_t)(kv->page_size - 1) * kv->token_stride + kv->head_dim);
}

int check_counts(const csgmv_token_counts *c) {
    if (!c) return fail(CSGMV_ERR_INVALID_ARG, "counts is NULL");
    if (c->max_seqs <= 0 || c->vocab_size <= 0) return fail(CSGMV_ERR_INVALID_ARG, "sizes of the counts must be positive");
    if (c->vocab_size > (1 << 18) || c->max_seqs > (1 << 20))
        return fail(CSGMV_ERR_UNSUPPORTED, "counts of at most 2^18 tokens and 2^20 sequences");
    const size_t table = 4 * (size_t)c->max_seqs * c->vocab_size, seqs = 4 * (size_t)c->max_seqs;
    const struct { const void *at; size_t bytes; } all[] = {{c->counts, table}, {c->seen, table}, {c->num_seen, seqs}, {c->status, 4}};
    for (int i = 0; i < 4; ++i) {
        if (!all[i].at || !aligned4(all[i].at)) return fail(CSGMV_ERR_INVALID_ARG, "a buffer of the counts is NULL or not 4-byte aligned");
        for (int j = 0; j < i; ++j)
            if (overlaps(all[i].at, all[i].bytes, all[j].at, all[j].bytes))
                return fail(CSGMV_ERR_INVALID_ARG, "buffers of the counts overlap");
    }
    return CSGMV_OK;
}
bool overlaps_counts(const csgmv_token_counts *c, const void *at, size_t bytes) {
    const size_t table = 4 * (size_t)c->max_seqs * c->vocab_size;
    return overlaps(at, bytes, c->counts, table) || overlaps(at, bytes, c->seen, table) ||
           overlaps(at, bytes, c->num_seen, 4 * (size_t)c->max_seqs) || overlaps(at, bytes, c->status, 4);
}
csgmv::CountParams count_params(const csgmv_token_counts *c) {
    csgmv::CountParams p = {};
    p.counts = c->counts;
    p.seen = c->seen;
    p.num_seen = c->num_seen;
    p.status = c->status;
    p.max_seqs = c->max_seqs;
    p.vocab = c->vocab_size;
    return p;
}

// Queries or keys of a call, and their outputs: 0 or an error.
int check_heads(const char *name, const csgmv::Heads &h, int64_t n, int d, int bytes, bool need_out) {
    if (h.n < 0 || h.n > 4096) return fail(CSGMV_ERR_UNSUPPORTED, "%d heads of %s outside 0..4096", h.n, name);
    if (h.n == 0) return CSGMV_OK;
    if (!h.in || (need_out && !h.out)) return fail(CSGMV_ERR_INVALID_ARG, "%s or its output is NULL", name);
    if (!aligned_to(h.in, bytes) || !aligned_to(h.out, bytes))
        return fail(CSGMV_ERR_INVALID_ARG, "%s or its output is not aligned to its type", name);
    if (!stride_ok(h.ts) || !stride_ok(h.hs) || !stride_ok(h.o_ts) || !stride_ok(h.o_hs))
        return fail(CSGMV_ERR_INVALID_ARG, "a stride of %s or its output is negative or above 2^40", name);
    if (h.out && !apart(d, {{n, h.o_ts}, {h.n, h.o_hs}}))
        return fail(CSGMV_ERR_INVALID_ARG, "rows of the output of %s overlap", name);
    return CSGMV_OK;
}
Rows in_rows(const csgmv::Heads &h, int64_t n, int d, int bytes) { return rows_of(h.in, bytes, n, h.ts, h.n, h.hs, d); }
Rows out_rows(const csgmv::Heads &h, int64_t n, int d, int bytes) { return rows_of(h.out, bytes, n, h.o_ts, h.n, h.o_hs, d); }

}  // namespace

extern "C" {

int csgmv_add_norm(const void *x, int64_t x_stride, int dtype, const void *residual, int64_t residual_stride,
                   int residual_dtype, const void *gate, int64_t gate_stride, const csgmv_norm *post,
                   const csgmv_norm *pre, float residual_scale, int64_t num_tokens, int hidden, void *residual_out,
                   int64_t residual_out_stride, void *out, int64_t out_stride, csgmv_stream_t stream) {
    if (!known_type(dtype) || (residual_dtype != dtype && residual_dtype != CSGMV_DTYPE_F32))
        return fail(CSGMV_ERR_INVALID_ARG, "dtype %d must be bf16, f16 or f32, residual_dtype %d the same or f32", dtype,
                    residual_dtype);
    if (num_tokens < 0) return fail(CSGMV_ERR_INVALID_ARG, "negative num_tokens");
    if (num_tokens > INT32_MAX) return fail(CSGMV_ERR_UNSUPPORTED, "num_tokens exceeds int32");
    if (hidden < 1 || hidden > csgmv::kNormMaxHidden)
        return fail(CSGMV_ERR_UNSUPPORTED, "hidden %d outside 1..%d", hidden, csgmv::kNormMaxHidden);
    csgmv::AddNormParams p = {};
    const int e = csgmv::dtype_bytes(dtype), re = csgmv::dtype_bytes(residual_dtype);
    const struct { const csgmv_norm *from; csgmv::NormSide *to; } sides[] = {{post, &p.post}, {pre, &p.pre}};
    for (const auto &s : sides) {
        if (!s.from) continue;
        if (s.from->kind != CSGMV_NORM_NONE && s.from->kind != CSGMV_NORM_RMS && s.from->kind != CSGMV_NORM_LAYER)
            return fail(CSGMV_ERR_INVALID_ARG, "kind %d of a norm", s.from->kind);
        if (!(s.from->eps >= 0.0f) || s.from->eps > 1e30f)
            return fail(CSGMV_ERR_INVALID_ARG, "a norm's eps must be finite and not negative");
        if (!aligned_to(s.from->weight, e) || !aligned_to(s.from->bias, e))
            return fail(CSGMV_ERR_INVALID_ARG, "a norm's weight or bias is not aligned to its type");
        *s.to = {s.from->weight, s.from->bias, s.from->eps, s.from->kind};
    }
    if (!(residual_scale - residual_scale == 0.0f)) return fail(CSGMV_ERR_INVALID_ARG, "residual_scale must be finite");
    if (num_tokens == 0) return CSGMV_OK;
    if (!x || (!out && !residual_out)) return fail(CSGMV_ERR_INVALID_ARG, "NULL tensor");
    if (!out && p.pre.kind != CSGMV_NORM_NONE) return fail(CSGMV_ERR_INVALID_ARG, "a norm of the sum without out");
    if (!aligned_to(x, e) || !aligned_to(gate, e) || !aligned_to(out, e) || !aligned_to(residual, re) || !aligned_to(residual_out, re))
        return fail(CSGMV_ERR_INVALID_ARG, "a tensor is not aligned to its type");
    if (!stride_ok(x_stride) || !stride_ok(residual_stride) || !stride_ok(gate_stride) || !stride_ok(residual_out_stride) ||
        !stride_ok(out_stride))
        return fail(CSGMV_ERR_INVALID_ARG, "a stride is negative or above 2^40");
    if (num_tokens > 1 && ((out && out_stride < hidden) || (residual_out && residual_out_stride < hidden)))
        return fail(CSGMV_ERR_INVALID_ARG, "rows of an output overlap");
    auto rows = [&](const void *at, int bytes, int64_t stride) { return rows_of(at, bytes, num_tokens, stride, 1, 0, hidden); };
    const Rows outs[] = {rows(out, e, out_stride), rows(residual_out, re, residual_out_stride)};
    const Rows ins[] = {rows(x, e, x_stride), rows(residual, re, residual_stride), rows(gate, e, gate_stride)};
    for (const Rows &o : outs) {
        for (const Rows &i : ins)
            if (!in_place_or_apart(o, i))
                return fail(CSGMV_ERR_INVALID_ARG, "an output overlaps an input that it is not");
        for (const auto &s : sides)
            if (s.from && (meet(o, plain(s.from->weight, (size_t)hidden * e)) || meet(o, plain(s.from->bias, (size_t)hidden * e))))
                return fail(CSGMV_ERR_INVALID_ARG, "an output overlaps a norm's weight or bias");
    }
    if (meet(outs[0], outs[1])) return fail(CSGMV_ERR_INVALID_ARG, "the outputs overlap each other");
    p.x = x;
    p.r = residual;
    p.gate = gate;
    p.r_out = residual_out;
    p.out = out;
    p.x_s = x_stride;
    p.r_s = residual_stride;
    p.g_s = gate_stride;
    p.ro_s = residual_out_stride;
    p.o_s = out_stride;
    p.scale = residual_scale;
    p.n = (int)num_tokens;
    p.hidden = hidden;
    p.dtype = dtype;
    p.r_dtype = residual_dtype;
    return launched(csgmv::launch_add_norm(p, st(stream)), "csgmv_add_norm");
}

int csgmv_rope_turns(const double *freq, int n, uint64_t *turns) {
    if (n < 0) return fail(CSGMV_ERR_INVALID_ARG, "negative n");
    if (n > 0 && (!freq || !turns)) return fail(CSGMV_ERR_INVALID_ARG, "freq / turns is NULL");
    for (int i = 0; i < n; ++i)
        if (!std::isfinite(freq[i])) return fail(CSGMV_ERR_INVALID_ARG, "freq[%d] is not finite", i);
    constexpr double whole = 6.283185307179586476925286766559;
    for (int i = 0; i < n; ++i) {
        // what is left of whole turns, a bit of its quotient at a time: every step is exact
        double rest = std::fmod(std::fabs(freq[i]), whole);
        uint64_t steps = 0;
        auto bit = [&] {
            rest += rest;
            const bool one = rest >= whole;
            if (one) rest -= whole;
            return one;
        };
        for (int k = 0; k < 64; ++k) steps = 2 * steps + bit();
        steps += bit();  // the nearest one (a whole turn is none)
        turns[i] = freq[i] < 0 ? 0 - steps : steps;
    }
    return CSGMV_OK;
}

int csgmv_rotary(const csgmv_rope *rope, int dtype, int head_dim, const int32_t *positions, int64_t num_tokens,
                 const void *q, int64_t q_token_stride, int64_t q_head_stride, int num_q_heads, const void *k,
                 int64_t k_token_stride, int64_t k_head_stride, int num_k_heads, void *q_out, int64_t qo_token_stride,
                 int64_t qo_head_stride, void *k_out, int64_t ko_token_stride, int64_t ko_head_stride, int inverse,
                 csgmv_stream_t stream) {
    if (!known_type(dtype)) return fail(CSGMV_ERR_INVALID_ARG, "dtype %d must be bf16, f16 or f32", dtype);
    if (head_dim < 1 || head_dim > 1024) return fail(CSGMV_ERR_UNSUPPORTED, "head_dim %d outside 1..1024", head_dim);
    if (!rope) return fail(CSGMV_ERR_INVALID_ARG, "rope is NULL");
    int rc = check_rope(rope, head_dim);
    if (rc) return rc;
    if (num_tokens < 0) return fail(CSGMV_ERR_INVALID_ARG, "negative num_tokens");
    if (num_tokens > INT32_MAX) return fail(CSGMV_ERR_UNSUPPORTED, "num_tokens exceeds int32");
    if (inverse != 0 && inverse != 1) return fail(CSGMV_ERR_INVALID_ARG, "inverse must be 0 or 1");
    csgmv::RotaryParams p = {};
    p.q = {q, q_out, q_token_stride, q_head_stride, qo_token_stride, qo_head_stride, num_q_heads};
    p.k = {k, k_out, k_token_stride, k_head_stride, ko_token_stride, ko_head_stride, num_k_heads};
    const int e = csgmv::dtype_bytes(dtype);
    if (num_tokens == 0) return CSGMV_OK;
    if ((rc = check_heads("q", p.q, num_tokens, head_dim, e, true)) || (rc = check_heads("k", p.k, num_tokens, head_dim, e, true)))
        return rc;
    if (num_q_heads == 0 && num_k_heads == 0) return CSGMV_OK;
    if (!positions || !aligned4(positions)) return fail(CSGMV_ERR_INVALID_ARG, "positions is NULL or not 4-byte aligned");
    const Rows qi = in_rows(p.q, num_tokens, head_dim, e), ki = in_rows(p.k, num_tokens, head_dim, e);
    const Rows qo = out_rows(p.q, num_tokens, head_dim, e), ko = out_rows(p.k, num_tokens, head_dim, e);
    const Rows steer[] = {plain(positions, 4 * (size_t)num_tokens), plain(rope->turns, 4 * (size_t)rope->rotary_dim)};
    bool bad = !in_place_or_apart(qo, qi) || !in_place_or_apart(ko, ki) || meet(qo, ki) || meet(ko, qi) || meet(qo, ko);
    for (const Rows &s : steer) bad = bad || meet(qo, s) || meet(ko, s);
    if (bad) return fail(CSGMV_ERR_INVALID_ARG, "an output overlaps an input that it is not, or the other output");
    p.turns = rope->turns;
    p.positions = positions;
    p.scale = rope->scale;
    p.sign = inverse ? -1.0f : 1.0f;
    p.rot = rope->rotary_dim;
    p.interleaved = rope->interleaved;
    p.d = head_dim;
    // (outputs that begin where their inputs do are those)
    p.rest = (num_q_heads == 0 || q_out == q) && (num_k_heads == 0 || k_out == k) ? 0 : head_dim - rope->rotary_dim;
    p.dtype = dtype;
    p.num_tokens = num_tokens;
    return launched(csgmv::launch_rotary(p, st(stream)), "csgmv_rotary");
}

int csgmv_kv_extend(const csgmv_kv_cache *kv, const int32_t *add_lens, const int32_t *tree_indptr,
                    const int32_t *seq_slots, int bs, int64_t num_tokens, int64_t *slots, int32_t *positions,
                    int32_t *lens_before, csgmv_stream_t stream) {
    int rc = check_kv(kv);
    if (rc) return rc;
    if (bs < 0 || num_tokens < 0) return fail(CSGMV_ERR_INVALID_ARG, "negative bs / num_tokens");
    if (bs > kv->max_seqs) return fail(CSGMV_ERR_CAPACITY, "bs %d exceeds max_seqs %d", bs, kv->max_seqs);
    if (num_tokens > INT32_MAX) return fail(CSGMV_ERR_UNSUPPORTED, "num_tokens exceeds int32");
    if (bs > 0 && !tree_indptr) return fail(CSGMV_ERR_INVALID_ARG, "tree_indptr is NULL");
    if (num_tokens > 0 && (!slots || !positions)) return fail(CSGMV_ERR_INVALID_ARG, "slots / positions is NULL");
    if (!aligned4(add_lens) || !aligned4(tree_indptr) || !aligned4(seq_slots) || !aligned_to(slots, 8) || !aligned4(positions) ||
        !aligned4(lens_before))
        return fail(CSGMV_ERR_INVALID_ARG, "a buffer is not aligned to its type");
    const size_t pool = kv_pool_bytes(kv);
    const struct { const void *at; size_t bytes; } all[] = {
        {slots, 8 * (size_t)num_tokens}, {positions, 4 * (size_t)num_tokens}, {lens_before, 4 * (size_t)kv->max_seqs},
        {add_lens, 4 * (size_t)bs}, {tree_indptr, bs ? 4 * (size_t)bs + 4 : 0}, {seq_slots, 4 * (size_t)bs}};
    for (int i = 0; i < 6; ++i) {
        bool bad = overlaps_plan(kv, static_cast<const int32_t *>(all[i].at), all[i].bytes / 4) ||
                   overlaps(all[i].at, all[i].bytes, kv->k_pages, pool) || overlaps(all[i].at, all[i].bytes, kv->v_pages, pool);
        for (int j = 0; j < i && j < 3; ++j) bad = bad || overlaps(all[i].at, all[i].bytes, all[j].at, all[j].bytes);
        if (bad) return fail(CSGMV_ERR_INVALID_ARG, "a buffer of the call overlaps another one or the cache");
    }
    if (bs == 0 && num_tokens == 0 && !lens_before) return CSGMV_OK;
    csgmv::ExtendParams p = {};
    p.plan.num_tokens = num_tokens;
    p.plan.accept_len = add_lens;
    p.plan.tree_indptr = tree_indptr;
    p.plan.seq_slots = seq_slots;
    p.plan.bs = bs;
    p.slots = slots;
    p.positions = positions;
    p.lens_before = lens_before;
    return launched(csgmv::launch_kv_extend(*kv, p, st(stream)), "csgmv_kv_extend");
}

int csgmv_kv_append(const csgmv_kv_cache *kv, int layer, const csgmv_rope *rope, const int32_t *positions,
                    const int64_t *slots, int64_t num_tokens, const void *q, int64_t q_token_stride,
                    int64_t q_head_stride, int num_q_heads, const void *k, int64_t k_token_stride,
                    int64_t k_head_stride, const void *v, int64_t v_token_stride, int64_t v_head_stride, void *q_out,
                    int64_t qo_token_stride, int64_t qo_head_stride, void *k_out, int64_t ko_token_stride,
                    int64_t ko_head_stride, csgmv_stream_t stream) {
    int rc = check_kv(kv);
    if (rc) return rc;
    if (layer < 0 || layer >= kv->num_layers)
        return fail(CSGMV_ERR_INVALID_ARG, "layer %d outside [0, %d)", layer, kv->num_layers);
    if (rope && (rc = check_rope(rope, kv->head_dim))) return rc;
    if (num_tokens < 0) return fail(CSGMV_ERR_INVALID_ARG, "negative num_tokens");
    if (num_tokens > INT32_MAX) return fail(CSGMV_ERR_UNSUPPORTED, "num_tokens exceeds int32");
    if (num_tokens == 0) return CSGMV_OK;
    const int d = kv->head_dim, e = 2;
    csgmv::RotaryParams p = {};
    p.q = {q, q_out, q_token_stride, q_head_stride, qo_token_stride, qo_head_stride, num_q_heads};
    p.k = {k, k_out, k_token_stride, k_head_stride, ko_token_stride, ko_head_stride, kv->num_kv_heads};
    p.v = {v, nullptr, v_token_stride, v_head_stride, 0, 0, kv->num_kv_heads};
    if ((rc = check_heads("q", p.q, num_tokens, d, e, true)) || (rc = check_heads("k", p.k, num_tokens, d, e, false)) ||
        (rc = check_heads("v", p.v, num_tokens, d, e, false)))
        return rc;
    if (!slots || !aligned_to(slots, 8)) return fail(CSGMV_ERR_INVALID_ARG, "slots is NULL or not 8-byte aligned");
    if (rope && (!positions || !aligned4(positions)))
        return fail(CSGMV_ERR_INVALID_ARG, "positions is NULL or not 4-byte aligned");
    const Rows qi = in_rows(p.q, num_tokens, d, e), ki = in_rows(p.k, num_tokens, d, e), vi = in_rows(p.v, num_tokens, d, e);
    const Rows qo = out_rows(p.q, num_tokens, d, e), ko = out_rows(p.k, num_tokens, d, e);
    bool bad = !in_place_or_apart(qo, qi) || !in_place_or_apart(ko, ki) || meet(qo, ki) || meet(qo, vi) || meet(ko, qi) ||
               meet(ko, vi) || meet(qo, ko);
    // the pages of the cache, all layers of them, are an output too
    const size_t pool = kv_pool_bytes(kv);
    const Rows pools[] = {plain(kv->k_pages, pool), plain(kv->v_pages, pool)};
    const Rows steer[] = {plain(slots, 8 * (size_t)num_tokens), plain(rope ? positions : nullptr, 4 * (size_t)num_tokens),
                          plain(rope ? rope->turns : nullptr, rope ? 4 * (size_t)rope->rotary_dim : 0),
                          plain(kv->page_table, 4 * (size_t)kv->max_seqs * kv->max_pages_per_seq),
                          plain(kv->seq_lens, 4 * (size_t)kv->max_seqs), plain(kv->page_refs, 4 * (size_t)kv->num_pages),
                          plain(kv->status, 4)};
    for (const Rows &x : {qo, ko}) {
        for (const Rows &s : steer) bad = bad || meet(x, s);
        for (const Rows &s : pools) bad = bad || meet(x, s);
    }
    for (const Rows &x : {qi, ki, vi, steer[0], steer[1], steer[2]})
        for (const Rows &s : pools) bad = bad || meet(x, s);
    if (bad) return fail(CSGMV_ERR_INVALID_ARG, "an output overlaps an input that it is not, another output or the cache");
    if (rope) {
        p.turns = rope->turns;
        p.scale = rope->scale;
        p.rot = rope->rotary_dim;
        p.interleaved = rope->interleaved;
    }
    p.sign = 1.0f;
    p.positions = positions;
    p.d = d;
    p.rest = d - p.rot;
    p.dtype = kv->dtype;
    p.num_tokens = num_tokens;
    p.slots = slots;
    p.k_pages = static_cast<uint16_t *>(kv->k_pages) + (int64_t)layer * kv->layer_stride;
    p.v_pages = static_cast<uint16_t *>(kv->v_pages) + (int64_t)layer * kv->layer_stride;
    p.page_stride = kv->page_stride;
    p.head_stride = kv->head_stride;
    p.token_stride = kv->token_stride;
    p.num_slots = (int64_t)kv->num_pages * kv->page_size;
    p.page_shift = __builtin_ctz((unsigned)kv->page_size);
    p.status = kv->status;
    return launched(csgmv::launch_rotary(p, st(stream)), "csgmv_kv_append");
}

int csgmv_count_tokens(const csgmv_token_counts *counts, const int32_t *tokens, int64_t num_tokens,
                       const int32_t *tree_indptr, const int32_t *accept_index, int accept_width,
                       const int32_t *accept_len, const int32_t *seq_slots, int bs, int prompt, csgmv_stream_t stream) {
    int rc = check_counts(counts);
    if (rc) return rc;
    if (bs < 0 || num_tokens < 0) return fail(CSGMV_ERR_INVALID_ARG, "negative bs / num_tokens");
    if (num_tokens > INT32_MAX) return fail(CSGMV_ERR_UNSUPPORTED, "num_tokens exceeds int32");
    if (prompt != 0 && prompt != 1) return fail(CSGMV_ERR_INVALID_ARG, "prompt must be 0 or 1");
    if (bs == 0 || num_tokens == 0) return CSGMV_OK;
    if (!tokens || !tree_indptr) return fail(CSGMV_ERR_INVALID_ARG, "tokens / tree_indptr is NULL");
    if (accept_index && (accept_width <= 0 || !accept_len))
        return fail(CSGMV_ERR_INVALID_ARG, "accept_index needs a positive accept_width and accept_len");
    if (accept_index && accept_width > kMaxList) return fail(CSGMV_ERR_UNSUPPORTED, "accept_width exceeds 2^30");
    const size_t b4 = 4 * (size_t)bs;
    const struct { const void *at; size_t bytes; } lists[] = {{tokens, 4 * (size_t)num_tokens},
                                                              {tree_indptr, b4 + 4},
                                                              {accept_index, b4 * (accept_index ? accept_width : 0)},
                                                              {accept_len, b4},
                                                              {seq_slots, b4}};
    for (const auto &l : lists)
        if (!aligned4(l.at) || overlaps_counts(counts, l.at, l.bytes))
            return fail(CSGMV_ERR_INVALID_ARG, "a list of the call is not 4-byte aligned or overlaps the counts");
    csgmv::CountParams p = count_params(counts);
    p.prompt = prompt;
    p.accept_width = accept_width;
    p.num_tokens = num_tokens;
    p.tokens = tokens;
    p.indptr = tree_indptr;
    p.accept_index = accept_index;
    p.accept_len = accept_len;
    p.slots = seq_slots;
    return launched(csgmv::launch_count_tokens(p, bs, st(stream)), "csgmv_count_tokens");
}

int csgmv_count_reset(const csgmv_token_counts *counts, const int32_t *seqs, int n, csgmv_stream_t stream) {
    int rc = check_counts(counts);
    if (rc) return rc;
    if (n < 0) return fail(CSGMV_ERR_INVALID_ARG, "negative n");
    if (n == 0) return CSGMV_OK;
    if (!seqs || !aligned4(seqs) || overlaps_counts(counts, seqs, 4 * (size_t)n))
        return fail(CSGMV_ERR_INVALID_ARG, "seqs is NULL, not 4-byte aligned or overlaps the counts");
    csgmv::CountParams p = count_params(counts);
    p.slots = seqs;
    return launched(csgmv::launch_count_reset(p, n, st(stream)), "csgmv_count_reset");
}

int csgmv_count_fork(const csgmv_token_counts *counts, const int32_t *parents, const int32_t *children, int n,
                     csgmv_stream_t stream) {
    int rc = check_counts(counts);
    if (rc) return rc;
    if (n < 0) return fail(CSGMV_ERR_INVALID_ARG, "negative n");
    if (n > counts->max_seqs) return fail(CSGMV_ERR_CAPACITY, "n %d exceeds max_seqs %d", n, counts->max_seqs);
    if (n == 0) return CSGMV_OK;
    for (const int32_t *l : {parents, children})
        if (!l || !aligned4(l) || overlaps_counts(counts, l, 4 * (size_t)n))
            return fail(CSGMV_ERR_INVALID_ARG, "parents / children is NULL, not 4-byte aligned or overlaps the counts");
    return launched(csgmv::launch_count_fork(count_params(counts), parents, children, n, st(stream)), "csgmv_count_fork");
}

int csgmv_process_logits(const void *logits, int dtype, int64_t logits_stride, const int32_t *tree_indptr,
                         const int32_t *seq_slots, int bs, int64_t num_tokens, int vocab_size,
                         const csgmv_logit_rules *rules, const int32_t *draft_tokens, const int32_t *mask, int mask_words,
                         int softmax, float *out, int64_t out_stride, csgmv_stream_t stream) {
    if (!known_type(dtype)) return fail(CSGMV_ERR_INVALID_ARG, "dtype %d must be bf16, f16 or f32", dtype);
    if (bs < 0 || num_tokens < 0) return fail(CSGMV_ERR_INVALID_ARG, "negative bs / num_tokens");
    if (num_tokens >= (1 << 24)) return fail(CSGMV_ERR_UNSUPPORTED, "num_tokens exceeds 2^24 - 1");
    if (bs > kMaxList) return fail(CSGMV_ERR_UNSUPPORTED, "bs exceeds 2^30");
    if (vocab_size < 1 || vocab_size > (1 << 18))
        return fail(CSGMV_ERR_UNSUPPORTED, "vocab_size %d outside 1..2^18", vocab_size);
    if (!rules || !rules->status || !aligned4(rules->status))
        return fail(CSGMV_ERR_INVALID_ARG, "rules or its status is NULL or not 4-byte aligned");
    const csgmv_logit_rules &r = *rules;
    const csgmv_token_counts *counts = r.counts;
    if (counts) {
        int rc = check_counts(counts);
        if (rc) return rc;
        if (counts->vocab_size != vocab_size)
            return fail(CSGMV_ERR_INVALID_ARG, "counts of %d tokens, logits of %d", counts->vocab_size, vocab_size);
    }
    if (r.bias_total < 0 || r.bias_total > kMaxList) return fail(CSGMV_ERR_INVALID_ARG, "bias_total outside [0, 2^30]");
    if (r.bias_indptr && r.bias_total > 0 && (!r.bias_tokens || !r.bias_values))
        return fail(CSGMV_ERR_INVALID_ARG, "bias_tokens / bias_values is NULL");
    if (r.num_allow < 0) return fail(CSGMV_ERR_INVALID_ARG, "negative num_allow");
    if (r.allow_index && r.num_allow > 0 && (!r.allow || r.allow_words < (vocab_size + 31) / 32))
        return fail(CSGMV_ERR_INVALID_ARG, "allow is NULL or allow_words %d below %d", r.allow_words, (vocab_size + 31) / 32);
    if (softmax != 0 && softmax != 1) return fail(CSGMV_ERR_INVALID_ARG, "softmax must be 0 or 1");
    const bool branch = draft_tokens && mask;
    if (branch && (mask_words < 1 || mask_words > csgmv::kTreeMaxWords))
        return fail(CSGMV_ERR_UNSUPPORTED, "mask_words %d outside 1..%d", mask_words, csgmv::kTreeMaxWords);
    if (bs == 0 || num_tokens == 0) return CSGMV_OK;
    if (!logits || !out || !tree_indptr) return fail(CSGMV_ERR_INVALID_ARG, "NULL tensor");
    const int e = csgmv::dtype_bytes(dtype);
    if (!aligned_to(logits, e) || !aligned4(out)) return fail(CSGMV_ERR_INVALID_ARG, "logits or out is not aligned to its type");
    if (!stride_ok(logits_stride) || !stride_ok(out_stride) || (num_tokens > 1 && out_stride < vocab_size))
        return fail(CSGMV_ERR_INVALID_ARG, "a stride is negative or above 2^40, or rows of out overlap");
    const Rows in = rows_of(logits, e, num_tokens, logits_stride, 1, 0, vocab_size);
    const Rows to = rows_of(out, 4, num_tokens, out_stride, 1, 0, vocab_size);
    if (!in_place_or_apart(to, in)) return fail(CSGMV_ERR_INVALID_ARG, "out overlaps logits");
    const size_t b4 = 4 * (size_t)bs, n4 = 4 * (size_t)num_tokens;
    const struct { const void *at; size_t bytes; } read[] = {
        {tree_indptr, b4 + 4}, {seq_slots, b4}, {r.repetition, b4}, {r.frequency, b4}, {r.presence, b4}, {r.temperature, b4},
        {r.bias_indptr, b4 + 4}, {r.bias_tokens, 4 * (size_t)r.bias_total}, {r.bias_values, 4 * (size_t)r.bias_total},
        {r.allow, r.allow_index ? 4 * (size_t)r.num_allow * (size_t)std::max(r.allow_words, 0) : 0}, {r.allow_index, n4},
        {draft_tokens, branch ? n4 : 0}, {mask, branch ? n4 * mask_words : 0}};
    for (const auto &l : read)
        if (!aligned4(l.at) || meet(to, plain(l.at, l.bytes)) || overlaps(l.at, l.bytes, r.status, 4))
            return fail(CSGMV_ERR_INVALID_ARG, "a list of the call is not 4-byte aligned or overlaps out or the status");
    if (meet(to, plain(r.status, 4)) || meet(in, plain(r.status, 4)) ||
        (counts && (overlaps_counts(counts, r.status, 4) && r.status != counts->status)))
        return fail(CSGMV_ERR_INVALID_ARG, "the status overlaps a tensor");
    if (counts) {
        const size_t table = 4 * (size_t)counts->max_seqs * vocab_size;
        if (meet(to, plain(counts->counts, table)) || meet(to, plain(counts->seen, table)) ||
            meet(to, plain(counts->num_seen, 4 * (size_t)counts->max_seqs)))
            return fail(CSGMV_ERR_INVALID_ARG, "out overlaps the counts");
    }
    csgmv::LogitParams p = {};
    p.logits = logits;
    p.out = out;
    p.logits_s = logits_stride;
    p.out_s = out_stride;
    p.num_tokens = num_tokens;
    p.bias_total = r.bias_total;
    p.indptr = tree_indptr;
    p.slots = seq_slots;
    if (counts) {
        p.counts = counts->counts;
        p.seen = counts->seen;
        p.num_seen = counts->num_seen;
        p.max_seqs = counts->max_seqs;
    }
    p.repetition = r.repetition;
    p.frequency = r.frequency;
    p.presence = r.presence;
    p.temperature = r.temperature;
    p.bias_indptr = r.bias_indptr;
    p.bias_tokens = r.bias_tokens;
    p.bias_values = r.bias_values;
    p.allow = r.allow;
    p.allow_index = r.allow_index;
    p.num_allow = r.num_allow;
    p.allow_words = r.allow_words;
    p.drafts = branch ? draft_tokens : nullptr;
    p.mask = branch ? mask : nullptr;
    p.mask_words = branch ? mask_words : 0;
    p.status = r.status;
    p.bs = bs;
    p.vocab = vocab_size;
    p.softmax = softmax;
    p.dtype = dtype;
    return launched(csgmv::launch_process_logits(p, st(stream)), "csgmv_process_logits");
}

}  // extern "C"
