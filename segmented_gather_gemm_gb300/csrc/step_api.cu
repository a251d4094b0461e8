// C ABI of what a decoder does between the projections, the attention and the
// verification: argument checks on the host, then the launches of each call
// on the caller's stream.  Nothing here allocates, frees or synchronizes.
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
Rows plain(const void *at, size_t bytes) { return {bytes ? at : nullptr, 1, 0, 1, 0, (int64_t)bytes}; }

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

constexpr int64_t kMaxStride = (int64_t)1 << 40;  // elements; a row's offset stays within 64 bits
bool stride_ok(int64_t s) { return s >= 0 && s <= kMaxStride; }

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

}  // extern "C"
