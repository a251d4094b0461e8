// Rotary positions of queries and keys, and the same with keys and values
// written into a layer of the paged cache on the way.  See include/csgmv.h
// (csgmv_rotary, csgmv_kv_append).
//
// A pair (u, v) becomes scale (u cos a - v sin a, u sin a + v cos a) with a = p f.
// f is held in 2^-64 turns: p f in 64-bit whole numbers wraps at whole turns by
// itself, so no angle loses bits however far its position is, and no table of
// cosines is read.  A thread owns W neighbouring pairs of a head (two vectors of
// W elements, or one of 2 W where pairs lie side by side) of one token: it takes
// their sines and cosines once and turns that part of several heads, four at a
// time so that their loads are in flight together.
#include "elements.cuh"
#include "serving.cuh"
#include "step.h"

#include <algorithm>

namespace csgmv {
namespace {

constexpr int kThreads = 256;

// A thread's place: `lanes` head lanes of `units` units a token, `tokens` tokens a block.
struct Shape {
    int units, pairs, lanes, slots, tokens;
};

template <typename T, int W, bool IL, bool APPEND>
__global__ void __launch_bounds__(kThreads) rotary(RotaryParams p, Shape s) {
    griddep_launch_dependents();
    griddep_wait();
    const int local = threadIdx.x / s.slots, slot0 = threadIdx.x - local * s.slots;
    const int64_t t = (int64_t)blockIdx.x * s.tokens + local;
    if (local >= s.tokens || t >= p.num_tokens) return;
    int64_t to = 0;  // of the token, in a head of the pages
    if (APPEND) {
        const int64_t at = p.slots[t];
        if (at < 0 || at >= p.num_slots) {
            if (at != -1 && slot0 == 0) atomicOr(p.status, CSGMV_KV_STATUS_BAD_PAGE);
            return;
        }
        to = (at >> p.page_shift) * p.page_stride + (at & ((1 << p.page_shift) - 1)) * p.token_stride;
    }
    const T *q = static_cast<const T *>(p.q.in) + t * p.q.ts, *k = static_cast<const T *>(p.k.in) + t * p.k.ts;
    T *qo = static_cast<T *>(p.q.out) + t * p.q.o_ts;
    T *ko = p.k.out ? static_cast<T *>(p.k.out) + t * p.k.o_ts : nullptr;
    T *kc = APPEND ? static_cast<T *>(p.k_pages) + to : nullptr;
    const int heads = p.q.n + p.k.n;
    for (int slot = slot0; slot < s.units * s.lanes; slot += s.slots) {
        const int lane = slot / s.units, unit = slot - lane * s.units;
        const bool turned = unit < s.pairs;
        // the unit's first element and, of pairs apart, how far their second ones are
        const int e = turned ? unit * (IL ? 2 * W : W) : p.rot + (unit - s.pairs) * W, apart = IL ? W : p.rot / 2;
        float c[W], z[W];
        if (turned) {
            const uint64_t pos = (uint64_t)(int64_t)p.positions[t];
#pragma unroll
            for (int i = 0; i < W; ++i) {
                const int64_t turn = (int64_t)(pos * p.turns[unit * W + i]);  // 2^-64 turns, modulo a whole one
                float sn, cs;
                sincospif(__ll2float_rn(turn) * 0x1p-63f, &sn, &cs);
                c[i] = cs * p.scale;
                z[i] = sn * p.scale * p.sign;
            }
        }
        constexpr int U = 4;
        for (int h0 = lane; h0 < heads; h0 += U * s.lanes) {
            Vec<T, W> a[U], b[U];
#pragma unroll
            for (int x = 0; x < U; ++x) {
                const int h = h0 + x * s.lanes;
                if (h >= heads) continue;
                const T *at = (h < p.q.n ? q + h * p.q.hs : k + (h - p.q.n) * p.k.hs) + e;
                a[x] = ld_vec<T, W>(at);
                if (turned) b[x] = ld_vec<T, W>(at + apart);
            }
#pragma unroll
            for (int x = 0; x < U; ++x) {
                const int h = h0 + x * s.lanes;
                if (h >= heads) continue;
                if (turned) {
#pragma unroll
                    for (int i = 0; i < W; ++i) {
                        // pair i: elements i of both, or neighbours in the two vectors laid end to end
                        T &u = IL ? (2 * i < W ? a[x].e[(2 * i) % W] : b[x].e[(2 * i) % W]) : a[x].e[i];
                        T &v = IL ? (2 * i + 1 < W ? a[x].e[(2 * i + 1) % W] : b[x].e[(2 * i + 1) % W]) : b[x].e[i];
                        const float uf = to_f32(u), vf = to_f32(v);
                        u = from_f32<T>(uf * c[i] - vf * z[i]);
                        v = from_f32<T>(uf * z[i] + vf * c[i]);
                    }
                }
                T *out[2] = {nullptr, nullptr};
                if (h < p.q.n) {
                    out[0] = qo + h * p.q.o_hs;
                } else {
                    if (ko) out[0] = ko + (h - p.q.n) * p.k.o_hs;
                    if (APPEND) out[1] = kc + (h - p.q.n) * p.head_stride;
                }
#pragma unroll
                for (int o = 0; o < (APPEND ? 2 : 1); ++o) {
                    if (!out[o]) continue;
                    st_vec<T, W>(out[o] + e, a[x]);
                    if (turned) st_vec<T, W>(out[o] + e + apart, b[x]);
                }
            }
        }
    }
    if (APPEND) {
        const T *v = static_cast<const T *>(p.v.in) + t * p.v.ts;
        T *vc = static_cast<T *>(p.v_pages) + to;
        const int chunks = p.d / W, n = p.v.n * chunks;
        for (int i = slot0; i < n; i += s.slots) {
            const int h = i / chunks, e = (i - h * chunks) * W;
            st_vec<T, W>(vc + h * p.head_stride + e, ld_vec<T, W>(v + h * p.v.hs + e));
        }
    }
}

// The widest units (16 bytes of elements, or two, or one): W pairs and W elements
// of what is not turned, all addresses multiples of W elements.
int width_for(const RotaryParams &p, int bytes) {
    uint64_t at = 0;
    int64_t strides = 0;
    for (const Heads *h : {&p.q, &p.k, &p.v}) {
        if (h->n == 0) continue;
        at |= reinterpret_cast<uintptr_t>(h->in) | reinterpret_cast<uintptr_t>(h->out);
        strides |= h->ts | h->hs | (h->out ? h->o_ts | h->o_hs : 0);
    }
    if (p.slots) {
        at |= reinterpret_cast<uintptr_t>(p.k_pages) | reinterpret_cast<uintptr_t>(p.v_pages);
        strides |= p.page_stride | p.head_stride | p.token_stride;
    }
    for (int w : {16 / bytes, 2}) {
        const int align = w * bytes;
        if (p.rot / 2 % w == 0 && p.d % w == 0 && at % align == 0 && strides * bytes % align == 0) return w;
    }
    return 1;
}

template <typename T, int W, bool APPEND>
cudaError_t go(const RotaryParams &p, cudaStream_t stream) {
    Shape s;
    s.pairs = p.rot / 2 / W;
    s.units = s.pairs + (p.d - p.rot) / W;
    const int heads = std::max(1, p.q.n + p.k.n);
    // Four heads a thread share its sines; few tokens spread over all lanes instead.
    const int64_t wide = p.num_tokens * heads * s.units;
    const int each = wide >= 152 * 1024 * 4 ? 4 : 1;
    s.lanes = std::max(1, std::min((heads + each - 1) / each, kThreads / s.units));
    s.slots = std::min(kThreads, s.units * s.lanes);
    s.tokens = kThreads / s.slots;
    const int64_t blocks = (p.num_tokens + s.tokens - 1) / s.tokens;
    if (blocks > INT32_MAX) return cudaErrorInvalidValue;
    const dim3 grid((unsigned)blocks);
    return p.interleaved ? launch_kernel(rotary<T, W, true, APPEND>, grid, kThreads, 0, stream, 0, true, p, s)
                         : launch_kernel(rotary<T, W, false, APPEND>, grid, kThreads, 0, stream, 0, true, p, s);
}

template <typename T, bool APPEND>
cudaError_t pick(const RotaryParams &p, cudaStream_t stream) {
    constexpr int kWide = 16 / (int)sizeof(T);
    switch (width_for(p, (int)sizeof(T))) {
        case kWide: return go<T, kWide, APPEND>(p, stream);
        case 2: return go<T, 2, APPEND>(p, stream);
        default: return go<T, 1, APPEND>(p, stream);
    }
}

}  // namespace

cudaError_t launch_rotary(const RotaryParams &p, cudaStream_t stream) {
    switch (p.dtype) {
        case CSGMV_DTYPE_BF16:
            return p.slots ? pick<__nv_bfloat16, true>(p, stream) : pick<__nv_bfloat16, false>(p, stream);
        case CSGMV_DTYPE_F16:
            return p.slots ? pick<__half, true>(p, stream) : pick<__half, false>(p, stream);
        default:
            return pick<float, false>(p, stream);
    }
}

}  // namespace csgmv
