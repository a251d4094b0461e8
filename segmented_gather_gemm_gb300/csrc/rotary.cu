// Rotary positions of queries and keys, and the same with keys and values
// written into a layer of the paged cache on the way.  See include/csgmv.h
// (csgmv_rotary, csgmv_kv_append).
//
// A pair (u, v) becomes scale (u cos a - v sin a, u sin a + v cos a) with a = p f.
// f is held in 2^-64 turns: p f in 64-bit whole numbers wraps at whole turns by
// itself, so no angle loses bits however far its position is, and no table of
// cosines is read.  A CTA takes the sines and cosines of its tokens once, into
// shared memory.  A thread owns W neighbouring pairs (two vectors of W elements, or
// one of 2 W where pairs lie side by side) of one token in some of its heads.  What is not
// turned is moved two vectors at a time too, or, in place, not touched.  One
// head at a time, its angles from shared memory: more loads under way a thread, or
// angles in registers, take room from the warps that hide loads (four heads: 220 us
// where one took 117, angles in shared memory 113; six CTAs an SM spill: 116).
//
// Measured (device time): 35507 tokens of 32 + 8 heads of 128, bf16 (727 MB) 113 us,
// 6.4 TB/s; with values into a layer's pages, 35700 tokens in half (880 MB) 136 us;
// 12 tokens 3.0 us, a launch and two rounds of loads.  With 32 of the 128 turned 113 us
// (149 by single vectors of the rest), 53 in place.  What bounds the large ones is
// HBM; where a token has few heads (one of each: 2.5 TB/s) its angles.
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

// n floats of shared memory, read where they are used each time (in registers from
// head to head they take room from the warps that hide the loads).
template <int n>
__device__ __forceinline__ void shared_floats(float (&x)[n], const float *p) {
    const uint32_t at = smem_u32(p);
    if constexpr (n == 4) asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(x[0]), "=f"(x[1]), "=f"(x[2]), "=f"(x[3]) : "r"(at));
    else if constexpr (n == 2) asm volatile("ld.shared.v2.f32 {%0, %1}, [%2];" : "=f"(x[0]), "=f"(x[1]) : "r"(at));
    else asm volatile("ld.shared.f32 %0, [%1];" : "=f"(x[0]) : "r"(at));
}
// W pairs: elements i of both vectors, or neighbours in the two laid end to end.
template <typename T, int W, bool IL>
__device__ __forceinline__ void turn_pairs(Vec<T, W> &a, Vec<T, W> &b, const float *cosines, const float *sines) {
    constexpr int G = W < 4 ? W : 4;
#pragma unroll
    for (int i0 = 0; i0 < W; i0 += G) {
        float c[G], z[G];
        shared_floats(c, cosines + i0), shared_floats(z, sines + i0);
#pragma unroll
        for (int j = 0; j < G; ++j) {
            const int i = i0 + j;
            T &u = IL ? (2 * i < W ? a.e[(2 * i) % W] : b.e[(2 * i) % W]) : a.e[i];
            T &v = IL ? (2 * i + 1 < W ? a.e[(2 * i + 1) % W] : b.e[(2 * i + 1) % W]) : b.e[i];
            const float uf = to_f32(u), vf = to_f32(v);
            u = from_f32<T>(uf * c[j] - vf * z[j]);
            v = from_f32<T>(uf * z[j] + vf * c[j]);
        }
    }
}

template <typename T, int W, bool IL, bool APPEND>
__global__ void __launch_bounds__(kThreads, 5) rotary(RotaryParams p, Shape s) {
    extern __shared__ float4 angles4[];
    float *cosines = reinterpret_cast<float *>(angles4), *sines = cosines + s.tokens * s.pairs * W;
    griddep_launch_dependents();
    griddep_wait();
    const int local = threadIdx.x / s.slots, slot0 = threadIdx.x - local * s.slots;
    const int64_t t0 = (int64_t)blockIdx.x * s.tokens, t = t0 + local;
    bool mine = local < s.tokens && t < p.num_tokens;
    int64_t to = 0;  // of the token, in a head of the pages
    if (APPEND && mine) {
        const int64_t at = p.slots[t];
        if (at < 0 || at >= p.num_slots) {
            if (at != -1 && slot0 == 0) atomicOr(p.status, CSGMV_KV_STATUS_BAD_PAGE);
            mine = false;
        } else {
            to = (at >> p.page_shift) * p.page_stride + (at & ((1 << p.page_shift) - 1)) * p.token_stride;
        }
    }
    for (int i = threadIdx.x; i < s.tokens * s.pairs * W; i += kThreads) {
        const int token = i / (s.pairs * W);
        if (t0 + token >= p.num_tokens) break;
        const uint64_t pos = (uint64_t)(int64_t)p.positions[t0 + token];
        const int64_t turn = (int64_t)(pos * p.turns[i - token * (s.pairs * W)]);  // 2^-64 turns, modulo a whole one
        float sn, cs;
        sincospif(__ll2float_rn(turn) * 0x1p-63f, &sn, &cs);
        cosines[i] = cs * p.scale;
        sines[i] = sn * p.scale * p.sign;
    }
    __syncthreads();
    if (!mine) return;
    for (int slot = slot0; slot < s.units * s.lanes; slot += s.slots) {
        // the thread's unit: its first element, and how far its second vector is (nowhere, so
        // that it moves one twice, where an odd number of them is not turned)
        const int lane = slot / s.units, unit = slot - lane * s.units;
        const bool turned = unit < s.pairs;
        const int e = turned ? unit * (IL ? 2 * W : W) : p.rot + (unit - s.pairs) * W;
        int apart = !turned ? (s.units - s.pairs) * W : IL ? W : p.rot / 2;
        if (e + apart >= p.d) apart = 0;
        const int first = turned ? (local * s.pairs + unit) * W : 0;
        // the unit in heads lane, lane + lanes, ... of a tensor, to up to two places
        auto heads = [&](const Heads &x, bool turn, T *page) {
            const T *in = static_cast<const T *>(x.in) + t * x.ts + lane * x.hs + e;
            T *out = x.out ? static_cast<T *>(x.out) + t * x.o_ts + lane * x.o_hs + e : nullptr;
            if (APPEND && !turned && out == in && !page) return;  // (queries in place, nothing to turn)
            if (APPEND && page) page += to + lane * p.head_stride + e;
            for (int h = lane; h < x.n; h += s.lanes) {
                Vec<T, W> a = ld_vec<T, W>(in), b = ld_vec<T, W>(in + apart);
                in += s.lanes * x.hs;
                if (turn && turned) turn_pairs<T, W, IL>(a, b, cosines + first, sines + first);
                if (out) {
                    st_vec<T, W>(out, a);
                    st_vec<T, W>(out + apart, b);
                    out += s.lanes * x.o_hs;
                }
                if (APPEND && page) {
                    st_vec<T, W>(page, a);
                    st_vec<T, W>(page + apart, b);
                    page += s.lanes * p.head_stride;
                }
            }
        };
        heads(p.q, true, nullptr);
        heads(p.k, true, APPEND ? static_cast<T *>(p.k_pages) : nullptr);
        if (APPEND) heads(p.v, false, static_cast<T *>(p.v_pages));
    }
}

// The widest units (16 bytes of elements, four, two or one): W pairs or 2 W
// elements of what is not turned (nobody's where all is turned in place), all
// addresses multiples of W elements.
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
    for (int w : {16 / bytes, 4, 2}) {
        const int align = w * bytes;
        if (p.rot / 2 % w == 0 && p.rest % w == 0 && at % align == 0 && strides * bytes % align == 0) return w;
    }
    return 1;
}

template <typename T, int W, bool APPEND>
cudaError_t go(const RotaryParams &p, cudaStream_t stream) {
    Shape s;
    s.pairs = p.rot / 2 / W;
    s.units = s.pairs + (p.rest / W + 1) / 2;
    if (s.units == 0) return cudaSuccess;  // all in place, nothing to turn
    const int heads = std::max(1, p.q.n + p.k.n + p.v.n);
    // A warp a token where there are enough of them to fill the GPU (35507 tokens of 40
    // heads of 128: 113 us; twice as many threads a token 113, half as many 116); with
    // fewer, more threads share a token's heads (12 of them: 3.0 us, with a warp each 4).
    const int64_t fill = 152 * 5 * kThreads / (p.num_tokens * s.units);
    s.lanes = (int)std::max<int64_t>(1, std::min<int64_t>({std::max<int64_t>(fill, 32 / s.units), heads, kThreads / s.units}));
    s.slots = std::min(kThreads, s.units * s.lanes);
    s.tokens = kThreads / s.slots;
    const int64_t blocks = (p.num_tokens + s.tokens - 1) / s.tokens;
    if (blocks > INT32_MAX) return cudaErrorInvalidValue;
    const dim3 grid((unsigned)blocks);
    const size_t smem = 8 * (size_t)s.tokens * s.pairs * W;
    return p.interleaved ? launch_kernel(rotary<T, W, true, APPEND>, grid, kThreads, smem, stream, 0, true, p, s)
                         : launch_kernel(rotary<T, W, false, APPEND>, grid, kThreads, smem, stream, 0, true, p, s);
}

template <typename T, bool APPEND>
cudaError_t pick(const RotaryParams &p, cudaStream_t stream) {
    constexpr int kWide = 16 / (int)sizeof(T);
    const int w = width_for(p, (int)sizeof(T));
    if (w == kWide) return go<T, kWide, APPEND>(p, stream);
    if (w == 4) return go<T, 4, APPEND>(p, stream);
    return w == 2 ? go<T, 2, APPEND>(p, stream) : go<T, 1, APPEND>(p, stream);
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
