// Attention of draft trees over the paged cache (include/csgmv.h,
// csgmv_tree_attention).
//
// The plain kernel: a block a query row and head, a thread a token for the
// scores and a thread an element for the sums, with the running maximum and
// sum of a softmax over tiles of 128 tokens.
#include <cuda_fp16.h>

#include "serving.cuh"

namespace csgmv {
namespace {

constexpr int kThreads = 128;

__device__ __forceinline__ float to_f32(uint16_t x, int f16) {
    return f16 ? __half2float(__ushort_as_half(x)) : __uint_as_float((uint32_t)x << 16);
}
__device__ __forceinline__ uint16_t from_f32(float x, int f16) {
    return f16 ? __half_as_ushort(__float2half_rn(x)) : __bfloat16_as_ushort(__float2bfloat16_rn(x));
}

__global__ void __launch_bounds__(kThreads) attend(AttnParams p) {
    __shared__ float q[128], e[kThreads], red[kThreads / 32];
    const int t = blockIdx.x, h = blockIdx.y, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    // the request that owns row t
    int b = 0;
    {
        int lo = 0, hi = p.bs;
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (p.indptr[mid] <= t) lo = mid; else hi = mid;
        }
        b = lo;
    }
    const int r0 = p.indptr[b], r1 = p.indptr[b + 1], n = r1 - r0;
    if (t < r0 || t >= r1) return;  // a row of no request
    const int slot = p.slots ? p.slots[b] : b;
    int bad = 0, len = 0;
    if (slot < 0 || slot >= p.max_seqs) bad = CSGMV_KV_STATUS_BAD_SEQ;
    else if ((len = p.seq_lens[slot]) < 0 || len > p.max_pages * p.page_size || r0 < 0 || r1 > p.num_tokens ||
             (p.mask && n > 32 * p.mask_words))
        bad = CSGMV_KV_STATUS_BAD_LENS;
    if (bad) {
        if (tid == 0) atomicOr(p.status, bad);
        return;
    }
    const int g = h / p.group;
    if (tid < p.d) q[tid] = to_f32(p.q[t * p.q_ts + h * p.q_hs + tid], p.f16);
    __syncthreads();
    const int32_t *table = p.page_table + (int64_t)slot * p.max_pages;
    auto place = [&](int i, const uint16_t *pages, const uint16_t *fresh) -> const uint16_t * {
        if (i >= len) return fresh + (int64_t)(r0 + i - len) * p.n_ts + g * p.n_hs;
        const int page = table[i / p.page_size];
        if (page < 0 || page >= p.num_pages) return nullptr;
        return pages + page * p.page_stride + g * p.head_stride + (int64_t)(i % p.page_size) * p.token_stride;
    };
    float m = -INFINITY, l = 0.0f, o = 0.0f;
    for (int i0 = 0; i0 < len + n; i0 += kThreads) {
        const int i = i0 + tid;
        bool sees = i < len;
        if (i >= len && i < len + n) {
            const int j = i - len;
            sees = p.mask ? (p.mask[(int64_t)t * p.mask_words + (j >> 5)] >> (j & 31)) & 1 : j <= t - r0;
        }
        float s = -INFINITY;
        if (sees) {
            const uint16_t *k = place(i, p.k_pages, p.k_new);
            if (k) {
                s = 0.0f;
                for (int x = 0; x < p.d; ++x) s += q[x] * to_f32(k[x], p.f16);
                s *= p.scale;
            } else {
                atomicOr(p.status, CSGMV_KV_STATUS_BAD_PAGE);
                sees = false;
            }
        }
        float top = s;
        for (int x = 16; x > 0; x >>= 1) top = fmaxf(top, __shfl_xor_sync(kFullMask, top, x));
        if (lane == 0) red[warp] = top;
        __syncthreads();
        top = fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3]));
        const float mn = fmaxf(m, top), base = mn == -INFINITY ? 0.0f : mn;
        const float w = sees ? expf(s - base) : 0.0f, f = expf(m - base);
        e[tid] = sees ? w : -1.0f;
        float sum = warp_sum(w);
        __syncthreads();
        if (lane == 0) red[warp] = sum;
        __syncthreads();
        l = l * f + red[0] + red[1] + red[2] + red[3];
        o *= f;
        m = mn;
        if (tid < p.d)
            for (int y = 0; y < kThreads && i0 + y < len + n; ++y) {
                if (e[y] == -1.0f) continue;  // not seen: no influence whatever it holds
                o += e[y] * to_f32(place(i0 + y, p.v_pages, p.v_new)[tid], p.f16);
            }
        __syncthreads();
    }
    if (tid < p.d) p.out[t * p.o_ts + h * p.o_hs + tid] = from_f32(l == 0.0f ? 0.0f : o / l, p.f16);
    if (tid == 0 && p.lse) p.lse[(int64_t)t * p.hq + h] = l == 0.0f ? -INFINITY : m + logf(l);
}

}  // namespace

size_t attn_workspace_bytes(int head_dim) { return 0; }

cudaError_t launch_tree_attention(const AttnParams &p, void *workspace, cudaStream_t stream) {
    return launch_kernel(attend, dim3((unsigned)p.num_tokens, (unsigned)p.hq), kThreads, 0, stream, 0, false, p);
}

}  // namespace csgmv
