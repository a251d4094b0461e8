// Logits of drafted tokens to what verification takes: penalties, biases,
// masks, temperature, softmax; and the counts of tokens that penalties go by.
// See include/csgmv.h (csgmv_process_logits, csgmv_count_*).
//
// A row is read once and written once: a cluster of up to eight CTAs holds it in
// shared memory as f32, a stretch each.  What is sparse (the tokens that a
// sequence has, a row's branch, biases) is then put right in place: a sequence's
// distinct tokens come as a list beside the dense counts, so a row costs as many
// gathers as it has tokens, not a pass over the vocabulary.  A thread takes the
// maximum and the sum of exponentials of its elements together (rescaled when
// a vector of them has a larger one); the CTAs exchange one pair of numbers, in a
// fixed order.
#include <algorithm>
#include <atomic>

#include "elements.cuh"
#include "serving.cuh"
#include "step.h"

namespace csgmv {
namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxBranch = 32 * kTreeMaxWords;
constexpr int kPrompt = 1 << 30;
constexpr int kMaxVocab = 1 << 18, kMaxCtas = 8;
constexpr float kLargest = 3.402823466e+38f;

struct Pair {
    float top, sum;
    int at, bad;  // lowest place of top; whether there is a NaN
};
struct Smem {
    int branch[kMaxBranch];
    int n_branch;
    Pair warp[kWarps];
    Pair cta;
};

// The sum of two parts' exponentials about the larger of their maxima.
__device__ __forceinline__ Pair join(const Pair &a, const Pair &b, float heat) {
    Pair r;
    r.top = fmaxf(a.top, b.top);
    // (two maxima of -infinity, or of infinity, are no difference)
    const float fa = a.top == r.top ? 1.0f : exp2f((a.top - r.top) * heat), fb = b.top == r.top ? 1.0f : exp2f((b.top - r.top) * heat);
    r.sum = a.sum * fa + b.sum * fb;
    r.at = a.top > b.top || (a.top == b.top && a.at < b.at) ? a.at : b.at;
    r.bad = a.bad | b.bad;
    return r;
}
__device__ __forceinline__ Pair shfl_xor(const Pair &p, int o) {
    Pair r;
    r.top = __shfl_xor_sync(kFullMask, p.top, o);
    r.sum = __shfl_xor_sync(kFullMask, p.sum, o);
    r.at = __shfl_xor_sync(kFullMask, p.at, o);
    r.bad = __shfl_xor_sync(kFullMask, p.bad, o);
    return r;
}
__device__ __forceinline__ Pair warp_join(Pair p, float heat) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        const Pair q = shfl_xor(p, o);
        p = join(p, q, heat);
    }
    return p;
}

// z after what has been given before, each step rounded: `word` the sequence's
// count (and prompt bit), `extra` more of the row's branch.
__device__ __forceinline__ float penalized(float z, int word, int extra, float rho, float alpha, float beta) {
    const int c = (word & (kPrompt - 1)) + extra;
    if ((word | extra) != 0) z = z > 0.0f ? __fdiv_rn(z, rho) : __fmul_rn(z, rho);
    if (c > 0) z = __fsub_rn(__fsub_rn(z, __fmul_rn(alpha, (float)c)), beta);
    return z;
}

template <typename T, int V>
__global__ void __launch_bounds__(kThreads) process(LogitParams p) {
    extern __shared__ float4 stretch4[];
    float *z = reinterpret_cast<float *>(stretch4);
    __shared__ Smem sm;
    griddep_launch_dependents();
    griddep_wait();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int ctas = (int)cluster_size(), rank = (int)cluster_rank();
    const int t = blockIdx.x / ctas;
    // this CTA's stretch of the row
    const int lo = min(p.vocab, rank * p.chunk), n = min(p.vocab, lo + p.chunk) - lo;
    // the row's request: the last one that begins at or before it, 32 tried at once
    int b = 0;
    for (int len = p.bs; len > 1;) {
        const int step = (len + 31) >> 5, at = lane * step;
        const unsigned m = __ballot_sync(kFullMask, at < len && p.indptr[b + at] <= t);
        const int k = m ? 31 - __clz(m) : 0;
        b += k * step;
        len = min(step, len - k * step);
    }
    const int first = p.indptr[b], end = p.indptr[b + 1];
    const int seq = p.slots ? p.slots[b] : b;
    const float rho = p.repetition ? p.repetition[b] : 1.0f, alpha = p.frequency ? p.frequency[b] : 0.0f,
                beta = p.presence ? p.presence[b] : 0.0f, temperature = p.temperature ? p.temperature[b] : 1.0f;
    int b0 = 0, b1 = 0;
    if (p.bias_indptr) b0 = p.bias_indptr[b], b1 = p.bias_indptr[b + 1];
    const int gate = p.allow_index ? p.allow_index[t] : -1;
    // (rows of no request say nothing)
    bool mine = t >= first && t < end;
    int bad = 0;
    if (mine) {
        if (first < 0 || end > p.num_tokens) bad = CSGMV_KV_STATUS_BAD_LENS;
        else if (p.counts && (seq < 0 || seq >= p.max_seqs)) bad = CSGMV_KV_STATUS_BAD_SEQ;
        else if (!(rho > 0.0f) || !(rho <= kLargest) || !(temperature >= 0.0f) || !(temperature <= kLargest) || alpha != alpha ||
                 beta != beta || gate < -1 || gate >= p.num_allow ||
                 b0 < 0 || b1 < b0 || b1 > p.bias_total)
            bad = CSGMV_KV_STATUS_BAD_VALUE;
        else if (p.bias_indptr) {  // in order?
            bool torn = false;
            for (int i = b0 + 1 + tid; i < b1; i += kThreads) torn |= p.bias_tokens[i] < p.bias_tokens[i - 1];
            if (__syncthreads_or(torn)) bad = CSGMV_KV_STATUS_BAD_VALUE;
        }
        if (bad) {
            mine = false;
            if (rank == 0 && tid == 0) atomicOr(p.status, bad);
        }
    }
    if (!mine) return;  // every CTA of the cluster alike
    const uint32_t *allow = gate >= 0 ? reinterpret_cast<const uint32_t *>(p.allow) + (int64_t)gate * p.allow_words : nullptr;
    auto allowed = [&](int v) { return !allow || (allow[v >> 5] >> (v & 31) & 1u); };
    const T *row = static_cast<const T *>(p.logits) + t * p.logits_s;
    const float none = __int_as_float(0xff800000);
    // the row, what is not allowed out of it
    for (int i = tid * V; i < n; i += kThreads * V) {
        const Vec<T, V> x = ld_vec<T, V>(row + lo + i);
        const uint32_t pass = allow ? allow[(lo + i) >> 5] >> ((lo + i) & 31) : ~0u;
#pragma unroll
        for (int e = 0; e < V; ++e) z[i + e] = pass >> e & 1u ? to_f32(x.e[e]) : none;
    }
    // its branch
    const bool branch = p.mask != nullptr;
    if (branch && warp == 0) {
        int k = 0;
        for (int w = 0; w < p.mask_words; ++w) {
            const uint32_t bits = (uint32_t)p.mask[(int64_t)t * p.mask_words + w];
            const int j = 32 * w + lane;
            int v = -1;
            if ((bits >> lane & 1u) && j < end - first) {
                v = p.drafts[first + j];
                if (v < 0 || v >= p.vocab) {
                    if (rank == 0) atomicOr(p.status, CSGMV_KV_STATUS_BAD_TOKEN);
                    v = -1;
                }
            }
            const unsigned m = __ballot_sync(kFullMask, v >= 0);
            if (v >= 0) sm.branch[k + __popc(m & ((1u << lane) - 1u))] = v;
            k += __popc(m);
        }
        if (lane == 0) sm.n_branch = k;
    }
    __syncthreads();
    const bool punish = rho != 1.0f || alpha != 0.0f || beta != 0.0f;
    const int32_t *counts = p.counts ? p.counts + (int64_t)seq * p.vocab : nullptr;
    if (punish && counts) {
        const int32_t *seen = p.seen + (int64_t)seq * p.vocab;
        const int k = min(p.num_seen[seq], p.vocab);
        for (int i = tid; i < k; i += kThreads) {
            const int v = seen[i];
            if (v < lo || v >= lo + n || !allowed(v)) continue;
            z[v - lo] = penalized(z[v - lo], counts[v], 0, rho, alpha, beta);
        }
    }
    if (punish && branch) {
        __syncthreads();
        // the first of equal tokens counts for all; what the list did to it is undone
        const int k = sm.n_branch;
        for (int i = tid; i < k; i += kThreads) {
            const int v = sm.branch[i];
            if (v < lo || v >= lo + n || !allowed(v)) continue;
            int times = 0;
            bool leads = true;
            for (int j = 0; j < k; ++j) {
                const bool same = sm.branch[j] == v;
                times += same;
                leads &= !(same && j < i);
            }
            if (leads) z[v - lo] = penalized(to_f32(row[v]), counts ? counts[v] : 0, times, rho, alpha, beta);
        }
    }
    if (b1 > b0) {
        __syncthreads();
        for (int i = b0 + tid; i < b1; i += kThreads) {
            const int v = p.bias_tokens[i];
            if (v < 0 || v >= p.vocab) {
                if (rank == 0) atomicOr(p.status, CSGMV_KV_STATUS_BAD_TOKEN);
                continue;
            }
            if (v < lo || v >= lo + n || !allowed(v) || (i > b0 && p.bias_tokens[i - 1] == v)) continue;
            float s = z[v - lo];
            for (int j = i; j < b1 && p.bias_tokens[j] == v; ++j) s = __fadd_rn(s, p.bias_values[j]);
            z[v - lo] = s;
        }
    }
    __syncthreads();
    float *out = p.out + t * p.out_s + lo;
    if (!p.softmax) {
        for (int i = tid * V; i < n; i += kThreads * V) {
            Vec<float, V> o;
#pragma unroll
            for (int e = 0; e < V; ++e) o.e[e] = z[i + e];
            st_vec<float, V>(out + i, o);
        }
        return;
    }
    // exp((z - top) / temperature) = 2^((z - top) heat)
    const bool greedy = temperature == 0.0f;
    const float heat = greedy ? 0.0f : fminf(1.4426950408889634f / temperature, kLargest);
    Pair mine_p = {none, 0.0f, INT32_MAX, 0};
    for (int i = tid * V; i < n; i += kThreads * V) {
        float x[V], top = none;
#pragma unroll
        for (int e = 0; e < V; ++e) x[e] = z[i + e], top = fmaxf(top, x[e]), mine_p.bad |= x[e] != x[e];
        if (top > mine_p.top) {
            mine_p.sum *= exp2f((mine_p.top - top) * heat);
            mine_p.top = top;
#pragma unroll
            for (int e = V - 1; e >= 0; --e)
                if (x[e] == top) mine_p.at = lo + i + e;
        }
        if (mine_p.top != none)
#pragma unroll
            for (int e = 0; e < V; ++e) mine_p.sum += exp2f((x[e] - mine_p.top) * heat);
    }
    mine_p = warp_join(mine_p, heat);
    if (lane == 0) sm.warp[warp] = mine_p;
    __syncthreads();
    if (warp == 0) {
        const Pair q = warp_join(lane < kWarps ? sm.warp[lane] : Pair{none, 0.0f, INT32_MAX, 0}, heat);
        if (lane == 0) sm.cta = q;
    }
    cluster_sync();
    Pair all = {none, 0.0f, INT32_MAX, 0};
    for (int r = 0; r < ctas; ++r) {
        const uint32_t at = dsmem_addr(&sm.cta, r);
        const Pair q = {dsmem_ld_f32(at), dsmem_ld_f32(at + 4), dsmem_ld_i32(at + 8), dsmem_ld_i32(at + 12)};
        all = join(all, q, heat);
    }
    cluster_arrive();
    const float nan = __int_as_float(0x7fc00000);
    const bool infinite = all.top == __int_as_float(0x7f800000);
    const bool empty = all.top == none, lost = all.bad || (infinite && !greedy);
    const float share = empty ? 0.0f : __fdiv_rn(1.0f, all.sum);
    for (int i = tid * V; i < n; i += kThreads * V) {
        Vec<float, V> o;
#pragma unroll
        for (int e = 0; e < V; ++e) {
            const float x = z[i + e];
            if (greedy) o.e[e] = !empty && lo + i + e == all.at ? 1.0f : 0.0f;
            else o.e[e] = empty ? 0.0f : exp2f((x - all.top) * heat) * share;
            if (lost) o.e[e] = nan;
        }
        st_vec<float, V>(out + i, o);
    }
    cluster_wait();  // no CTA's numbers go before all have been read
}

// ------------------------------------------------------------------- counts
// A CTA a stretch of a request's tokens (blockIdx.y).  Order does not matter: the
// counts are sums, and seen is a set.
constexpr int kCountThreads = 256;
__global__ void __launch_bounds__(kCountThreads) count_tokens(CountParams p) {
    griddep_launch_dependents();
    griddep_wait();
    const int b = blockIdx.x;
    const int lo = p.indptr[b], hi = p.indptr[b + 1], seq = p.slots ? p.slots[b] : b;
    const int add = p.accept_len ? p.accept_len[b] : hi - lo;
    int bad = 0;
    if (seq < 0 || seq >= p.max_seqs) bad = CSGMV_KV_STATUS_BAD_SEQ;
    else if (add < 0 || lo < 0 || hi < lo || hi > p.num_tokens || add > (p.accept_index ? p.accept_width : hi - lo))
        bad = CSGMV_KV_STATUS_BAD_LENS;
    else if (p.accept_index) {
        bool wrong = false;
        for (int j = threadIdx.x; j < add; j += kCountThreads) {
            const int node = p.accept_index[(int64_t)b * p.accept_width + j];
            wrong |= node < 0 || node >= hi - lo;
        }
        if (__syncthreads_or(wrong)) bad = CSGMV_KV_STATUS_BAD_TREE;
    }
    if (bad) {
        if (threadIdx.x == 0 && blockIdx.y == 0) atomicOr(p.status, bad);
        return;
    }
    int32_t *counts = p.counts + (int64_t)seq * p.vocab, *seen = p.seen + (int64_t)seq * p.vocab;
    for (int64_t j = (int64_t)blockIdx.y * kCountThreads + threadIdx.x; j < add; j += (int64_t)gridDim.y * kCountThreads) {
        const int node = p.accept_index ? p.accept_index[(int64_t)b * p.accept_width + j] : (int)j;
        const int v = p.tokens[lo + node];
        if (v < 0 || v >= p.vocab) {
            atomicOr(p.status, CSGMV_KV_STATUS_BAD_TOKEN);
            continue;
        }
        const int was = p.prompt ? atomicOr(counts + v, kPrompt) : atomicAdd(counts + v, 1);
        if (was == 0) {  // the first to come lists it
            const int at = atomicAdd(p.num_seen + seq, 1);
            if (at >= 0 && at < p.vocab) seen[at] = v;
        }
    }
}

__global__ void __launch_bounds__(kThreads) count_reset(CountParams p) {
    griddep_launch_dependents();
    griddep_wait();
    const int seq = p.slots[blockIdx.x];
    if (seq < 0 || seq >= p.max_seqs) {
        if (threadIdx.x == 0) atomicOr(p.status, CSGMV_KV_STATUS_BAD_SEQ);
        return;
    }
    int32_t *counts = p.counts + (int64_t)seq * p.vocab;
    const int32_t *seen = p.seen + (int64_t)seq * p.vocab;
    // (a sequence that is listed twice may be found empty already)
    const int k = min(*(volatile int32_t *)(p.num_seen + seq), p.vocab);
    for (int i = threadIdx.x; i < k; i += kThreads) {
        const int v = seen[i];
        if (v >= 0 && v < p.vocab) counts[v] = 0;
    }
    __syncthreads();
    if (threadIdx.x == 0) p.num_seen[seq] = 0;
}

__global__ void __launch_bounds__(kThreads) count_fork(CountParams p, const int32_t *parents, const int32_t *children, int n) {
    griddep_launch_dependents();
    griddep_wait();
    const int i = blockIdx.x, a = parents[i], b = children[i];
    bool wrong = a < 0 || a >= p.max_seqs || b < 0 || b >= p.max_seqs;
    if (!wrong) {
        for (int j = threadIdx.x; j < n; j += kThreads) wrong |= parents[j] == b || (j < i && children[j] == b);
        wrong |= p.num_seen[b] != 0;
    }
    if (__syncthreads_or(wrong)) {
        if (threadIdx.x == 0) atomicOr(p.status, CSGMV_KV_STATUS_BAD_SEQ);
        return;
    }
    const int64_t from = (int64_t)a * p.vocab, to = (int64_t)b * p.vocab;
    const int k = min(p.num_seen[a], p.vocab);
    for (int j = threadIdx.x; j < k; j += kThreads) {
        const int v = p.seen[from + j];
        if (v < 0 || v >= p.vocab) continue;
        p.seen[to + j] = v;
        p.counts[to + v] = p.counts[from + v];
    }
    __syncthreads();  // (all have found it empty)
    if (threadIdx.x == 0) p.num_seen[b] = k;
}

constexpr int kMaxDevices = 64;
std::atomic<bool> g_ready[kMaxDevices];  // whether the kernels may use all the shared memory they need (twice does no harm)

cudaError_t prepare() {
    int dev;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < kMaxDevices && g_ready[dev].load(std::memory_order_acquire)) return cudaSuccess;
    for (const void *fn : {reinterpret_cast<const void *>(process<__nv_bfloat16, 8>), reinterpret_cast<const void *>(process<__nv_bfloat16, 1>),
                           reinterpret_cast<const void *>(process<__half, 8>), reinterpret_cast<const void *>(process<__half, 1>),
                           reinterpret_cast<const void *>(process<float, 4>), reinterpret_cast<const void *>(process<float, 1>)}) {
        if ((e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxVocab / kMaxCtas * 4)) != cudaSuccess)
            return e;
        if ((e = cudaFuncSetAttribute(fn, cudaFuncAttributePreferredSharedMemoryCarveout, cudaSharedmemCarveoutMaxShared)) != cudaSuccess)
            return e;
    }
    if (dev < kMaxDevices) g_ready[dev].store(true, std::memory_order_release);
    return cudaSuccess;
}

template <typename T, int V>
cudaError_t go(const LogitParams &p, int ctas, cudaStream_t stream) {
    const cudaError_t e = prepare();
    if (e != cudaSuccess) return e;
    return launch_kernel(process<T, V>, dim3((unsigned)(p.num_tokens * ctas)), kThreads, (size_t)p.chunk * sizeof(float), stream,
                         ctas, true, p);
}

template <typename T>
cudaError_t pick(LogitParams p, cudaStream_t stream) {
    // The fewest CTAs whose stretch leaves room for three of them in an SM, and more
    // of them for a row while there are not enough rows for the SMs.
    int ctas = 1;
    while (ctas < kMaxCtas && ((int64_t)p.vocab > (int64_t)ctas * 16384 || (p.num_tokens * ctas * 2 <= 152 && p.vocab > ctas * 2048))) ctas *= 2;
    p.chunk = ((p.vocab + ctas - 1) / ctas + 31) & ~31;
    constexpr int V = 16 / (int)sizeof(T);
    const bool wide = p.logits_s % V == 0 && p.out_s % 4 == 0 && p.vocab % V == 0 &&
                      ((reinterpret_cast<uintptr_t>(p.logits) | reinterpret_cast<uintptr_t>(p.out)) & 15) == 0;
    return wide ? go<T, V>(p, ctas, stream) : go<T, 1>(p, ctas, stream);
}

}  // namespace

cudaError_t launch_process_logits(const LogitParams &p, cudaStream_t stream) {
    switch (p.dtype) {
        case CSGMV_DTYPE_BF16: return pick<__nv_bfloat16>(p, stream);
        case CSGMV_DTYPE_F16: return pick<__half>(p, stream);
        default: return pick<float>(p, stream);
    }
}

cudaError_t launch_count_tokens(const CountParams &p, int bs, cudaStream_t stream) {
    // enough CTAs a request for a long prompt, few where there are many requests
    const int64_t per = (p.num_tokens + bs - 1) / bs;
    const unsigned y = (unsigned)std::max<int64_t>(1, std::min<int64_t>(64, (per + kCountThreads - 1) / kCountThreads));
    return launch_kernel(count_tokens, dim3((unsigned)bs, y), kCountThreads, 0, stream, 0, true, p);
}
cudaError_t launch_count_reset(const CountParams &p, int n, cudaStream_t stream) {
    return launch_kernel(count_reset, dim3((unsigned)n), kThreads, 0, stream, 0, true, p);
}
cudaError_t launch_count_fork(const CountParams &p, const int32_t *parents, const int32_t *children, int n, cudaStream_t stream) {
    return launch_kernel(count_fork, dim3((unsigned)n), kThreads, 0, stream, 0, true, p, parents, children, n);
}

}  // namespace csgmv
