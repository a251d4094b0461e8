// Logits of drafted tokens to what verification takes: penalties, biases,
// masks, temperature, softmax; and the counts of tokens that penalties go by.
// See include/csgmv.h (csgmv_process_logits, csgmv_count_*).
//
// A cluster of up to eight CTAs has a row, a stretch each, that it copies to
// shared memory as it is, before it knows whose it is.  What is sparse is put
// right while that arrives: the tokens that a sequence holds (they come as a list
// beside the dense counts, so a row costs as many gathers as it has tokens, not a
// pass over the vocabulary), the row's branch, biases; each such token has one
// thread (a bit for each, the number of bits before it: a list in the order of
// the vocabulary, whatever that of the counts' list, so results do not depend on
// it).  f32 scores go back to their places; those of 16-bit logits are kept beside, and
// their places become -infinity.  Two passes over the stretch follow, both in shared memory: the
// maximum and the sum of exponentials together, then the probabilities.  The
// CTAs of a row exchange one pair of numbers in between.
#include <algorithm>
#include <atomic>

#include "elements.cuh"
#include "serving.cuh"
#include "step.h"

namespace csgmv {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxBranch = 32 * kTreeMaxWords;
constexpr int kPrompt = 1 << 30;
constexpr int kMaxVocab = 1 << 18, kMaxCtas = 8;
constexpr int kKept = 1024;  // scores beside a stretch of 16-bit logits; further ones wait in out
constexpr float kLargest = 3.402823466e+38f;

// A part of a row: its largest score, and the sum of 2^((z - top) heat), which
// is NaN where a score is.  (temperature 0: the sum is 0 or NaN.)
struct Part {
    float top, sum;
    int at;  // temperature 0: the lowest place of top
};
struct Smem {
    int branch[kMaxBranch];
    float kept[kKept];
    uint16_t place[kKept];
    int n_branch;
    int scan[33];
    Part warp[kWarps];
    Part ctas[kMaxCtas];
};
// Shared memory of a stretch of up to `chunk` elements, which begins up to 15
// bytes behind a 16-byte boundary: the elements; a bit for each of those whose score
// is another; how many of these are set before each word.
struct Stretch {
    int elements, words;  // bytes, and words of bits
};
__host__ __device__ inline Stretch stretch_of(int chunk, int bytes) { return {(chunk * bytes + 16 + 15) & ~15, (chunk + 16 + 31) >> 5}; }

// 2^x to two units in the last place, what is below 2^-126 as 0.
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// What a sum about `top` counts about `about` (equal infinities are no difference).
__device__ __forceinline__ float shifted(float sum, float top, float about, float heat) {
    return top == about ? sum : sum * ex2((top - about) * heat);
}
__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(kFullMask, v, o));
    return v;
}
// The parts of a warp's lanes as one, in all of them.
__device__ __forceinline__ Part warp_join(Part p, bool greedy, float heat) {
    Part r;
    r.top = warp_max(p.top);
    r.sum = warp_sum(shifted(p.sum, p.top, r.top, heat));
    r.at = greedy ? __reduce_min_sync(kFullMask, p.top == r.top ? p.at : INT32_MAX) : 0;
    return r;
}

// z after what has been given before, each step rounded: `word` the sequence's
// count (and prompt bit), `extra` more of the row's branch.
__device__ __forceinline__ float penalized(float z, int word, int extra, float rho, float alpha, float beta) {
    const int c = (word & (kPrompt - 1)) + extra;
    if ((word | extra) != 0) z = z > 0.0f ? __fdiv_rn(z, rho) : __fmul_rn(z, rho);
    if (c > 0) z = __fsub_rn(__fsub_rn(z, __fmul_rn(alpha, (float)c)), beta);
    return z;
}

template <int W>
__device__ __forceinline__ void store(float *p, const float (&x)[W]) {
    if constexpr (W == 8)
        asm volatile("st.global.cs.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "f"(x[0]), "f"(x[1]), "f"(x[2]), "f"(x[3]),
                     "f"(x[4]), "f"(x[5]), "f"(x[6]), "f"(x[7])
                     : "memory");
    else
        __stcs(reinterpret_cast<float4 *>(p), make_float4(x[0], x[1], x[2], x[3]));
}
__device__ __forceinline__ void prefetch(const void *p) { asm volatile("prefetch.global.L1 [%0];" ::"l"(p)); }
__device__ __forceinline__ bool has(const uint32_t *bits, int i) { return (bits[i >> 5] >> (i & 31) & 1u) != 0; }
__device__ __forceinline__ void mark(uint32_t *bits, int i) { atomicOr(bits + (i >> 5), 1u << (i & 31)); }

template <typename T>
__global__ void __launch_bounds__(kThreads, 5) process(LogitParams p) {
    extern __shared__ uint4 dynamic[];
    __shared__ Smem sm;
    constexpr int W = 16 / (int)sizeof(T);  // elements of a vector
    constexpr bool kBeside = sizeof(T) == 2;
    const Stretch shape = stretch_of(p.chunk, sizeof(T));
    T *z = reinterpret_cast<T *>(dynamic);
    uint32_t *set = reinterpret_cast<uint32_t *>(reinterpret_cast<char *>(dynamic) + shape.elements);
    uint16_t *before = reinterpret_cast<uint16_t *>(set + shape.words);
    griddep_launch_dependents();
    cluster_arrive();
    griddep_wait();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int ctas = (int)cluster_size(), rank = (int)cluster_rank();
    const int t = blockIdx.x / ctas;
    // this CTA's stretch of the row: elements begin .. end of z, as far behind a vector as in memory
    const int lo = min(p.vocab, rank * p.chunk), n = min(p.vocab, lo + p.chunk) - lo;
    const T *row = static_cast<const T *>(p.logits) + t * p.logits_s + lo;
    const int begin = (int)(reinterpret_cast<uintptr_t>(row) % 16 / sizeof(T)), end = begin + n;
    const float none = __int_as_float(0xff800000);
    for (int i = tid * W; i < end; i += kThreads * W) {
        if (i >= begin && i + W <= end) cp_async16(z + i, row + (i - begin), 16);
        else
            for (int e = i; e < i + W; ++e) z[e] = e >= begin && e < end ? row[e - begin] : from_f32<T>(none);
    }
    // the row's request: the last one that begins at or before it, 32 tried at once
    int b = 0;
    for (int len = p.bs; len > 1;) {
        const int step = (len + 31) >> 5, at = lane * step;
        const unsigned m = __ballot_sync(kFullMask, at < len && p.indptr[b + at] <= t);
        const int k = m ? 31 - __clz(m) : 0;
        b += k * step;
        len = min(step, len - k * step);
    }
    const int first = p.indptr[b], last = p.indptr[b + 1];
    const int seq = p.slots ? p.slots[b] : b;
    const float rho = p.repetition ? p.repetition[b] : 1.0f, alpha = p.frequency ? p.frequency[b] : 0.0f,
                beta = p.presence ? p.presence[b] : 0.0f, temperature = p.temperature ? p.temperature[b] : 1.0f;
    int b0 = 0, b1 = 0;
    if (p.bias_indptr) b0 = p.bias_indptr[b], b1 = p.bias_indptr[b + 1];
    const int gate = p.allow_index ? p.allow_index[t] : -1;
    // (rows of no request say nothing)
    bool mine = t >= first && t < last;
    if (mine) {
        int bad = 0;
        if (first < 0 || last > p.num_tokens) bad = CSGMV_KV_STATUS_BAD_LENS;
        else if (p.counts && (seq < 0 || seq >= p.max_seqs)) bad = CSGMV_KV_STATUS_BAD_SEQ;
        else if (!(rho > 0.0f) || !(rho <= kLargest) || !(temperature >= 0.0f) || !(temperature <= kLargest) || alpha != alpha ||
                 beta != beta || gate < -1 || gate >= p.num_allow || b0 < 0 || b1 < b0 || b1 > p.bias_total)
            bad = CSGMV_KV_STATUS_BAD_VALUE;
        if (bad) {
            mine = false;
            if (rank == 0 && tid == 0) atomicOr(p.status, bad);
        }
    }
    if (!mine) {  // every CTA of the cluster alike
        cp_async_wait_all();
        return;
    }
    const uint32_t *allow = gate >= 0 ? reinterpret_cast<const uint32_t *>(p.allow) + (int64_t)gate * p.allow_words : nullptr;
    float *out = p.out + t * p.out_s + lo - begin;  // out[i] is the place of z[i]
    // where a token is in z if it is this CTA's to put right, or -1
    auto place = [&](int token) { return token >= lo && token < lo + n && (!allow || has(allow, token)) ? token - lo + begin : -1; };
    const bool punish = rho != 1.0f || alpha != 0.0f || beta != 0.0f, branch = punish && p.mask;
    const int32_t *counts = punish && p.counts ? p.counts + (int64_t)seq * p.vocab + lo - begin : nullptr;
    const int32_t *seen = counts ? p.seen + (int64_t)seq * p.vocab : nullptr;
    const int held = counts ? min(p.num_seen[seq], p.vocab) : 0;
    const bool sparse = held > 0 || branch || b1 > b0;
    // the first tokens that the sequence holds, where they are, and their counts on the way
    constexpr int S = 4;
    int held_at[S];
    auto load_held = [&](int i0) {
#pragma unroll
        for (int u = 0; u < S; ++u) held_at[u] = i0 + tid + u * kThreads < held ? seen[i0 + tid + u * kThreads] : -1;
#pragma unroll
        for (int u = 0; u < S; ++u) held_at[u] = place(held_at[u]);
    };
    load_held(0);
#pragma unroll
    for (int u = 0; u < S; ++u)
        if (held_at[u] >= 0) prefetch(counts + held_at[u]);
    if (sparse) {
        if (b0 + tid < b1) prefetch(p.bias_tokens + b0 + tid), prefetch(p.bias_values + b0 + tid);
        for (int i = tid; i < shape.words; i += kThreads) set[i] = 0;
        if (branch && warp == 0) {
            int k = 0;
            for (int w = 0; w < p.mask_words; ++w) {
                const uint32_t bits = (uint32_t)p.mask[(int64_t)t * p.mask_words + w];
                const int j = 32 * w + lane;
                int token = -1;
                if ((bits >> lane & 1u) && j < last - first) {
                    token = p.drafts[first + j];
                    if (token < 0 || token >= p.vocab) {
                        if (rank == 0) atomicOr(p.status, CSGMV_KV_STATUS_BAD_TOKEN);
                        token = -1;
                    }
                }
                const unsigned m = __ballot_sync(kFullMask, token >= 0);
                if (token >= 0) sm.branch[k + __popc(m & ((1u << lane) - 1u))] = token;
                k += __popc(m);
            }
            if (lane == 0) sm.n_branch = k;
        }
    }
    cp_async_wait_all();
    __syncthreads();
    if (allow) {  // what is not allowed, out of the stretch
#pragma unroll 4
        for (int i = tid * W; i < end; i += kThreads * W) {
            const int token = lo + i - begin, from = max(token, 0);  // of the first element, which may be before the stretch
            uint32_t bits = allow[from >> 5] >> (from & 31);
            if ((from & 31) + W > 32 && (from | 31) + 1 < p.vocab) bits |= allow[(from >> 5) + 1] << (32 - (from & 31));
            bits <<= from - token;
            Vec<T, W> v = *reinterpret_cast<const Vec<T, W> *>(z + i);
#pragma unroll
            for (int e = 0; e < W; ++e) v.e[e] = bits >> e & 1u ? v.e[e] : from_f32<T>(none);
            *reinterpret_cast<Vec<T, W> *>(z + i) = v;
        }
    }
    int done = 0;  // scores that are not the row's own
    if (sparse) {
        const int k = branch ? sm.n_branch : 0;
        for (int i = tid; i < k; i += kThreads)
            if (const int at = place(sm.branch[i]); at >= 0) mark(set, at);
        bool torn = false;
        for (int i = b0 + tid; i < b1; i += kThreads) {
            const int token = p.bias_tokens[i];
            torn |= i > b0 && token < p.bias_tokens[i - 1];
            if (token < 0 || token >= p.vocab) {
                if (rank == 0) atomicOr(p.status, CSGMV_KV_STATUS_BAD_TOKEN);
            } else if (const int at = place(token); at >= 0) {
                mark(set, at);
            }
        }
        for (int i0 = 0; i0 < held; i0 += S * kThreads) {
            if (i0 > 0) load_held(i0);
#pragma unroll
            for (int u = 0; u < S; ++u)
                if (held_at[u] >= 0) mark(set, held_at[u]);
        }
        if (__syncthreads_or(torn)) {  // biases out of order; every CTA of the cluster alike
            if (rank == 0 && tid == 0) atomicOr(p.status, CSGMV_KV_STATUS_BAD_VALUE);
            return;
        }
        for (int w0 = 0; w0 < shape.words; w0 += kThreads) {
            const int w = w0 + tid;
            const uint32_t word = w < shape.words ? set[w] : 0;
            int more, r = done + block_scan_ex(__popc(word), sm.scan, &more);
            if (w < shape.words) before[w] = (uint16_t)r;
            for (uint32_t bits = word; bits && r < kKept; bits &= bits - 1, ++r) sm.place[r] = (uint16_t)(32 * w + __ffs(bits) - 1);
            done += more;
        }
        __syncthreads();
        auto score = [&](int at, int r) {
            const int token = lo + at - begin;
            float x = to_f32(z[at]);
            if (punish) {
                const int word = counts ? counts[at] : 0;
                int more = 0;
                for (int j = 0; j < k; ++j) more += sm.branch[j] == token;
                x = penalized(x, word, more, rho, alpha, beta);
            }
            if (b1 > b0) {
                int i = b0;  // the first bias of the token
                for (int len = b1 - b0; len > 0;) {
                    const int half = len >> 1;
                    if (p.bias_tokens[i + half] < token) i += half + 1, len -= half + 1;
                    else len = half;
                }
                for (; i < b1 && p.bias_tokens[i] == token; ++i) x = __fadd_rn(x, p.bias_values[i]);
            }
            if constexpr (kBeside) {
                if (r < kKept) sm.kept[r] = x;
                else out[at] = x;
                z[at] = from_f32<T>(none);
            } else {
                z[at] = x;
            }
        };
        for (int r = tid; r < min(done, kKept); r += kThreads) score(sm.place[r], r);
        if (done > kKept)
            for (int w = tid; w < shape.words; w += kThreads) {
                int r = before[w];
                for (uint32_t bits = set[w]; bits; bits &= bits - 1, ++r)
                    if (r >= kKept) score(32 * w + __ffs(bits) - 1, r);
            }
    }
    if (sparse || allow) __syncthreads();
    auto vector = [&](int i, float (&x)[W]) {
        const Vec<T, W> v = *reinterpret_cast<const Vec<T, W> *>(z + i);
#pragma unroll
        for (int e = 0; e < W; ++e) x[e] = to_f32(v.e[e]);
    };
    // f(score, place) for those beside the stretch
    auto beside = [&](auto f) {
        for (int r = tid; kBeside && r < min(done, kKept); r += kThreads) f(sm.kept[r], sm.place[r]);
        if (kBeside && done > kKept)
            for (int w = tid; w < shape.words; w += kThreads) {
                int r = before[w];
                for (uint32_t bits = set[w]; bits; bits &= bits - 1, ++r)
                    if (r >= kKept) f(out[32 * w + __ffs(bits) - 1], 32 * w + __ffs(bits) - 1);
            }
    };
    // out = f(score, place), in vectors where those of out are where those of z are
    // and no score waits in out
    const bool wide = reinterpret_cast<uintptr_t>(out) % (4 * W) == 0 && (!kBeside || done <= kKept);
    auto write = [&](auto f) {
        if (wide) {
            for (int i = tid * W; i < end; i += kThreads * W) {
                float x[W];
                vector(i, x);
#pragma unroll
                for (int e = 0; e < W; ++e) x[e] = f(x[e], i + e);
                if (i >= begin && i + W <= end) store<W>(out + i, x);
                else
#pragma unroll
                    for (int e = 0; e < W; ++e)
                        if (i + e >= begin && i + e < end) out[i + e] = x[e];
            }
        } else {
#pragma unroll 4
            for (int i = begin + tid; i < end; i += kThreads)
                if (!kBeside || done <= kKept || !has(set, i)) out[i] = f(to_f32(z[i]), i);
        }
        if (kBeside && done > 0) {
            __syncthreads();
            beside([&](float x, int at) { out[at] = f(x, at); });
        }
    };
    if (!p.softmax) {
        write([](float x, int) { return x; });
        return;
    }
    // exp((z - top) / temperature) = 2^((z - top) heat)
    const bool greedy = temperature == 0.0f;
    const float heat = greedy ? 1.0f : fminf(1.4426950408889634f / temperature, kLargest);
    Part part = {none, 0.0f, INT32_MAX};
    if (greedy) {
        for (int i = tid * W; i < end; i += kThreads * W) {
            float x[W];
            vector(i, x);
#pragma unroll
            for (int e = 0; e < W; ++e) {
                if (x[e] > part.top) part.top = x[e], part.at = lo + i + e - begin;
                if (x[e] != x[e]) part.sum = x[e];
            }
        }
        beside([&](float x, int at) {
            const int token = lo + at - begin;
            if (x > part.top || (x == part.top && token < part.at)) part.top = x, part.at = token;
            if (x != x) part.sum = x;
        });
    } else {
        for (int i = tid * W; i < end; i += kThreads * W) {
            float x[W], s[W];
            vector(i, x);
            float top = x[0];
#pragma unroll
            for (int e = 1; e < W; ++e) top = fmaxf(top, x[e]);
            if (top > part.top) {
                part.sum *= ex2((part.top - top) * heat);
                part.top = top;
            }
            const float about = part.top == none ? 0.0f : part.top;
#pragma unroll
            for (int e = 0; e < W; ++e) s[e] = ex2((x[e] - about) * heat);
#pragma unroll
            for (int o = W / 2; o > 0; o >>= 1)
#pragma unroll
                for (int e = 0; e < o; ++e) s[e] += s[e + o];
            part.sum += s[0];
        }
        beside([&](float x, int) {
            if (x > part.top) {
                part.sum *= ex2((part.top - x) * heat);
                part.top = x;
            }
            part.sum += ex2((x - (part.top == none ? 0.0f : part.top)) * heat);
        });
    }
    part = warp_join(part, greedy, heat);
    if (lane == 0) sm.warp[warp] = part;
    __syncthreads();
    cluster_wait();  // (all have begun)
    if (warp == 0) {
        part = warp_join(lane < kWarps ? sm.warp[lane] : Part{none, 0.0f, INT32_MAX}, greedy, heat);
        if (lane < ctas) {  // to every CTA of the cluster
            const uint32_t to = dsmem_addr(&sm.ctas[rank], lane);
            dsmem_st_f32(to, part.top);
            dsmem_st_f32(to + 4, part.sum);
            dsmem_st_f32(to + 8, __int_as_float(part.at));
        }
    }
    cluster_sync();
    float top = none, sum = 0.0f;
    for (int r = 0; r < ctas; ++r) top = fmaxf(top, sm.ctas[r].top);
    for (int r = 0; r < ctas; ++r) sum += shifted(sm.ctas[r].sum, sm.ctas[r].top, top, heat);
    // a sum that is NaN makes all of the row that; nothing but -infinity makes it 0
    const float share = sum != sum ? sum : top == none ? 0.0f : greedy ? 1.0f : __fdiv_rn(1.0f, sum);
    if (greedy) {
        int at = INT32_MAX;
        for (int r = 0; r < ctas; ++r)
            if (sm.ctas[r].top == top) at = min(at, sm.ctas[r].at);
        write([&](float, int i) { return (lo + i - begin == at ? 1.0f : 0.0f) * share; });
    } else {
        // the exponential by halves: their product may be subnormal, they are not
        const float about = top == none ? 0.0f : top, half = 0.5f * heat;
        write([&](float x, int) {
            const float y = ex2((x - about) * half);
            return y * (y * share);
        });
    }
}

// ------------------------------------------------------------------- counts
// A CTA a stretch of a request's tokens (blockIdx.y).  Order does not matter: the
// counts are sums, and seen is a set.
constexpr int kCountThreads = 512;
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

__global__ void __launch_bounds__(kCountThreads) count_reset(CountParams p) {
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
    for (int i = threadIdx.x; i < k; i += kCountThreads) {
        const int v = seen[i];
        if (v >= 0 && v < p.vocab) counts[v] = 0;
    }
    __syncthreads();
    if (threadIdx.x == 0) p.num_seen[seq] = 0;
}

__global__ void __launch_bounds__(kCountThreads) count_fork(CountParams p, const int32_t *parents, const int32_t *children, int n) {
    griddep_launch_dependents();
    griddep_wait();
    const int i = blockIdx.x, a = parents[i], b = children[i];
    bool wrong = a < 0 || a >= p.max_seqs || b < 0 || b >= p.max_seqs;
    if (!wrong) {
        for (int j = threadIdx.x; j < n; j += kCountThreads) wrong |= parents[j] == b || (j < i && children[j] == b);
        wrong |= p.num_seen[b] != 0;
    }
    if (__syncthreads_or(wrong)) {
        if (threadIdx.x == 0) atomicOr(p.status, CSGMV_KV_STATUS_BAD_SEQ);
        return;
    }
    const int64_t from = (int64_t)a * p.vocab, to = (int64_t)b * p.vocab;
    const int k = min(p.num_seen[a], p.vocab);
    for (int j = threadIdx.x; j < k; j += kCountThreads) {
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

size_t smem_of(int chunk, int bytes) {
    const Stretch s = stretch_of(chunk, bytes);
    return (size_t)s.elements + 6 * (size_t)s.words;
}

cudaError_t prepare() {
    int dev;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < kMaxDevices && g_ready[dev].load(std::memory_order_acquire)) return cudaSuccess;
    const struct { const void *fn; int bytes; } all[] = {{reinterpret_cast<const void *>(process<__nv_bfloat16>), 2},
                                                         {reinterpret_cast<const void *>(process<__half>), 2},
                                                         {reinterpret_cast<const void *>(process<float>), 4}};
    for (const auto &f : all) {
        if ((e = cudaFuncSetAttribute(f.fn, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem_of(kMaxVocab / kMaxCtas, f.bytes))) !=
            cudaSuccess)
            return e;
        if ((e = cudaFuncSetAttribute(f.fn, cudaFuncAttributePreferredSharedMemoryCarveout, cudaSharedmemCarveoutMaxShared)) != cudaSuccess)
            return e;
    }
    if (dev < kMaxDevices) g_ready[dev].store(true, std::memory_order_release);
    return cudaSuccess;
}

template <typename T>
cudaError_t go(LogitParams p, cudaStream_t stream) {
    const cudaError_t e = prepare();
    if (e != cudaSuccess) return e;
    // CTAs of a row: stretches of up to 16384 elements (32768 where those would be more
    // than eight), and more of them while there are not enough rows for the SMs.
    int ctas = 1;
    while (ctas < kMaxCtas && ((int64_t)p.vocab > (int64_t)ctas * 16384 || (p.num_tokens * ctas * 2 <= 152 && p.vocab > ctas * 2048)))
        ctas *= 2;
    p.chunk = ((p.vocab + ctas - 1) / ctas + 31) & ~31;
    return launch_kernel(process<T>, dim3((unsigned)(p.num_tokens * ctas)), kThreads, smem_of(p.chunk, sizeof(T)), stream, ctas, true, p);
}

}  // namespace

cudaError_t launch_process_logits(const LogitParams &p, cudaStream_t stream) {
    switch (p.dtype) {
        case CSGMV_DTYPE_BF16: return go<__nv_bfloat16>(p, stream);
        case CSGMV_DTYPE_F16: return go<__half>(p, stream);
        default: return go<float>(p, stream);
    }
}

cudaError_t launch_count_tokens(const CountParams &p, int bs, cudaStream_t stream) {
    // enough CTAs a request for a long prompt, few where there are many requests
    const int64_t per = (p.num_tokens + bs - 1) / bs;
    const unsigned y = (unsigned)std::max<int64_t>(1, std::min<int64_t>(64, (per + kCountThreads - 1) / kCountThreads));
    return launch_kernel(count_tokens, dim3((unsigned)bs, y), kCountThreads, 0, stream, 0, true, p);
}
cudaError_t launch_count_reset(const CountParams &p, int n, cudaStream_t stream) {
    return launch_kernel(count_reset, dim3((unsigned)n), kCountThreads, 0, stream, 0, true, p);
}
cudaError_t launch_count_fork(const CountParams &p, const int32_t *parents, const int32_t *children, int n, cudaStream_t stream) {
    return launch_kernel(count_fork, dim3((unsigned)n), kCountThreads, 0, stream, 0, true, p, parents, children, n);
}

}  // namespace csgmv
