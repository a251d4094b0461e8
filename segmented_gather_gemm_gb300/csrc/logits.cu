// Logits of drafted tokens to what verification takes: penalties, biases,
// masks, temperature, softmax; and the counts of tokens that penalties go by.
// See include/csgmv.h (csgmv_process_logits, csgmv_count_*).
//
// A cluster of up to eight CTAs has a row, every eighth block of it a CTA (low
// numbers are frequent tokens: they are everyone's), that it copies to shared
// memory as it is, before it knows whose it is.  What is sparse is found
// while that arrives: the tokens that a sequence holds (they come as a list beside
// the dense counts, so a row costs as many gathers as it has tokens, not a pass
// over the vocabulary), the row's branch, biases.  Whoever finds a token first (a bit
// for each) takes its logit out of there, into a list, and leaves -infinity.  Two
// passes follow, both in shared memory: the maximum and the sum
// of exponentials together, then the probabilities; the list's counts come
// during the first.  The list is in no certain order, so its exponentials are summed in
// whole steps of 2^-40 of the CTA's largest: results do not depend on timing.
// The CTAs of a row exchange a pair of numbers a warp between the passes.
//
// Measured (device time): 768 bf16 rows of 128256 (64 drafted trees with counts,
// biases, a quarter of them with masks; 595 MB) 158 us; without any rule 108 us, 5.5
// TB/s; scores without softmax 93 us.  256 f32 rows of 100003 63 us, without rules 45 us.
// A row's chain of dependent loads and barriers (27600 clocks for a CTA, 14400 of them to ask
// for, find and score what is sparse) is hidden by the other CTAs of the SM: what holds
// it up is room for more of them.  Of 16 bits there are five up to 139000 tokens, four up
// to 184000, three up to 253000, then two.  Of f32 there are four where a row's share has
// at most 12800 elements (up to 12800, 25600, 51200 or 102400 tokens in 1, 2, 4 or 8
// CTAs), three of larger ones (16000, 32000, 65536, 128256), two from 139000, one from
// 213000 on: 4.9 TB/s of 128256, 3.9 of 151936, 3.1 of 262144.  A sequence that holds more
// tokens than the lists of a row's CTAs have room for costs passes over all bits: 2400
// bf16 rows of 32000 (two CTAs) with none 87 us, with 1000 127, 2000 185, 3000 348, 8000
// 1000; 600 of 128256 (eight) 91, 114, 135, 155 and 296.  (Also tried: scores in f32 shared memory, three CTAs an SM,
// 286 us; the row read again from L2 with a test for each vector, 210 us; the list
// in the order of the vocabulary by prefix sums, 172 us; 128 to 512 threads, 165 to
// 190 us; exponents in one fused operation, 180 us, or two at a time, 170 us; one
// atomic a warp for places in the list, 172 us.)
#include <algorithm>
#include <atomic>

#include "elements.cuh"
#include "serving.cuh"
#include "step.h"

namespace csgmv {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kPrompt = 1 << 30;
constexpr int kMaxVocab = 1 << 18, kMaxCtas = 8;
constexpr int kBlock = 512;  // elements; blocks of a row go to its CTAs in turn
// Scores in a CTA's list; further ones wait in out.  f32 has fewer, and room for a
// branch only where there is one: then four CTAs are on an SM for shares of up to 12800
// elements, with as many as 16 bits have for up to 11776 (256 rows of 100003, shares of
// 12800: 45 us, else 51).  What it costs: 2400 rows of 32000 with 2000 tokens held 406 us,
// bf16 185.
template <typename T>
constexpr int kKeptOf = sizeof(T) == 2 ? 1024 : 512;
constexpr float kLargest = 3.402823466e+38f;

// A part of a row: its largest score, and the sum of 2^((z - top) heat), which
// is NaN where a score is.  (temperature 0: the sum is 0 or NaN.)
struct Part {
    float top, sum;
    int at;  // temperature 0: the lowest place of top
};
template <typename T>
struct Smem {
    int branch[sizeof(T) == 2 ? 32 * kTreeMaxWords : 1];
    float kept[kKeptOf<T>];
    uint16_t place[kKeptOf<T>];
    int n_branch, n_kept;
    uint32_t drawn[32], biased[32];  // bits of the branch's and the biases' places modulo 1024
    float most[kWarps];
    unsigned long long steps;
    int list_at, lost;
    Part parts[kMaxCtas * (kWarps + 1)];  // of the row: each CTA's warps, and its list
};
// Shared memory of a CTA's blocks of a row: the elements, a bit for each, and (f32) the
// tokens of the row's branch.
struct Share {
    int elements, words, branch;  // bytes, words of bits, tokens
};
__host__ __device__ inline Share share_of(int chunk, int bytes, int mask_words) { return {chunk * bytes, chunk >> 5, bytes == 2 ? 0 : 32 * mask_words}; }

// 2^x to two units in the last place, what is below 2^-126 as 0.
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// What a sum about `top` counts about another (equal infinities are no difference).
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

template <typename T>
__global__ void __launch_bounds__(kThreads, sizeof(T) == 2 ? 5 : 4) process(LogitParams p) {
    extern __shared__ uint4 dynamic[];
    __shared__ Smem<T> sm;
    constexpr int kKept = kKeptOf<T>;
    constexpr int W = 16 / (int)sizeof(T);  // elements of a vector
    const Share shape = share_of(p.chunk, sizeof(T), p.mask_words);
    T *z = reinterpret_cast<T *>(dynamic);
    uint32_t *set = reinterpret_cast<uint32_t *>(reinterpret_cast<char *>(dynamic) + shape.elements);
    int *tokens = sizeof(T) == 2 ? sm.branch : reinterpret_cast<int *>(set + shape.words);  // of the branch
    griddep_launch_dependents();
    cluster_arrive();
    griddep_wait();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int ctas = (int)cluster_size(), rank = (int)cluster_rank();
    const int t = blockIdx.x / ctas;
    // This CTA's blocks of the row.  Blocks are counted from the 16-byte boundary at or
    // before it; z[i] is the logit of token(i), which is outside the vocabulary before
    // the row's first element and behind its last one.
    const T *row = static_cast<const T *>(p.logits) + t * p.logits_s;
    const int begin = (int)(reinterpret_cast<uintptr_t>(row) % 16 / sizeof(T)), turns = 31 - __clz(ctas);
    const int blocks = (begin + p.vocab + kBlock - 1) / kBlock, n = rank < blocks ? ((blocks - 1 - rank) >> turns) * kBlock + kBlock : 0;
    auto token = [&](unsigned i) { return (int)((((i / kBlock) << turns) + rank) * kBlock + i % kBlock) - begin; };
    auto inside = [&](int token) { return (unsigned)token < (unsigned)p.vocab; };
    const float none = __int_as_float(0xff800000);
    const int v_first = token(tid * W), v_step = (kThreads * W) << turns;  // tokens of a thread's vectors
    static_assert(kThreads * W % kBlock == 0, "a thread's vectors have one place in their blocks");
    auto whole = [&](int v) { return (unsigned)v <= (unsigned)(p.vocab - W) && p.vocab >= W; };
    for (int i = tid * W, v = v_first; i < n; i += kThreads * W, v += v_step) {
        if (whole(v)) cp_async16(z + i, row + v, 16);
        else
            for (int e = 0; e < W; ++e) z[i + e] = inside(v + e) ? row[v + e] : from_f32<T>(none);
    }
    // (a word of the row's mask a lane: eight at most)
    const uint32_t mask_word = warp == 0 && p.mask && lane < p.mask_words ? (uint32_t)p.mask[(int64_t)t * p.mask_words + lane] : 0;
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
    float *out = p.out + t * p.out_s;
    // where a token is in z if it is this CTA's to put right, or -1
    auto place = [&](int token) {
        const unsigned j = token + begin, block = j / kBlock;
        return inside(token) && (int)(block & (ctas - 1)) == rank && (!allow || has(allow, token)) ? (int)((block >> turns) * kBlock + j % kBlock) : -1;
    };
    const bool punish = rho != 1.0f || alpha != 0.0f || beta != 0.0f, branch = punish && p.mask;
    const int32_t *counts = punish && p.counts ? p.counts + (int64_t)seq * p.vocab : nullptr;
    const int32_t *seen = counts ? p.seen + (int64_t)seq * p.vocab : nullptr;
    const int held = counts ? min(p.num_seen[seq], p.vocab) : 0;
    const bool sparse = held > 0 || branch || b1 > b0;
    if (tid == 0) sm.n_kept = 0, sm.steps = 0, sm.list_at = INT32_MAX, sm.lost = 0;
    if (warp == 0) sm.drawn[lane] = sm.biased[lane] = 0;
    // the first tokens that the sequence holds, where they are, and their counts on the way
    constexpr int S = 4;
    int held_at[S];
    auto load_held = [&](int i0) {
#pragma unroll
        for (int u = 0; u < S; ++u) held_at[u] = i0 + tid + u * kThreads < held ? seen[i0 + tid + u * kThreads] : -1;
#pragma unroll
        for (int u = 0; u < S; ++u) held_at[u] = place(held_at[u]);
    };
    // the last warp has the first biases, the first one the branch: loads before all that waits
    const int bias_i = b0 + (tid ^ (kThreads - 32));
    int bias_v = 0, bias_before = 0;
    if (bias_i < b1) {
        bias_v = p.bias_tokens[bias_i];
        bias_before = bias_i > b0 ? p.bias_tokens[bias_i - 1] : bias_v;
        prefetch(p.bias_values + bias_i);
    }
    if (branch && warp == 0) {
        int k = 0;
        for (int w = 0; w < p.mask_words; ++w) {
            const uint32_t bits = __shfl_sync(kFullMask, mask_word, w);
            const int j = 32 * w + lane;
            int v = -1;
            if ((bits >> lane & 1u) && j < last - first) {
                v = p.drafts[first + j];
                if (!inside(v)) {
                    if (rank == 0) atomicOr(p.status, CSGMV_KV_STATUS_BAD_TOKEN);
                    v = -1;
                }
            }
            const unsigned m = __ballot_sync(kFullMask, v >= 0);
            if (v >= 0) tokens[k + __popc(m & ((1u << lane) - 1u))] = v;
            k += __popc(m);
        }
        if (lane == 0) sm.n_branch = k;
    }
    load_held(0);
#pragma unroll
    for (int u = 0; u < S; ++u)
        if (held_at[u] >= 0) prefetch(counts + token(held_at[u]));
    if (allow && tid * kBlock < n) prefetch(allow + (max(token(tid * kBlock), 0) >> 5));
    if (sparse)
        for (int i = tid; i < shape.words; i += kThreads) set[i] = 0;
    bool torn = bias_v < bias_before;
    for (int i = bias_i + kThreads; i < b1; i += kThreads) torn |= p.bias_tokens[i] < p.bias_tokens[i - 1];
    cp_async_wait_all();
    if (__syncthreads_or(torn)) {  // biases out of order; every CTA of the cluster alike
        if (rank == 0 && tid == 0) atomicOr(p.status, CSGMV_KV_STATUS_BAD_VALUE);
        return;
    }
    if (allow) {  // what is not allowed, out of there
#pragma unroll 4
        for (int i = tid * W, v0 = v_first; i < n; i += kThreads * W, v0 += v_step) {
            const int from = min(max(v0, 0), p.vocab - 1);  // (the vector may begin before the row)
            uint32_t bits = allow[from >> 5] >> (from & 31);
            if ((from & 31) + W > 32 && (from | 31) + 1 < p.vocab) bits |= allow[(from >> 5) + 1] << (32 - (from & 31));
            bits <<= max(from - v0, 0);
            Vec<T, W> v = *reinterpret_cast<const Vec<T, W> *>(z + i);
#pragma unroll
            for (int e = 0; e < W; ++e) v.e[e] = bits >> e & 1u ? v.e[e] : from_f32<T>(none);
            *reinterpret_cast<Vec<T, W> *>(z + i) = v;
        }
    }
    int done = 0;  // tokens in the list, and behind it
    if (sparse) {
        if (allow) __syncthreads();
        auto take = [&](int at) {
            const uint32_t bit = 1u << (at & 31);
            if (atomicOr(set + (at >> 5), bit) & bit) return;
            const int r = atomicAdd(&sm.n_kept, 1);
            if (r < kKept) sm.kept[r] = to_f32(z[at]), sm.place[r] = (uint16_t)at;
            else out[token(at)] = to_f32(z[at]);
            z[at] = from_f32<T>(none);
        };
        const int k = branch ? sm.n_branch : 0;
        for (int i = tid; i < k; i += kThreads)
            if (const int at = place(tokens[i]); at >= 0) {
                atomicOr(&sm.drawn[at >> 5 & 31], 1u << (at & 31));
                take(at);
            }
        for (int i = bias_i; i < b1; i += kThreads) {
            if (i > bias_i) bias_v = p.bias_tokens[i];
            if (!inside(bias_v)) {
                if (rank == 0) atomicOr(p.status, CSGMV_KV_STATUS_BAD_TOKEN);
            } else if (const int at = place(bias_v); at >= 0) {
                atomicOr(&sm.biased[at >> 5 & 31], 1u << (at & 31));
                take(at);
            }
        }
        for (int i0 = 0; i0 < held; i0 += S * kThreads) {
            if (i0 > 0) load_held(i0);
#pragma unroll
            for (int u = 0; u < S; ++u)
                if (held_at[u] >= 0) take(held_at[u]);
        }
        __syncthreads();
        done = sm.n_kept;
        if (done > kKept) {  // bits of those that the list has no room for are left
            for (int r = tid; r < kKept; r += kThreads) atomicAnd(set + (sm.place[r] >> 5), ~(1u << (sm.place[r] & 31)));
            __syncthreads();
        }
    } else if (allow) {
        __syncthreads();
    }
    // f(score, place) for each of the list, and behind it
    auto each = [&](auto f) {
        for (int r = tid; r < min(done, kKept); r += kThreads) f(sm.kept[r], (int)sm.place[r]);
        if (done > kKept)
            for (int w = tid; w < shape.words; w += kThreads)
                for (uint32_t bits = set[w]; bits; bits &= bits - 1) f(out[token(32 * w + __ffs(bits) - 1)], 32 * w + __ffs(bits) - 1);
    };
    auto score = [&](float &x, int at, int word) {
        const int v = token(at);
        float y = x;
        if (punish) {
            int more = 0;
            if (branch && (sm.drawn[at >> 5 & 31] >> (at & 31) & 1u)) {
                const int k = sm.n_branch;
                for (int j = 0; j < k; ++j) more += tokens[j] == v;
            }
            y = penalized(y, word, more, rho, alpha, beta);
        }
        if (b1 > b0 && (sm.biased[at >> 5 & 31] >> (at & 31) & 1u)) {
            int i = b0;  // the first bias of the token
            for (int len = b1 - b0; len > 0;) {
                const int half = len >> 1;
                if (p.bias_tokens[i + half] < v) i += half + 1, len -= half + 1;
                else len = half;
            }
            for (; i < b1 && p.bias_tokens[i] == v; ++i) y = __fadd_rn(y, p.bias_values[i]);
        }
        x = y;
    };
    // the counts of the list, on the way during the first pass
    constexpr int C = (kKept + kThreads - 1) / kThreads;
    int word[C];
#pragma unroll
    for (int u = 0; u < C; ++u) word[u] = counts && tid + u * kThreads < min(done, kKept) ? counts[token(sm.place[tid + u * kThreads])] : 0;
    auto score_all = [&]() {
#pragma unroll
        for (int u = 0; u < C; ++u)
            if (const int r = tid + u * kThreads; r < min(done, kKept)) score(sm.kept[r], sm.place[r], word[u]);
        if (done > kKept)
            for (int w = tid; w < shape.words; w += kThreads)
                for (uint32_t bits = set[w]; bits; bits &= bits - 1) {
                    const int at = 32 * w + __ffs(bits) - 1;
                    score(out[token(at)], at, counts ? counts[token(at)] : 0);
                }
    };
    auto vector = [&](int i, float (&x)[W]) {
        widen(*reinterpret_cast<const Vec<T, W> *>(z + i), x);
    };
    // out = f(score, token), in vectors where those of out are where those of z are
    // and no score waits in out
    const bool wide = reinterpret_cast<uintptr_t>(out - begin) % (4 * W) == 0 && done <= kKept;
    auto write = [&](auto f) {
        if (wide) {
            for (int i = tid * W, v = v_first; i < n; i += kThreads * W, v += v_step) {
                float x[W];
                vector(i, x);
#pragma unroll
                for (int e = 0; e < W; ++e) x[e] = f(x[e], v + e);
                if (whole(v)) store<W>(out + v, x);
                else
#pragma unroll
                    for (int e = 0; e < W; ++e)
                        if (inside(v + e)) out[v + e] = x[e];
            }
        } else {
#pragma unroll 4
            for (int i = tid; i < n; i += kThreads)
                if (const int v = token(i); inside(v) && (done <= kKept || !has(set, i))) out[v] = f(to_f32(z[i]), v);
        }
        if (done > 0) {
            __syncthreads();
            each([&](float &x, int at) { out[token(at)] = f(x, token(at)); });
        }
    };
    if (!p.softmax) {
        score_all();
        write([](float x, int) { return x; });
        return;
    }
    // exp((z - top) / temperature) = 2^((z - top) heat)
    const bool greedy = temperature == 0.0f;
    const float heat = greedy ? 1.0f : fminf(1.4426950408889634f / temperature, kLargest);
    Part part = {none, 0.0f, INT32_MAX};
    if (greedy) {
        for (int i = tid * W, v = v_first; i < n; i += kThreads * W, v += v_step) {
            float x[W];
            vector(i, x);
#pragma unroll
            for (int e = 0; e < W; ++e) {
                if (x[e] > part.top) part.top = x[e], part.at = v + e;
                if (x[e] != x[e]) part.sum = x[e];
            }
        }
    } else {
        for (int i = tid * W; i < n; i += kThreads * W) {
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
    }
    // Each warp's part, and the list's, to every CTA of the cluster.
    auto tell = [&](const Part &x, int slot) {
        if (lane >= ctas) return;
        const uint32_t to = dsmem_addr(&sm.parts[rank * (kWarps + 1) + slot], lane);
        dsmem_st_f32(to, x.top);
        dsmem_st_f32(to + 4, x.sum);
        dsmem_st_f32(to + 8, __int_as_float(x.at));
    };
    part = warp_join(part, greedy, heat);
    cluster_wait();  // (all have begun)
    tell(part, warp);
    // The list's part: by the first warp alone where it has them all, without barriers.
    Part list = {none, 0.0f, INT32_MAX};
    const bool many = done > 32;
    if (many || (done > 0 && warp == 0)) {
        score_all();
        float most = none;
        each([&](float &x, int) { most = fmaxf(most, x); });
        most = warp_max(most);
        if (many) {
            if (lane == 0) sm.most[warp] = most;
            __syncthreads();
            most = warp_max(lane < kWarps ? sm.most[lane] : none);
        }
        list.top = most;
        const float about = most == none ? 0.0f : most;
        unsigned long long steps = 0;
        int lost = 0;
        each([&](float &x, int at) {
            if (greedy) {
                if (x == most) list.at = min(list.at, token(at));
                lost |= x != x;
            } else {
                const float y = ex2((x - about) * heat);
                if (y > 0.0f) steps += (unsigned long long)(y * 0x1p40f);
                lost |= y != y;
            }
        });
        // (whole numbers: in any order)
        steps = warp_sum(steps);
        list.at = __reduce_min_sync(kFullMask, list.at);
        lost = __any_sync(kFullMask, lost);
        if (many) {
            if (lane == 0) {
                atomicAdd(&sm.steps, steps), atomicMin(&sm.list_at, list.at);
                if (lost) sm.lost = 1;
            }
            __syncthreads();
            steps = sm.steps, list.at = sm.list_at, lost = sm.lost;
        }
        list.sum = lost ? __int_as_float(0x7fc00000) : (float)steps * 0x1p-40f;
    }
    if (warp == 0) tell(list, kWarps);
    cluster_sync();
    // (up to 72 parts, three a lane)
    Part row_part = {none, 0.0f, INT32_MAX};
#pragma unroll
    for (int u = 0; u < 3; ++u) {
        const int i = lane + 32 * u;
        if (i >= ctas * (kWarps + 1)) break;
        const Part x = sm.parts[i];
        const float most = fmaxf(row_part.top, x.top);
        if (x.top == most) row_part.at = row_part.top == most ? min(row_part.at, x.at) : x.at;
        row_part.sum = shifted(row_part.sum, row_part.top, most, heat) + shifted(x.sum, x.top, most, heat);
        row_part.top = most;
    }
    row_part = warp_join(row_part, greedy, heat);
    const float top = row_part.top, sum = row_part.sum;
    // a sum that is NaN makes all of the row that; nothing but -infinity makes it 0
    const float share = sum != sum ? sum : top == none ? 0.0f : greedy ? 1.0f : __fdiv_rn(1.0f, sum);
    if (greedy) {
        write([&](float, int v) { return (v == row_part.at ? 1.0f : 0.0f) * share; });
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

// Elements of the largest share of a row among ctas CTAs, wherever it begins.
int chunk_of(int vocab, int ctas, int bytes) {
    const int blocks = (16 / bytes - 1 + vocab + kBlock - 1) / kBlock;
    return (blocks + ctas - 1) / ctas * kBlock;
}
size_t smem_of(int chunk, int bytes, int mask_words) {
    const Share s = share_of(chunk, bytes, mask_words);
    return (size_t)s.elements + 4 * (size_t)s.words + 4 * (size_t)s.branch;
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
        if ((e = cudaFuncSetAttribute(f.fn, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem_of(chunk_of(kMaxVocab, kMaxCtas, f.bytes), f.bytes, kTreeMaxWords))) !=
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
    // CTAs of a row: shares of about 16384 elements (32768 where those would be more than
    // eight), and more of them while there are not enough rows for the SMs.
    int ctas = 1;
    while (ctas < kMaxCtas && ((int64_t)p.vocab > (int64_t)ctas * 16384 || (p.num_tokens * ctas * 2 <= 152 && p.vocab > ctas * 2048)))
        ctas *= 2;
    p.chunk = chunk_of(p.vocab, ctas, (int)sizeof(T));
    return launch_kernel(process<T>, dim3((unsigned)(p.num_tokens * ctas)), kThreads, smem_of(p.chunk, sizeof(T), p.mask_words), stream, ctas, true, p);
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
