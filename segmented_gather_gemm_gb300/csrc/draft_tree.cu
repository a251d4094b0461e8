// Draft trees: derived fields (masks, depths, child lists) and the
// verification walk.  See include/csgmv.h for the definitions.
#include "serving.cuh"

namespace csgmv {
namespace {

constexpr int kMaxNodes = 32 * kTreeMaxWords;  // nodes of one request

// ------------------------------------------------------------------ building
constexpr int kTreeThreads = 64;

// A block a request.  A node walks up its ancestors and sets a bit for each,
// in shared memory; siblings are found by scanning forward.  A request is a
// few dozen nodes, so the whole call is a launch and a few shared-memory
// latencies.
__global__ void __launch_bounds__(kTreeThreads) build_tree(TreeParams p) {
    __shared__ int par[kMaxNodes];
    __shared__ uint32_t bits[kMaxNodes * kTreeMaxWords];
    __shared__ int bad_s;
    griddep_launch_dependents();
    const int b = blockIdx.x, tid = threadIdx.x;
    const int lo = p.indptr[b], hi = p.indptr[b + 1];
    if (lo < 0 || hi < lo || hi > p.num_nodes) {
        if (tid == 0) atomicOr(p.status, CSGMV_KV_STATUS_BAD_TREE);
        return;
    }
    const int n = hi - lo;
    if (tid == 0) bad_s = n > 32 * p.words;
    __syncthreads();
    if (!bad_s) {
        bool wrong = false;
        for (int i = tid; i < n; i += kTreeThreads) {
            const int q = p.parents[lo + i];
            par[i] = q;
            wrong |= i == 0 ? q != -1 : q < 0 || q >= i;
        }
        if (wrong) bad_s = 1;
    }
    for (int i = tid; i < kMaxNodes * kTreeMaxWords; i += kTreeThreads) bits[i] = 0;
    __syncthreads();
    const bool bad = bad_s;
    if (bad && tid == 0) atomicOr(p.status, CSGMV_KV_STATUS_BAD_TREE);
    for (int i = tid; i < n; i += kTreeThreads) {
        int depth = 0, child = -1, next = -1;
        if (!bad) {
            uint32_t *row = bits + i * kTreeMaxWords;
            for (int k = i; k >= 0; k = par[k]) {
                row[k >> 5] |= 1u << (k & 31);
                ++depth;
            }
            --depth;
            for (int k = i + 1; k < n && (child < 0 || next < 0); ++k) {
                if (child < 0 && par[k] == i) child = k;
                if (next < 0 && i > 0 && par[k] == par[i]) next = k;
            }
        }
        for (int w = 0; w < p.words; ++w)
            p.mask[(int64_t)(lo + i) * p.words + w] = bad ? 0 : (int32_t)bits[i * kTreeMaxWords + w];
        p.depth[lo + i] = depth;
        p.first_child[lo + i] = child;
        p.next_sibling[lo + i] = next;
    }
}

// -------------------------------------------------------------- verification
constexpr int kVerMaxCtas = 8;    // CTAs of the cluster that walks one tree, at most
constexpr int kVerThreads = 512;
constexpr int kVerWarps = kVerThreads / 32;

// Probabilities count in steps of 2^-44.
__device__ __forceinline__ long long fixed44(float x) {
    return __float2ll_rz(fminf(fmaxf(x, 0.0f), 1.0f) * 17592186044416.0f);
}
// The same steps as a high and a low number of 22 bits each, whose sums over a
// thread's tokens fit 32 bits.  A float in [2, 4) counts steps of 2^-22 in its
// lower bits, so adding 2 towards zero leaves the high number there, and what
// that leaves out, exact, times 2^22 plus 2 the low one: no conversions (with
// three a number, 64 sampled trees over 128256 tokens took 37.6 us, now 36.2).
// The bits of the 2 itself cancel when a multiple of four are added.
struct Steps {
    uint32_t hi, lo;
    __device__ __forceinline__ void add(float x) {
        const float a = fminf(fmaxf(x, 0.0f), 1.0f), t = __fadd_rz(a, 2.0f);
        hi += __float_as_uint(t);
        lo += __float_as_uint(__fmaf_rz(__fsub_rn(a, __fsub_rn(t, 2.0f)), 4194304.0f, 2.0f));
    }
    __device__ __forceinline__ long long total() const { return ((long long)hi << 22) + lo; }
};
// One refusal: r = max(r - z q, 0), each operation rounded.
__device__ __forceinline__ float refuse(float r, float z, float q) {
    return fmaxf(__fsub_rn(r, __fmul_rn(z, q)), 0.0f);
}

struct VerSmem {
    int first[kMaxNodes], next[kMaxNodes], parent[kMaxNodes], token[kMaxNodes];
    float u[kMaxNodes], p[kMaxNodes], q[kMaxNodes], z[kMaxNodes];
    long long warp[kVerWarps], chunk[kVerWarps], total;
    int gone[kMaxNodes], ngone;  // children's distinct tokens in this CTA's part, taken out
};

// A cluster a request; CTA `rank` owns tokens [rank * per, (rank + 1) * per)
// of the vocabulary, a warp a contiguous stretch of them.  Every CTA walks the
// tree by itself from the drafted tokens' own probabilities, gathered at the
// start in one round of loads, so an accepted draft costs no pass over a
// distribution.  Rows are read where the sum of what is left matters: after a
// refusal with another sibling to try, and for the last token.  What is left
// is a function of the row, the draft's row and the z of each refusal, so it
// is worked out again where it is needed and nothing is kept.  Sums are whole
// numbers, so the reductions' order does not show.
//
// What bounds a batch is the rows' bytes, so there have to be enough loads in
// flight: a thread keeps four 16-byte loads (eight spill: 64 sampled trees 52 us
// instead of 36), and a cluster is as large as leaves the batch two CTAs an SM
// (launch_verify; four an SM, in turns: 41 us).  256 trees over 128256 tokens,
// one pass each: 37 us, the pass 22 us of it at 6 TB/s; one chain of 5 over
// 32000: 9.5 us.  In both the rest is dependent loads: lists, parents, the drafted
// tokens' probabilities, the draw.
__global__ void __launch_bounds__(kVerThreads, 2) verify(VerifyParams v, int per, int vec) {
    __shared__ VerSmem sm;
    const int ctas = (int)cluster_size();
    griddep_wait();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, rank = (int)cluster_rank();
    const int b = blockIdx.x / ctas;
    const int lo = v.indptr[b], hi = v.indptr[b + 1];
    const int V = v.vocab;
    int n = hi - lo;
    if (tid == 0) sm.ngone = 0;
    const bool sound = lo >= 0 && hi >= lo && hi <= v.num_nodes && n <= kMaxNodes;
    auto leave_out = [&](bool bad) {
        if (rank != 0) return;
        for (int j = tid; j < v.width; j += kVerThreads) v.accept_index[(int64_t)b * v.width + j] = -1;
        if (tid == 0) {
            v.accept_len[b] = 0;
            v.next_token[b] = -1;
            if (bad) atomicOr(v.status, CSGMV_KV_STATUS_BAD_TREE);
        }
    };
    if (!sound || n == 0) return leave_out(!sound);  // the same in every CTA of the cluster
    for (int i = tid; i < n; i += kVerThreads) {
        // numbers that do not increase would let the walk go in circles
        const int f = v.first_child[lo + i], s = v.next_sibling[lo + i];
        sm.first[i] = f > i && f < n ? f : -1;
        sm.next[i] = s > i && s < n ? s : -1;
        sm.u[i] = v.accept_u[lo + i];
        int t = v.tokens[lo + i];
        if (i > 0 && (t < 0 || t >= V)) {
            if (rank == 0) atomicOr(v.status, CSGMV_KV_STATUS_BAD_TOKEN);
            t = -1;
        }
        sm.token[i] = t;
        sm.parent[i] = -1;
    }
    __syncthreads();
    // (A node in two lists would have whichever parent comes last, not the same one in every CTA, and
    // CTAs that walk differently would wait for one another at the cluster's barriers.)
    bool twice = false;
    for (int i = tid; i < n; i += kVerThreads)
        for (int k = sm.first[i]; k >= 0; k = sm.next[k]) twice |= atomicExch(&sm.parent[k], i) >= 0;
    if (__syncthreads_or(twice)) return leave_out(true);
    for (int i = tid; i < n; i += kVerThreads) {
        const int c = sm.parent[i], t = sm.token[i];
        const bool on = c >= 0 && t >= 0;
        sm.p[i] = on ? v.target[(int64_t)(lo + c) * v.target_stride + t] : 0.0f;
        sm.q[i] = on && v.draft ? v.draft[(int64_t)(lo + c) * v.draft_stride + t] : 0.0f;
    }
    __syncthreads();

    const int v0 = min(V, rank * per), v1 = min(V, v0 + per);
    const int perw = ((per + kVerWarps - 1) / kVerWarps + 127) & ~127;
    const int w0 = min(v1, v0 + warp * perw), w1 = min(v1, w0 + perw);
    // Four tokens from i on (0 from `end` on); 16 bytes at once where the rows allow it.
    auto load4 = [&](const float *row, int i, int end) {
        if (vec && i + 4 <= end) return __ldg(reinterpret_cast<const float4 *>(row + i));
        float4 x = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        if (i < end) x.x = __ldg(row + i);
        if (i + 1 < end) x.y = __ldg(row + i + 1);
        if (i + 2 < end) x.z = __ldg(row + i + 2);
        if (i + 3 < end) x.w = __ldg(row + i + 3);
        return x;
    };
    // What is left of them after n refusals.
    auto left4 = [&](float4 x, float4 y, int n) {
#pragma unroll 1
        for (int m = 0; m < n; ++m) {
            const float z = sm.z[m];
            x = make_float4(refuse(x.x, z, y.x), refuse(x.y, z, y.y), refuse(x.z, z, y.z), refuse(x.w, z, y.w));
        }
        return x;
    };
    // The sum over the vocabulary of what is left of a row after n refusals.
    // sm.total: the CTA's part, sm.warp: the running sum ahead of each warp.
    auto pass = [&](const float *p, const float *q, int n) -> long long {
        Steps s = {0, 0};
        constexpr int kFar = 4;  // stretches of 128 tokens in flight
        for (int i0 = w0 + lane * 4; i0 - lane * 4 < w1; i0 += kFar * 128) {
            float4 x[kFar], y[kFar];
#pragma unroll
            for (int u = 0; u < kFar; ++u) {
                x[u] = load4(p, i0 + u * 128, w1);
                y[u] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                if (n) y[u] = load4(q, i0 + u * 128, w1);
            }
#pragma unroll
            for (int u = 0; u < kFar; ++u) {
                const float4 r = left4(x[u], y[u], n);
                s.add(r.x);
                s.add(r.y);
                s.add(r.z);
                s.add(r.w);
            }
        }
        long long t = warp_sum(s.total());
        for (int c = 0; c < sm.ngone; ++c) {
            const int i = sm.gone[c];
            if (i >= w0 && i < w1) t -= fixed44(__ldg(p + i));
        }
        if (lane == 0) sm.warp[warp] = t;
        __syncthreads();
        if (warp == 0) {
            const long long w = lane < kVerWarps ? sm.warp[lane] : 0, inc = warp_scan(w);
            if (lane < kVerWarps) sm.warp[lane] = inc - w;
            if (lane == 31) sm.total = inc;
        }
        __syncthreads();
        cluster_sync();
        const long long c = lane < ctas ? dsmem_ld_i64(dsmem_addr(&sm.total, lane)) : 0;
        return warp_sum(c);
    };
    // The walk, the same in every thread of the cluster.
    int cur = 0, count = 1;
    int32_t *path = v.accept_index + (int64_t)b * v.width;
    if (rank == 0 && tid == 0) path[0] = 0;
    int refused = 0;
    long long total = 0;
    while (true) {
        const float *p = v.target + (int64_t)(lo + cur) * v.target_stride;
        const float *q = v.draft ? v.draft + (int64_t)(lo + cur) * v.draft_stride : nullptr;
        int hit = -1;
        refused = 0;
        if (q) {
            float z = 1.0f;
            for (int k = sm.first[cur]; k >= 0 && z > 0.0f; k = sm.next[k]) {
                if (sm.token[k] < 0) continue;
                float rk = sm.p[k];
                for (int m = 0; m < refused; ++m) rk = refuse(rk, sm.z[m], sm.q[k]);
                if (__fmul_rn(__fmul_rn(sm.u[k], sm.q[k]), z) < rk) {
                    hit = k;
                    break;
                }
                // (sm.z[0] is always 1, and a later one is written behind a pass's barriers, so
                // no thread still reads the node before's)
                if (tid == 0) sm.z[refused] = z;
                ++refused;
                __syncthreads();
                total = pass(p, q, refused);
                cluster_sync();  // the other CTAs have read sm.total
                z = __fmul_rn(__ll2float_rn(total), 1.0f / 17592186044416.0f);
            }
        } else {
            long long mass = 0;
            const long long coin = (long long)(fminf(fmaxf(sm.u[cur], 0.0f), 1.0f) * 17592186044416.0f);
            for (int k = sm.first[cur]; k >= 0; k = sm.next[k]) {
                bool seen = sm.token[k] < 0;
                for (int e = sm.first[cur]; e != k; e = sm.next[e]) seen |= sm.token[e] == sm.token[k];
                if (seen) continue;
                mass += fixed44(sm.p[k]);
                if (coin < mass) {
                    hit = k;
                    break;
                }
            }
        }
        if (hit < 0) {
            if (refused == 0) {
                if (!q) {
                    if (tid == 0) {
                        int n = 0;
                        for (int k = sm.first[cur]; k >= 0; k = sm.next[k]) {
                            const int t = sm.token[k];
                            bool seen = t < v0 || t >= v1;
                            for (int e = 0; e < n; ++e) seen |= sm.gone[e] == t;
                            if (!seen) sm.gone[n++] = t;
                        }
                        sm.ngone = n;
                    }
                    __syncthreads();
                }
                total = pass(p, q, 0);
            }
            if (total == 0) {  // nothing is left: the distribution itself
                cluster_sync();
                if (tid == 0) sm.ngone = 0;
                __syncthreads();
                refused = 0;
                total = pass(p, q, 0);
            }
            break;
        }
        cur = hit;
        if (rank == 0 && tid == 0 && count < v.width) path[count] = cur;
        ++count;
    }
    const bool fits = count <= v.width;
    if (rank == 0) {
        if (fits) {
            for (int j = count + tid; j < v.width; j += kVerThreads) path[j] = -1;
        } else {
            __syncthreads();
            for (int j = tid; j < v.width; j += kVerThreads) path[j] = -1;
        }
        if (tid == 0) {
            v.accept_len[b] = fits ? count : 0;
            if (!fits) atomicOr(v.status, CSGMV_KV_STATUS_CAPACITY);
            if (fits && total == 0) atomicOr(v.status, CSGMV_KV_STATUS_BAD_TOKEN);
            if (!fits || total == 0) v.next_token[b] = -1;
        }
    }
    // The draw: the CTA, the warp and then the token whose running sum is the
    // first above aim.
    const long long U = (long long)(fminf(fmaxf(v.sample_u[b], 0.0f), 0.99999994f) * 2147483648.0f);
    const long long aim = U * (total >> 31) + ((U * (total & 0x7fffffffll)) >> 31);
    const long long t = lane < ctas ? dsmem_ld_i64(dsmem_addr(&sm.total, lane)) : 0;
    const long long before = warp_sum(lane < rank ? t : 0ll);
    const long long mine = __shfl_sync(kFullMask, t, rank);
    cluster_sync();  // no CTA leaves while another reads its shared memory
    if (!fits || total == 0 || aim < before || aim >= before + mine) return;
    // its warp's stretch, dealt out to all threads of the CTA
    int owner = 0;
    for (int w = 1; w < kVerWarps; ++w)
        if (before + sm.warp[w] <= aim) owner = w;  // the last: the warps after it that hold nothing start beyond aim
    const long long ahead = before + sm.warp[owner];
    const int o0 = min(v1, v0 + owner * perw), o1 = min(v1, o0 + perw);
    const int each = ((o1 - o0 + kVerThreads - 1) / kVerThreads + 3) & ~3;
    const int s0 = min(o1, o0 + tid * each), s1 = min(o1, s0 + each);
    const float *p = v.target + (int64_t)(lo + cur) * v.target_stride;
    const float *q = v.draft ? v.draft + (int64_t)(lo + cur) * v.draft_stride : nullptr;
    // What is left of the kDraw * 4 tokens from i on, all loads in flight at once.
    constexpr int kDraw = 2;  // (4: 0.3 to 0.7 us slower, more code that runs once)
    auto left = [&](int i, float4 (&r)[kDraw]) {
        float4 y[kDraw];
#pragma unroll
        for (int u = 0; u < kDraw; ++u) {
            r[u] = load4(p, i + 4 * u, s1);
            y[u] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            if (refused) y[u] = load4(q, i + 4 * u, s1);
        }
#pragma unroll
        for (int u = 0; u < kDraw; ++u) r[u] = left4(r[u], y[u], refused);
    };
    float4 r[kDraw];
    Steps part = {0, 0};
    for (int i = s0; i < s1; i += 4 * kDraw) {
        left(i, r);
#pragma unroll
        for (int u = 0; u < kDraw; ++u) {
            part.add(r[u].x);
            part.add(r[u].y);
            part.add(r[u].z);
            part.add(r[u].w);
        }
    }
    long long sum = part.total();
    for (int c = 0; c < sm.ngone; ++c)
        if (sm.gone[c] >= s0 && sm.gone[c] < s1) sum -= fixed44(__ldg(p + sm.gone[c]));
    long long inc = warp_scan(sum);
    if (lane == 31) sm.chunk[warp] = inc;
    __syncthreads();
    inc += ahead;
    for (int w = 0; w < warp; ++w) inc += sm.chunk[w];
    if (aim < inc - sum || aim >= inc) return;
    long long run = inc - sum;
#pragma unroll 1
    for (int i = s0; i < s1; i += 4) {  // one thread's; the loads again, from L1
        float4 x = load4(p, i, s1);
        if (refused) x = left4(x, load4(q, i, s1), refused);
        long long n[4] = {fixed44(x.x), fixed44(x.y), fixed44(x.z), fixed44(x.w)};
        for (int c = 0; c < sm.ngone; ++c) {
            const int at = sm.gone[c] - i;
#pragma unroll
            for (int k = 0; k < 4; ++k) n[k] = at == k ? 0 : n[k];
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            if (aim >= run && aim < run + n[k]) v.next_token[b] = i + k;
            run += n[k];
        }
    }
}

}  // namespace

cudaError_t launch_build_tree(const TreeParams &p, cudaStream_t stream) {
    return launch_kernel(build_tree, dim3((unsigned)p.bs), kTreeThreads, 0, stream, 0, false, p);
}

cudaError_t launch_verify(const VerifyParams &p, cudaStream_t stream) {
    // CTAs a request: as many as leave the batch at most two an SM (all at once), fewer
    // where a part of the vocabulary would be under 2048 tokens
    int ctas = kVerMaxCtas;
    while (ctas > 1 && ((int64_t)p.bs * ctas > 2 * 152 || p.vocab < 2048 * ctas)) ctas /= 2;
    const int per = ((p.vocab + ctas - 1) / ctas + 127) & ~127;
    auto rows16 = [](const float *q, int64_t stride) { return (reinterpret_cast<uintptr_t>(q) & 15) == 0 && stride % 4 == 0; };
    const int vec = rows16(p.target, p.target_stride) && (!p.draft || rows16(p.draft, p.draft_stride));
    return launch_kernel(verify, dim3((unsigned)(p.bs * ctas)), kVerThreads, 0, stream, ctas, true, p, per, vec);
}

}  // namespace csgmv
