// Draft trees: derived fields (masks, depths, child lists) and the
// verification walk.  See include/csgmv.h for the definitions.
#include <mutex>
#include <set>
#include <type_traits>

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
constexpr int kVerCtas = 8;       // CTAs of the cluster that walks one tree
constexpr int kVerThreads = 512;
constexpr int kVerWarps = kVerThreads / 32;

// Probabilities count in steps of 2^-44.
__device__ __forceinline__ long long fixed44(float x) {
    return __float2ll_rz(fminf(fmaxf(x, 0.0f), 1.0f) * 17592186044416.0f);
}
// The same steps as a high and a low number of 22 bits each: both products and
// the difference are exact, and sums over a thread's tokens fit 32 bits.
struct Steps {
    uint32_t hi, lo;
    __device__ __forceinline__ void add(float x) {
        const float a = fminf(fmaxf(x, 0.0f), 1.0f) * 4194304.0f;
        const uint32_t h = __float2uint_rz(a);
        hi += h;
        lo += __float2uint_rz((a - __uint2float_rn(h)) * 4194304.0f);
    }
    __device__ __forceinline__ long long total() const { return ((long long)hi << 22) + lo; }
};
// One refusal: r = max(r - z q, 0), each operation rounded.
__device__ __forceinline__ float refuse(float r, float z, float q) {
    return fmaxf(__fsub_rn(r, __fmul_rn(z, q)), 0.0f);
}

enum { kRowPlain = 0, kRowRefuse = 1, kRowAgain = 2 };

struct VerSmem {
    int first[kMaxNodes], next[kMaxNodes], parent[kMaxNodes], token[kMaxNodes];
    float u[kMaxNodes], p[kMaxNodes], q[kMaxNodes], z[kMaxNodes];
    long long warp[kVerWarps], total;
    int mine[kMaxNodes], nmine;  // children's tokens in this CTA's part
};

// A cluster a request; CTA `rank` owns tokens [rank * per, (rank + 1) * per)
// of the vocabulary, a warp a contiguous stretch of them.  Every CTA walks the
// tree by itself from the drafted tokens' own probabilities, gathered at the
// start in one round of loads, so an accepted draft costs no pass over a
// distribution.  Rows are read where the sum of what is left matters: after a
// refusal with another sibling to try, and for the last token.  `r` in shared
// memory holds the CTA's part of what is left.  Sums are whole numbers, so the
// reductions' order does not show.  What bounds a batch is the rows' bytes; a
// thread keeps four (eight with a draft) 16-byte loads in flight.
__global__ void __cluster_dims__(kVerCtas, 1, 1) __launch_bounds__(kVerThreads) verify(VerifyParams v, int per, int vec) {
    extern __shared__ __align__(16) float r[];
    __shared__ VerSmem sm;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, rank = (int)cluster_rank();
    const int b = blockIdx.x / kVerCtas;
    const int lo = v.indptr[b], hi = v.indptr[b + 1];
    const int V = v.vocab;
    int n = hi - lo;
    if (tid == 0) sm.nmine = 0;
    const bool sound = lo >= 0 && hi >= lo && hi <= v.num_nodes && n <= kMaxNodes;
    if (!sound || n == 0) {  // the same in every CTA of the cluster
        if (rank == 0) {
            for (int j = tid; j < v.width; j += kVerThreads) v.accept_index[(int64_t)b * v.width + j] = -1;
            if (tid == 0) {
                v.accept_len[b] = 0;
                v.next_token[b] = -1;
                if (!sound) atomicOr(v.status, CSGMV_KV_STATUS_BAD_TREE);
            }
        }
        return;
    }
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
    for (int i = tid; i < n; i += kVerThreads)
        for (int k = sm.first[i]; k >= 0; k = sm.next[k]) sm.parent[k] = i;
    __syncthreads();
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
    // What a row leaves in r, and its sum over the vocabulary: the row itself,
    // one refusal of it, or another refusal of what r holds.  sm.total: the
    // CTA's part, sm.warp: the running sum ahead of each warp.
    auto pass = [&](auto kind_tag, const float *p, const float *q, float z) -> long long {
        constexpr int kind = decltype(kind_tag)::value;
        Steps s = {0, 0};
        auto one = [&](float x, float y) { return kind == kRowPlain ? x : refuse(x, z, y); };
        int i0 = w0;
        if (vec) {
            constexpr int U = 4;
            for (; i0 + U * 128 <= w1; i0 += U * 128) {
                float4 a[U], b[U];
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const int i = i0 + u * 128 + lane * 4;
                    a[u] = kind == kRowAgain ? *reinterpret_cast<const float4 *>(r + i - v0)
                                             : __ldg(reinterpret_cast<const float4 *>(p + i));
                    if (kind != kRowPlain) b[u] = __ldg(reinterpret_cast<const float4 *>(q + i));
                }
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const int i = i0 + u * 128 + lane * 4;
                    float4 x = a[u];
                    if (kind != kRowPlain)
                        x = make_float4(one(a[u].x, b[u].x), one(a[u].y, b[u].y), one(a[u].z, b[u].z), one(a[u].w, b[u].w));
                    *reinterpret_cast<float4 *>(r + i - v0) = x;
                    s.add(x.x);
                    s.add(x.y);
                    s.add(x.z);
                    s.add(x.w);
                }
            }
        }
        for (int i = i0 + lane; i < w1; i += 32) {
            const float x = one(kind == kRowAgain ? r[i - v0] : __ldg(p + i), kind == kRowPlain ? 0.0f : __ldg(q + i));
            r[i - v0] = x;
            s.add(x);
        }
        // (a lane reads and writes its own part of r only, so another pass may follow)
        long long t = warp_sum(s.total());
        if (kind == kRowPlain) {  // the children's tokens are taken out
            __syncwarp();
            for (int c = 0; c < sm.nmine; ++c) {
                const int i = sm.mine[c];
                if (i >= w0 && i < w1) {
                    t -= fixed44(r[i - v0]);
                    __syncwarp();
                    if (lane == 0) r[i - v0] = 0.0f;
                    __syncwarp();
                }
            }
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
        const long long c = lane < kVerCtas ? dsmem_ld_i64(dsmem_addr(&sm.total, lane)) : 0;
        return warp_sum(c);
    };
    using Plain = std::integral_constant<int, kRowPlain>;
    using Refuse = std::integral_constant<int, kRowRefuse>;
    using Again = std::integral_constant<int, kRowAgain>;
    // The walk, the same in every thread of the cluster.
    int cur = 0, count = 1;
    int32_t *path = v.accept_index + (int64_t)b * v.width;
    if (rank == 0 && tid == 0) path[0] = 0;
    bool have_r = false;
    long long total = 0;
    while (true) {
        const float *p = v.target + (int64_t)(lo + cur) * v.target_stride;
        const float *q = v.draft ? v.draft + (int64_t)(lo + cur) * v.draft_stride : nullptr;
        int hit = -1;
        have_r = false;
        if (q) {
            float z = 1.0f;
            int refused = 0;
            for (int k = sm.first[cur]; k >= 0 && z > 0.0f; k = sm.next[k]) {
                if (sm.token[k] < 0) continue;
                float rk = sm.p[k];
                for (int m = 0; m < refused; ++m) rk = refuse(rk, sm.z[m], sm.q[k]);
                if (__fmul_rn(__fmul_rn(sm.u[k], sm.q[k]), z) < rk) {
                    hit = k;
                    break;
                }
                if (tid == 0) sm.z[refused] = z;
                ++refused;
                if (refused == 1) total = pass(Refuse{}, p, q, z);
                else total = pass(Again{}, p, q, z);
                cluster_sync();  // the other CTAs have read sm.total
                have_r = true;
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
            if (!have_r) {
                if (!q) {
                    // the children's distinct tokens in this CTA's part
                    if (tid == 0) {
                        int n = 0;
                        for (int k = sm.first[cur]; k >= 0; k = sm.next[k]) {
                            const int t = sm.token[k];
                            bool seen = t < v0 || t >= v1;
                            for (int e = 0; e < n; ++e) seen |= sm.mine[e] == t;
                            if (!seen) sm.mine[n++] = t;
                        }
                        sm.nmine = n;
                    }
                    __syncthreads();
                }
                total = pass(Plain{}, p, q, 0.0f);
            }
            if (total == 0) {  // nothing is left: the distribution itself
                cluster_sync();
                if (tid == 0) sm.nmine = 0;
                __syncthreads();
                total = pass(Plain{}, p, q, 0.0f);
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
    const long long t = lane < kVerCtas ? dsmem_ld_i64(dsmem_addr(&sm.total, lane)) : 0;
    const long long before = warp_sum(lane < rank ? t : 0ll);
    const long long mine = __shfl_sync(kFullMask, t, rank);
    cluster_sync();  // no CTA leaves while another reads its shared memory
    if (!fits || total == 0 || aim < before || aim >= before + mine) return;
    const long long ahead = before + sm.warp[warp];
    const long long end = warp + 1 < kVerWarps ? before + sm.warp[warp + 1] : before + mine;
    if (aim < ahead || aim >= end) return;
    long long run = ahead;
    // 128 tokens at a time, four a lane
    for (int i0 = w0; i0 < w1; i0 += 128) {
        long long x[4], sum = 0;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int i = i0 + lane * 4 + e;
            x[e] = i < w1 ? fixed44(r[i - v0]) : 0ll;
            sum += x[e];
        }
        const long long inc = run + warp_scan(sum);
        const unsigned above = __ballot_sync(kFullMask, inc > aim);
        if (above) {
            if (lane == __ffs(above) - 1) {
                long long at = inc - sum;
                int e = 0;
                while (e < 3 && at + x[e] <= aim) at += x[e++];
                v.next_token[b] = i0 + lane * 4 + e;
            }
            return;
        }
        run = __shfl_sync(kFullMask, inc, 31);
    }
}

}  // namespace

cudaError_t launch_build_tree(const TreeParams &p, cudaStream_t stream) {
    return launch_kernel(build_tree, dim3((unsigned)p.bs), kTreeThreads, 0, stream, 0, false, p);
}

cudaError_t launch_verify(const VerifyParams &p, cudaStream_t stream) {
    const int per = ((p.vocab + kVerCtas - 1) / kVerCtas + 127) & ~127;
    const size_t smem = (size_t)per * sizeof(float);
    static std::mutex mu;
    static std::set<int> ready;  // devices
    int dev;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    {
        std::lock_guard<std::mutex> lk(mu);
        if (!ready.count(dev)) {
            e = cudaFuncSetAttribute(verify, cudaFuncAttributeMaxDynamicSharedMemorySize, 4 * ((1 << 18) / kVerCtas + 128));
            if (e != cudaSuccess) return e;
            ready.insert(dev);
        }
    }
    auto rows16 = [](const float *q, int64_t stride) { return (reinterpret_cast<uintptr_t>(q) & 15) == 0 && stride % 4 == 0; };
    const int vec = rows16(p.target, p.target_stride) && (!p.draft || rows16(p.draft, p.draft_stride));
    return launch_kernel(verify, dim3((unsigned)p.bs * kVerCtas), kVerThreads, smem, stream, 0, false, p, per, vec);
}

}  // namespace csgmv
