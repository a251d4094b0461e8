// Residual and norms between two blocks: r' = a r + g post(x), out = pre(r').
// See include/csgmv.h (csgmv_add_norm).
//
// A row is held in registers from its one read to its one write: some lanes of a
// warp or a CTA have a row, a thread N vectors of V elements, 16 in all (8 where there
// are few rows or short ones), and there are as many threads as the row's width takes.
// Rows whose width or stride is no multiple of eight begin anywhere, but all tensors'
// rows alike: then (SHIFT) vectors begin at the last boundary before the row, the first
// and the last one are taken by elements, and weights, which lie otherwise, are moved
// into place from two vectors each (8000 bf16 rows of 4097: 60 us, with weights by elements
// and a row at a time 87, all by elements 175).
//
// Where many rows are to be had the next one's inputs are copied to shared memory
// while one is worked on (ahead() has the rule and both sides' figures).
//
// Means and mean squares are taken one after the other over those registers
// (centred values are squared, not moments subtracted), in f32: a thread's
// elements in order, then a butterfly over the warp, then over the warps' sums, so
// results do not depend on timing.
//
// Measured (device time): 35507 rows of 4096, bf16 with an f32 residual (1.75 GB)
// 247 us, 7.1 TB/s, a little above a plain copy's rate; 2051 half rows of 4096 with two
// norms and a gate (84 MB, partly from L2) 16 us; one row 2.5 us: a launch, two
// rounds of loads, a barrier.  Two centred norms with weights, biases and gates, 14600
// bf16 rows of 4096 (600 MB): 115 us, 5.2 TB/s, by their instructions: elements as halves
// of words and a bias in the multiplication took it there from 3.9.  (Operations on
// pairs of elements: no faster, and 17 us in place of 16: registers.)  Rows of 14336, a
// CTA of 896 threads to an SM: 6.0 TB/s, f32 5.3, two norms 4.8, centred 3.6.  1.4 million rows
// of 40: 3.8 TB/s, of 64, 128 and 256 5.7 (a vector a tensor under way in a thread, and a CTA
// ends with its rows).  f32 rows of many elements spill at 64 registers (96 bytes, where they
// begin anywhere 236), and so do the forms by elements (92 to 156).
#include <algorithm>
#include <atomic>

#include "elements.cuh"
#include "serving.cuh"
#include "step.h"

namespace csgmv {
namespace {

// Arithmetic on a thread's elements.
template <int V>
__device__ __forceinline__ void mul_all(float (&v)[V], const float (&a)[V]) {
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] *= a[i];
}
template <int V>
__device__ __forceinline__ void mul_all(float (&v)[V], float a) {
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] *= a;
}
template <int V>
__device__ __forceinline__ void add_all(float (&v)[V], float a) {
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] += a;
}
template <int V>  // v a + b
__device__ __forceinline__ void fma_all(float (&v)[V], const float (&a)[V], const float (&b)[V]) {
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] = fmaf(v[i], a[i], b[i]);
}
template <int V>  // v + a s
__device__ __forceinline__ void fma_onto(float (&v)[V], const float (&a)[V], float s) {
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] = fmaf(a[i], s, v[i]);
}
template <int N, int V>
__device__ __forceinline__ float squares(const float (&v)[N][V]) {
    float s = 0.0f;
#pragma unroll
    for (int k = 0; k < N; ++k)
#pragma unroll
        for (int i = 0; i < V; ++i) s = fmaf(v[k][i], v[k][i], s);
    return s;
}
template <int N, int V>
__device__ __forceinline__ float total(const float (&v)[N][V]) {
    float s = 0.0f;
#pragma unroll
    for (int k = 0; k < N; ++k)
#pragma unroll
        for (int i = 0; i < V; ++i) s += v[k][i];
    return s;
}
// The row's sum of v, in every thread of the row (CTA: of the block, else of
// `lanes` neighbouring lanes).  `red` holds two rounds, so that one barrier a sum is
// enough.
template <bool CTA>
__device__ __forceinline__ float row_sum(float v, int lanes, float (&red)[2][32], int &round) {
    if constexpr (!CTA) {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1)
            if (o < lanes) v += __shfl_xor_sync(kFullMask, v, o);
    } else {
        v = warp_sum(v);
        const int lane = threadIdx.x & 31;
        if (lane == 0) red[round][threadIdx.x >> 5] = v;
        __syncthreads();
        v = warp_sum(lane < (int)blockDim.x / 32 ? red[round][lane] : 0.0f);
        round ^= 1;
    }
    return v;
}

// Where a thread's vectors are in its row: vector k from element at(k) on.
template <int V, bool SHIFT>
struct Where {
    int hidden, lane, threads, shift;
    __device__ __forceinline__ int at(int k) const { return (k * threads + lane) * V - (SHIFT ? shift : 0); }
    __device__ __forceinline__ bool any(int k) const { return at(k) < hidden; }
    __device__ __forceinline__ bool in(int k, int i) const { return SHIFT ? (unsigned)(at(k) + i) < (unsigned)hidden : true; }
    __device__ __forceinline__ bool whole(int k) const { return !SHIFT || (at(k) >= 0 && at(k) + V <= hidden); }
    template <typename T>
    __device__ __forceinline__ Vec<T, V> load(const T *row, int k) const {
        if (whole(k)) return ld_vec<T, V>(row + at(k));
        return load_elements(row, k);
    }
    template <typename T>
    __device__ __forceinline__ Vec<T, V> load_elements(const T *row, int k) const {
        Vec<T, V> v;
#pragma unroll
        for (int i = 0; i < V; ++i) v.e[i] = in(k, i) ? row[at(k) + i] : from_f32<T>(0.0f);
        return v;
    }
    // of what does not lie as the rows do (weights): two vectors at its own boundaries, from
    // which the elements are taken; the row is as far behind those all along
    template <typename T>
    __device__ __forceinline__ Vec<T, V> load_other(const T *row, int k) const {
        if constexpr (!SHIFT) {
            return ld_vec<T, V>(row + at(k));
        } else {
            constexpr int P = 16 / (int)sizeof(T);
            const int behind = (int)((reinterpret_cast<uintptr_t>(row) / sizeof(T) + (unsigned)at(k)) % P), from = at(k) - behind;
            if (from < 0 || from + V + P > hidden) return load_elements(row, k);
            // moved down by `behind` elements: by four, two and one of them, or not
            const Vec<T, V + P> wide = ld_vec<T, V + P>(row + from);
            constexpr int W = (V + P) * (int)sizeof(T) / 4, PerWord = 4 / (int)sizeof(T);
            uint32_t w[W];
#pragma unroll
            for (int i = 0; i < W; ++i) w[i] = reinterpret_cast<const uint32_t *>(&wide)[i];
#pragma unroll
            for (int m = P / 2; m >= PerWord; m /= 2)
#pragma unroll
                for (int i = 0; i + m / PerWord < W; ++i) w[i] = behind & m ? w[i + m / PerWord] : w[i];
            Vec<T, V> v;
#pragma unroll
            for (int i = 0; i < V / PerWord; ++i)
                reinterpret_cast<uint32_t *>(&v)[i] = PerWord == 1 ? w[i] : __funnelshift_r(w[i], w[i + 1], (behind & 1) * 16);
            return v;
        }
    }
    template <typename T>
    __device__ __forceinline__ void store(T *row, int k, const Vec<T, V> &v) const {
        if (whole(k)) {
            st_vec<T, V>(row + at(k), v);
        } else {
#pragma unroll
            for (int i = 0; i < V; ++i)
                if (in(k, i)) row[at(k) + i] = v.e[i];
        }
    }
};

template <typename T, int V, int N, bool CTA, bool SHIFT>
__device__ __forceinline__ void normalize(float (&v)[N][V], const NormSide &s, const Where<V, SHIFT> &my, float (&red)[2][32], int &round) {
    // weights are asked for before the sums, and come while those are taken (of
    // single elements they would take a register each)
    constexpr bool kEarly = V > 1 && !SHIFT;
    Vec<T, V> w[N];
    if (kEarly && s.w) {
#pragma unroll
        for (int k = 0; k < N; ++k)
            if (my.any(k)) w[k] = my.load_other(static_cast<const T *>(s.w), k);
    }
    const float n = (float)my.hidden;
    if (s.kind == CSGMV_NORM_LAYER) {
        const float mean = row_sum<CTA>(total(v), my.threads, red, round) / n;
#pragma unroll
        for (int k = 0; k < N; ++k) {
            if (!my.any(k)) continue;
            add_all(v[k], -mean);
            if (!my.whole(k)) {
#pragma unroll
                for (int i = 0; i < V; ++i) v[k][i] = my.in(k, i) ? v[k][i] : 0.0f;
            }
        }
    }
    const float f = rsqrtf(row_sum<CTA>(squares(v), my.threads, red, round) / n + s.eps);
#pragma unroll
    for (int k = 0; k < N; ++k) {
        if (!my.any(k)) continue;
        float u[V];
        if (s.w) {
            if (!kEarly) w[k] = my.load_other(static_cast<const T *>(s.w), k);
            widen(w[k], u);
            mul_all(u, f);
        } else {
#pragma unroll
            for (int i = 0; i < V; ++i) u[i] = f;
        }
        if (s.b) {
            float b[V];
            widen(my.load_other(static_cast<const T *>(s.b), k), b);
            fma_all(v[k], u, b);
        } else {
            mul_all(v[k], u);
        }
    }
}

// Row t from x in f32 on; `live`: whether it is one.  Vectors of the gate and the
// residual come from gate(k) and residual(k), and then(): there are no more of them.
template <typename T, typename R, int V, int N, bool CTA, bool SHIFT, typename G, typename Q, typename F>
__device__ __forceinline__ void one_row(const AddNormParams &p, int64_t t, bool live, const Where<V, SHIFT> &my, float (&v)[N][V], G gate,
                                        Q residual, F then, float (&red)[2][32], int &round) {
    if (p.post.kind != CSGMV_NORM_NONE) normalize<T, V, N, CTA, SHIFT>(v, p.post, my, red, round);
#pragma unroll
    for (int k = 0; k < N; ++k) {
        if (!my.any(k)) continue;
        if (p.gate) {
            float g[V];
            widen(gate(k), g);
            mul_all(v[k], g);
        }
        if (p.r) {
            float r[V];
            widen(residual(k), r);
            fma_onto(v[k], r, p.scale);
        }
        if (p.r_out && live) {
            my.store(static_cast<R *>(p.r_out) + t * p.ro_s, k, narrow<R>(v[k]));
        }
    }
    then();
    if (!p.out) return;
    if (p.pre.kind != CSGMV_NORM_NONE) normalize<T, V, N, CTA, SHIFT>(v, p.pre, my, red, round);
#pragma unroll
    for (int k = 0; k < N; ++k) {
        if (!my.any(k) || !live) continue;
        my.store(static_cast<T *>(p.out) + t * p.o_s, k, narrow<T>(v[k]));
    }
}

template <int V, bool SHIFT>
__device__ __forceinline__ Where<V, SHIFT> where(const AddNormParams &p, const void *row, int bytes, int lane, int threads) {
    return {p.hidden, lane, threads, SHIFT ? (int)(reinterpret_cast<uintptr_t>(row) / bytes % V) : 0};
}

// A row to a CTA, or (not CTA) to `lanes` lanes of a warp.
template <typename T, typename R, int V, int N, bool CTA, bool SHIFT>
__global__ void __launch_bounds__(CTA ? 1024 : 128) add_norm(AddNormParams p, int lanes) {
    __shared__ float red[2][32];
    griddep_launch_dependents();
    griddep_wait();
    int round = 0;
    const int64_t at = CTA ? (int64_t)blockIdx.x : (int64_t)blockIdx.x * (128 / lanes) + threadIdx.x / lanes, t = CTA ? at : min(at, (int64_t)p.n - 1);
    const T *xr = static_cast<const T *>(p.x) + t * p.x_s, *gr = static_cast<const T *>(p.gate) + t * p.g_s;
    const R *rr = static_cast<const R *>(p.r) + t * p.r_s;
    const Where<V, SHIFT> my = where<V, SHIFT>(p, xr, sizeof(T), CTA ? threadIdx.x : threadIdx.x % lanes, CTA ? blockDim.x : lanes);
    Vec<T, V> x[N], g[N];
    Vec<R, V> r[N];
#pragma unroll
    for (int k = 0; k < N; ++k)
        if (my.any(k)) x[k] = my.load(xr, k);
    if (p.r) {
#pragma unroll
        for (int k = 0; k < N; ++k)
            if (my.any(k)) r[k] = my.load(rr, k);
    }
    if (V > 1 && p.gate) {
#pragma unroll
        for (int k = 0; k < N; ++k)
            if (my.any(k)) g[k] = SHIFT && p.g_s == 0 ? my.load_other(gr, k) : my.load(gr, k);
    }
    float v[N][V];
#pragma unroll
    for (int k = 0; k < N; ++k)
#pragma unroll
        for (int i = 0; i < V; ++i) v[k][i] = my.any(k) ? to_f32(x[k].e[i]) : 0.0f;
    // (gates of single elements would take a register each)
    one_row<T, R, V, N, CTA, SHIFT>(
        p, t, CTA || at < p.n, my, v, [&](int k) { return V > 1 ? g[k] : my.load(gr, k); }, [&](int k) { return r[k]; }, [] {}, red, round);
}

// Rows t, t + gridDim.x, ... to a CTA.  The next row's inputs come to shared memory
// while one is worked on; a warp reads there only what it has asked for itself, so
// no barrier is between the two.
template <typename T, typename R, int N, bool SHIFT>
__global__ void __launch_bounds__(1024) add_norms(AddNormParams p) {
    constexpr int V = 8;
    extern __shared__ uint4 staged[];
    __shared__ float red[2][32];
    griddep_launch_dependents();
    griddep_wait();
    int round = 0;
    const bool gates = p.gate && p.g_s != 0;
    constexpr int XS = V * sizeof(T) / 16, RS = V * sizeof(R) / 16;  // places of a vector
    const int r_from = N * XS, g_from = r_from + (p.r ? N * RS : 0);
    const T *xb = static_cast<const T *>(p.x), *gb = static_cast<const T *>(p.gate);
    const R *rb = static_cast<const R *>(p.r);
    auto where_of = [&](int64_t t) { return where<V, SHIFT>(p, xb + t * p.x_s, sizeof(T), threadIdx.x, blockDim.x); };
    // Vectors k of a row of the tensor `base` to the threads' places from `to` on.  A warp
    // asks for its vectors as they lie, lane by lane, and leaves them so: where a vector
    // is two accesses, half of them are for its neighbours.  (A lane's own two, 32 bytes
    // from the next one's: an access to L2 a sector, f32 rows at 4.5 TB/s.)
    const int lane = threadIdx.x & 31, of_warp = threadIdx.x - lane;
    auto ask = [&](auto *base, auto *row, int shift, int k, int to) {
        using E = std::remove_cv_t<std::remove_pointer_t<decltype(row)>>;
        constexpr int P = 16 / (int)sizeof(E), H = V / P;
#pragma unroll
        for (int j = 0; j < H; ++j) {
            const int q = j * 32 + lane, e = (k * (int)blockDim.x + of_warp) * V + q * P - shift;
            uint4 *place = staged + (to + j) * blockDim.x + threadIdx.x;
            if (e < p.hidden && (!SHIFT || e + P > 0)) {
                // (what is before the row in its first access comes too if it is the tensor's)
                if (!SHIFT || e >= 0 || row + e >= base) cp_async16(place, row + e, SHIFT ? min(P, p.hidden - e) * (int)sizeof(E) : 16);
                else
                    for (int i = -e; i < P && e + i < p.hidden; ++i) reinterpret_cast<E *>(place)[i] = row[e + i];
            }
        }
    };
    auto ask_x = [&](int64_t t) {
        const int shift = where_of(t).shift;
#pragma unroll
        for (int k = 0; k < N; ++k) ask(xb, xb + t * p.x_s, shift, k, k * XS);
    };
    auto ask_others = [&](int64_t t) {
        const int shift = where_of(t).shift;
#pragma unroll
        for (int k = 0; k < N; ++k) {
            if (p.r) ask(rb, rb + t * p.r_s, shift, k, r_from + k * RS);
            if (gates) ask(gb, gb + t * p.g_s, shift, k, g_from + k * XS);
        }
    };
    ask_x(blockIdx.x);
    ask_others(blockIdx.x);
    for (int64_t t = blockIdx.x; t < p.n; t += gridDim.x) {
        const int64_t next = t + gridDim.x;
        const Where<V, SHIFT> my = where_of(t);
        auto get = [&](auto element, int k, int from) {
            using E = decltype(element);
            constexpr int H = V * (int)sizeof(E) / 16;
            Vec<E, V> v;
#pragma unroll
            for (int j = 0; j < H; ++j) {
                const int q = lane * H + j;
                reinterpret_cast<uint4 *>(&v)[j] = staged[(from + q / 32) * blockDim.x + of_warp + q % 32];
            }
            if (SHIFT && !my.whole(k)) {
#pragma unroll
                for (int i = 0; i < V; ++i)
                    if (!my.in(k, i)) v.e[i] = from_f32<E>(0.0f);
            }
            return v;
        };
        cp_async_wait_all();
        __syncwarp();
        float v[N][V];
#pragma unroll
        for (int k = 0; k < N; ++k) {
            Vec<T, V> x;
            if (my.any(k)) x = get(T(), k, k * XS);
            if (my.any(k)) widen(x, v[k]);
            else
#pragma unroll
                for (int i = 0; i < V; ++i) v[k][i] = 0.0f;
        }
        __syncwarp();  // (read before it is written)
        if (next < p.n) ask_x(next);
        one_row<T, R, V, N, true, SHIFT>(
            p, t, true, my, v, [&](int k) { return gates ? get(T(), k, g_from + k * XS) : my.load_other(gb, k); },
            [&](int k) { return get(R(), k, r_from + k * RS); },
            [&] {
                __syncwarp();
                if (next < p.n) ask_others(next);
            },
            red, round);
    }
}

template <typename T, typename R, int V, int N, bool CTA, bool SHIFT>
cudaError_t go(const AddNormParams &p, cudaStream_t stream) {
    const int width = p.hidden + (SHIFT ? V - 1 : 0);
    const int threads = CTA ? (width + 32 * V * N - 1) / (32 * V * N) * 32 : 128;
    int lanes = 32;
    while (!CTA && lanes > 1 && lanes / 2 * V * N >= width) lanes /= 2;
    const int64_t blocks = CTA ? p.n : (p.n + (int64_t)(128 / lanes) - 1) / (128 / lanes);
    return launch_kernel(add_norm<T, R, V, N, CTA, SHIFT>, dim3((unsigned)blocks), threads, 0, stream, 0, true, p, lanes);
}

constexpr int kMaxDevices = 64;
constexpr int kSharedOfSm = 227 * 1024, kThreadsOfSm = 1024;  // (threads: of 64 registers)

template <typename T, typename R, int N, bool SHIFT>
cudaError_t stream_rows(const AddNormParams &p, cudaStream_t stream) {
    constexpr int V = 8;
    static std::atomic<bool> ready[kMaxDevices];  // whether the kernel may use all the shared memory it needs (twice does no harm)
    int dev;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev >= kMaxDevices || !ready[dev].load(std::memory_order_acquire)) {
        const void *fn = reinterpret_cast<const void *>(add_norms<T, R, N, SHIFT>);
        if ((e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, 1024 * N * V * (int)(2 * sizeof(T) + sizeof(R)))) != cudaSuccess)
            return e;
        if ((e = cudaFuncSetAttribute(fn, cudaFuncAttributePreferredSharedMemoryCarveout, cudaSharedmemCarveoutMaxShared)) != cudaSuccess)
            return e;
        if (dev < kMaxDevices) ready[dev].store(true, std::memory_order_release);
    }
    const int width = p.hidden + (SHIFT ? V - 1 : 0), threads = (width + 32 * V * N - 1) / (32 * V * N) * 32;
    const size_t smem = (size_t)threads * N * V * (sizeof(T) + (p.r ? sizeof(R) : 0) + (p.gate && p.g_s ? sizeof(T) : 0));
    const int per = std::max(1, std::min(kThreadsOfSm / threads, (int)(kSharedOfSm / (smem + 1024 + sizeof(float) * 64))));
    return launch_kernel(add_norms<T, R, N, SHIFT>, dim3((unsigned)std::min(p.n, 152 * per)), threads, smem, stream, 0, true, p);
}

// How rows lie: 0: all begin at vectors of eight (of f32: two of 16 bytes), 1: each
// tensor's as far behind one, 2: otherwise.
int layout_of(const AddNormParams &p) {
    const struct { const void *at; int64_t stride; int dtype; } rows[] = {
        {p.x, p.x_s, p.dtype}, {p.out, p.o_s, p.dtype}, {p.g_s ? p.gate : nullptr, p.g_s, p.dtype}, {p.r, p.r_s, p.r_dtype}, {p.r_out, p.ro_s, p.r_dtype}};
    uint64_t others = reinterpret_cast<uintptr_t>(p.post.w) | reinterpret_cast<uintptr_t>(p.post.b) | reinterpret_cast<uintptr_t>(p.pre.w) |
                      reinterpret_cast<uintptr_t>(p.pre.b) | (p.g_s ? 0 : reinterpret_cast<uintptr_t>(p.gate));
    const uint64_t first = reinterpret_cast<uintptr_t>(p.x) / dtype_bytes(p.dtype) % 8;
    bool aligned = others % 16 == 0 && p.hidden % 8 == 0, alike = true;
    for (const auto &r : rows) {
        if (!r.at) continue;
        const int bytes = dtype_bytes(r.dtype);
        const uint64_t begin = reinterpret_cast<uintptr_t>(r.at) / bytes;
        aligned = aligned && reinterpret_cast<uintptr_t>(r.at) % 16 == 0 && r.stride % 8 == 0;
        // an f32 row's vectors are of four: where those of eight begin, they do
        alike = alike && (bytes == 4 && p.dtype != r.dtype ? begin % 4 == first % 4 : begin % 8 == first) && (r.stride - p.x_s) % 8 == 0;
    }
    return aligned ? 0 : alike ? 1 : 2;
}

// Whether the next row's inputs come beside a row's work.  That pays where a row has few
// instructions for its bytes, or so many threads that little else is on the SM, and
// where a CTA has four rows at least.  TB/s with and without, 600 MB of bf16 rows: one norm, of
// 2048 5.8 and 5.9, of 4096 6.0 and 5.5, of 8192 6.5 and 5.2, of 14336 6.0 and 4.4; with an f32
// residual, of 4096 5.4 and 6.8, of 14336 6.1 and 6.2; two norms, of 4096 5.4 and 5.2 (centred 4.0
// and 4.5), of 14336 4.8 and 4.2 (3.6 and 3.5).  f32 rows of 14336 4.6 and 5.3.  (us: 700 and 3000 rows
// of 4096 5.1 and 4.7, 15.8 and 16.8.)  With a gate a token it pays for some and costs others, and none take
// it: of 4096 one norm 5.9 and 6.0, two centred 4.5 and 5.2; of 14336 one norm 6.2 and 5.1, two 5.0 and
// 4.8, centred 4.0 and 4.1, two with an f32 residual 5.2 and 5.5.
template <typename T, typename R>
bool ahead(const AddNormParams &p) {
    if (sizeof(T) != 2 || (p.gate && p.g_s)) return false;
    const bool one = p.post.kind == CSGMV_NORM_NONE || p.pre.kind == CSGMV_NORM_NONE;
    return (p.hidden > 8192 || (p.hidden >= 4096 && sizeof(R) == 2 && one)) && p.n >= 4ll * 152 * std::max(1, kThreadsOfSm * 16 / p.hidden);
}

template <typename T, typename R>
cudaError_t pick(const AddNormParams &p, cudaStream_t stream) {
    const int D = p.hidden, how = layout_of(p);
    if (how == 0) {
        if (D <= 256) return go<T, R, 8, 1, false, false>(p, stream);
        if (D <= 512) return go<T, R, 8, 2, false, false>(p, stream);
        // Eight elements a thread are the faster way to few rows (1 of 8192: 2.8 us, with
        // 16 4.5), sixteen to many (8000 of 4096: 46 us, with 8 58).
        if (p.n <= 152 && D <= 8192) return go<T, R, 8, 1, true, false>(p, stream);
        if constexpr (sizeof(T) == 2)
            if (ahead<T, R>(p)) return stream_rows<T, R, 2, false>(p, stream);
        return go<T, R, 8, 2, true, false>(p, stream);
    }
    if (how == 1 && D <= kNormMaxHidden - 8) {
        if (D <= 248) return go<T, R, 8, 1, false, true>(p, stream);
        if (D <= 504) return go<T, R, 8, 2, false, true>(p, stream);
        // (of 16 bits: 152 rows of 4097 3.6 us, one at a time 5.1; f32: 4.9 TB/s and 5.4)
        if constexpr (sizeof(T) == 2) return stream_rows<T, R, 2, true>(p, stream);
        else return go<T, R, 8, 2, true, true>(p, stream);
    }
    return D <= 512 ? go<T, R, 1, 16, false, false>(p, stream) : go<T, R, 1, 16, true, false>(p, stream);
}

}  // namespace

cudaError_t launch_add_norm(const AddNormParams &p, cudaStream_t stream) {
    const bool wide = p.r_dtype == CSGMV_DTYPE_F32;
    switch (p.dtype) {
        case CSGMV_DTYPE_BF16:
            return wide ? pick<__nv_bfloat16, float>(p, stream) : pick<__nv_bfloat16, __nv_bfloat16>(p, stream);
        case CSGMV_DTYPE_F16:
            return wide ? pick<__half, float>(p, stream) : pick<__half, __half>(p, stream);
        default:
            return pick<float, float>(p, stream);
    }
}

}  // namespace csgmv
