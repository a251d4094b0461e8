// Residual and norms between two blocks: r' = a r + g post(x), out = pre(r').
// See include/csgmv.h (csgmv_add_norm).
//
// A row is held in registers from its one read to its one write: a warp or a CTA
// has a row, a thread N vectors of V elements, 16 in all (8 where there are few
// rows), and there are as many threads as the row's width takes.  Rows whose width
// or stride is no multiple of eight begin anywhere, but all tensors' rows alike:
// then (SHIFT) vectors begin at the last boundary before the row, and the first
// and the last one are taken by elements (8000 rows of 4097: 175 us by elements).
// Means and mean squares are taken one after the other over those registers
// (centred values are squared, not moments subtracted), in f32: a thread's
// elements in order, then a butterfly over the warp, then over the warps' sums, so
// results do not depend on timing.
//
// Measured (device time): 35507 rows of 4096, bf16 with an f32 residual (1.75 GB)
// 247 us, 7.1 TB/s, a little above a plain copy's rate; 2051 half rows of 4096 with two
// norms and a gate (84 MB, partly from L2) 16 us; one row 2.5 us: a launch, two
// rounds of loads, a barrier.  Rows above 8192 take a CTA of up to 1024 threads with 64
// registers each, one to an SM, and reach 70 % of the copy rate: nothing runs
// beside a row's barriers.
#include <algorithm>

#include "elements.cuh"
#include "serving.cuh"
#include "step.h"

namespace csgmv {
namespace {

// The row's sum of v, in every thread of the row (CTA: of the block, else of
// the warp).  `red` holds two rounds, so that one barrier a sum is enough.
template <bool CTA>
__device__ __forceinline__ float row_sum(float v, float (&red)[2][32], int &round) {
    v = warp_sum(v);
    if constexpr (CTA) {
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
    // of what does not lie as the rows do (weights)
    template <typename T>
    __device__ __forceinline__ Vec<T, V> load_other(const T *row, int k) const {
        return SHIFT ? load_elements(row, k) : ld_vec<T, V>(row + at(k));
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
        float sum = 0.0f;
#pragma unroll
        for (int k = 0; k < N; ++k)
#pragma unroll
            for (int i = 0; i < V; ++i) sum += v[k][i];
        const float mean = row_sum<CTA>(sum, red, round) / n;
#pragma unroll
        for (int k = 0; k < N; ++k)
#pragma unroll
            for (int i = 0; i < V; ++i) v[k][i] = my.any(k) && my.in(k, i) ? v[k][i] - mean : 0.0f;
    }
    float sq = 0.0f;
#pragma unroll
    for (int k = 0; k < N; ++k)
#pragma unroll
        for (int i = 0; i < V; ++i) sq = fmaf(v[k][i], v[k][i], sq);
    const float f = rsqrtf(row_sum<CTA>(sq, red, round) / n + s.eps);
#pragma unroll
    for (int k = 0; k < N; ++k) {
        if (!my.any(k)) continue;
        if (s.w) {
            if (!kEarly) w[k] = my.load_other(static_cast<const T *>(s.w), k);
#pragma unroll
            for (int i = 0; i < V; ++i) v[k][i] *= f * to_f32(w[k].e[i]);
        } else {
#pragma unroll
            for (int i = 0; i < V; ++i) v[k][i] *= f;
        }
        if (s.b) {
            const Vec<T, V> b = my.load_other(static_cast<const T *>(s.b), k);
#pragma unroll
            for (int i = 0; i < V; ++i) v[k][i] += to_f32(b.e[i]);
        }
    }
}

template <typename T, typename R, int V, int N, bool CTA, bool SHIFT>
__global__ void __launch_bounds__(CTA ? 1024 : 128) add_norm(AddNormParams p) {
    __shared__ float red[2][32];
    griddep_launch_dependents();
    griddep_wait();
    int round = 0;
    const int64_t t = CTA ? (int64_t)blockIdx.x : (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5);
    if (!CTA && t >= p.n) return;
    const T *xr = static_cast<const T *>(p.x) + t * p.x_s, *gr = static_cast<const T *>(p.gate) + t * p.g_s;
    const R *rr = static_cast<const R *>(p.r) + t * p.r_s;
    const Where<V, SHIFT> my = {p.hidden, (int)(CTA ? threadIdx.x : threadIdx.x & 31), (int)(CTA ? blockDim.x : 32),
                                SHIFT ? (int)(reinterpret_cast<uintptr_t>(xr) / sizeof(T) % V) : 0};
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
            if (my.any(k)) g[k] = SHIFT && p.g_s == 0 ? my.load_elements(gr, k) : my.load(gr, k);
    }
    float v[N][V];
#pragma unroll
    for (int k = 0; k < N; ++k)
#pragma unroll
        for (int i = 0; i < V; ++i) v[k][i] = my.any(k) ? to_f32(x[k].e[i]) : 0.0f;
    if (p.post.kind != CSGMV_NORM_NONE) normalize<T, V, N, CTA, SHIFT>(v, p.post, my, red, round);
#pragma unroll
    for (int k = 0; k < N; ++k) {
        if (!my.any(k)) continue;
        if (p.gate) {
            if (V == 1) g[k] = my.load(gr, k);
#pragma unroll
            for (int i = 0; i < V; ++i) v[k][i] *= to_f32(g[k].e[i]);
        }
        if (p.r) {
#pragma unroll
            for (int i = 0; i < V; ++i) v[k][i] = fmaf(p.scale, to_f32(r[k].e[i]), v[k][i]);
        }
        if (p.r_out) {
            Vec<R, V> o;
#pragma unroll
            for (int i = 0; i < V; ++i) o.e[i] = from_f32<R>(v[k][i]);
            my.store(static_cast<R *>(p.r_out) + t * p.ro_s, k, o);
        }
    }
    if (!p.out) return;
    if (p.pre.kind != CSGMV_NORM_NONE) normalize<T, V, N, CTA, SHIFT>(v, p.pre, my, red, round);
#pragma unroll
    for (int k = 0; k < N; ++k) {
        if (!my.any(k)) continue;
        Vec<T, V> o;
#pragma unroll
        for (int i = 0; i < V; ++i) o.e[i] = from_f32<T>(v[k][i]);
        my.store(static_cast<T *>(p.out) + t * p.o_s, k, o);
    }
}

template <typename T, typename R, int V, int N, bool CTA, bool SHIFT>
cudaError_t go(const AddNormParams &p, cudaStream_t stream) {
    const int width = p.hidden + (SHIFT ? V - 1 : 0);
    const int threads = CTA ? (width + 32 * V * N - 1) / (32 * V * N) * 32 : 128;
    const int64_t blocks = CTA ? p.n : (p.n + 3ll) / 4;
    return launch_kernel(add_norm<T, R, V, N, CTA, SHIFT>, dim3((unsigned)blocks), threads, 0, stream, 0, true, p);
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

template <typename T, typename R>
cudaError_t pick(const AddNormParams &p, cudaStream_t stream) {
    const int D = p.hidden, how = layout_of(p);
    if (how == 0) {
        if (D <= 512) return go<T, R, 8, 2, false, false>(p, stream);
        // Eight elements a thread are the faster way to few rows (1 of 8192: 2.8 us, with
        // 16 4.5), sixteen to many (8000 of 4096: 46 us, with 8 58).
        return p.n <= 152 && D <= 8192 ? go<T, R, 8, 1, true, false>(p, stream) : go<T, R, 8, 2, true, false>(p, stream);
    }
    if (how == 1 && D <= kNormMaxHidden - 8)
        return D <= 504 ? go<T, R, 8, 2, false, true>(p, stream) : go<T, R, 8, 2, true, true>(p, stream);
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
