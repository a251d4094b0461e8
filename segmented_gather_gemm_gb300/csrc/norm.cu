// Residual and norms between two blocks: r' = a r + g post(x), out = pre(r').
// See include/csgmv.h (csgmv_add_norm).
//
// A row is held in registers from its one read to its one write: TPR threads a
// row (a warp, or a CTA of up to 1024 threads), N vectors of V elements each.
// Means and mean squares are taken one after the other over those registers
// (centred values are squared, not moments subtracted), in f32: a thread's
// elements in order, then a butterfly over the warp, then over the warps' sums, so
// results do not depend on timing.
#include "elements.cuh"
#include "serving.cuh"
#include "step.h"

namespace csgmv {
namespace {

// The row's sum of v, in every thread of the row.  `red` holds two rounds, so
// that one barrier a sum is enough.
template <int TPR>
__device__ __forceinline__ float row_sum(float v, float (&red)[2][32], int &round) {
    v = warp_sum(v);
    if constexpr (TPR > 32) {
        const int lane = threadIdx.x & 31;
        if (lane == 0) red[round][threadIdx.x >> 5] = v;
        __syncthreads();
        v = warp_sum(lane < TPR / 32 ? red[round][lane] : 0.0f);
        round ^= 1;
    }
    return v;
}

template <typename T, int V, int N, int TPR>
__device__ __forceinline__ void normalize(float (&v)[N][V], const NormSide &s, int hidden, int lane, float (&red)[2][32], int &round) {
    // weights are asked for before the sums, and come while those are taken (of
    // single elements they would take a register each)
    Vec<T, V> w[N];
    if (V > 1 && s.w) {
#pragma unroll
        for (int k = 0; k < N; ++k)
            if ((k * TPR + lane) * V < hidden) w[k] = ld_vec<T, V>(static_cast<const T *>(s.w) + (k * TPR + lane) * V);
    }
    const float n = (float)hidden;
    if (s.kind == CSGMV_NORM_LAYER) {
        float sum = 0.0f;
#pragma unroll
        for (int k = 0; k < N; ++k)
#pragma unroll
            for (int i = 0; i < V; ++i) sum += v[k][i];
        const float mean = row_sum<TPR>(sum, red, round) / n;
#pragma unroll
        for (int k = 0; k < N; ++k)
#pragma unroll
            for (int i = 0; i < V; ++i) v[k][i] = (k * TPR + lane) * V < hidden ? v[k][i] - mean : 0.0f;
    }
    float sq = 0.0f;
#pragma unroll
    for (int k = 0; k < N; ++k)
#pragma unroll
        for (int i = 0; i < V; ++i) sq = fmaf(v[k][i], v[k][i], sq);
    const float f = rsqrtf(row_sum<TPR>(sq, red, round) / n + s.eps);
#pragma unroll
    for (int k = 0; k < N; ++k) {
        if ((k * TPR + lane) * V >= hidden) continue;
        if (s.w) {
            if (V == 1) w[k] = ld_vec<T, V>(static_cast<const T *>(s.w) + (k * TPR + lane) * V);
#pragma unroll
            for (int i = 0; i < V; ++i) v[k][i] *= f * to_f32(w[k].e[i]);
        } else {
#pragma unroll
            for (int i = 0; i < V; ++i) v[k][i] *= f;
        }
        if (s.b) {
            const Vec<T, V> b = ld_vec<T, V>(static_cast<const T *>(s.b) + (k * TPR + lane) * V);
#pragma unroll
            for (int i = 0; i < V; ++i) v[k][i] += to_f32(b.e[i]);
        }
    }
}

template <typename T, typename R, int V, int N, int TPR>
__global__ void __launch_bounds__(TPR > 32 ? TPR : 128) add_norm(AddNormParams p) {
    __shared__ float red[2][32];
    griddep_launch_dependents();
    griddep_wait();
    int round = 0;
    const int lane = TPR > 32 ? threadIdx.x : threadIdx.x & 31;
    const int64_t t = TPR > 32 ? (int64_t)blockIdx.x : (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5);
    if (TPR <= 32 && t >= p.n) return;
    Vec<T, V> x[N], g[N];
    Vec<R, V> r[N];
#pragma unroll
    for (int k = 0; k < N; ++k)
        if ((k * TPR + lane) * V < p.hidden) x[k] = ld_vec<T, V>(static_cast<const T *>(p.x) + t * p.x_s + (k * TPR + lane) * V);
    if (p.r) {
#pragma unroll
        for (int k = 0; k < N; ++k)
            if ((k * TPR + lane) * V < p.hidden) r[k] = ld_vec<R, V>(static_cast<const R *>(p.r) + t * p.r_s + (k * TPR + lane) * V);
    }
    if (V > 1 && p.gate) {
#pragma unroll
        for (int k = 0; k < N; ++k)
            if ((k * TPR + lane) * V < p.hidden) g[k] = ld_vec<T, V>(static_cast<const T *>(p.gate) + t * p.g_s + (k * TPR + lane) * V);
    }
    float v[N][V];
#pragma unroll
    for (int k = 0; k < N; ++k)
#pragma unroll
        for (int i = 0; i < V; ++i) v[k][i] = (k * TPR + lane) * V < p.hidden ? to_f32(x[k].e[i]) : 0.0f;
    if (p.post.kind != CSGMV_NORM_NONE) normalize<T, V, N, TPR>(v, p.post, p.hidden, lane, red, round);
#pragma unroll
    for (int k = 0; k < N; ++k) {
        if ((k * TPR + lane) * V >= p.hidden) continue;
        if (p.gate) {
            if (V == 1) g[k] = ld_vec<T, V>(static_cast<const T *>(p.gate) + t * p.g_s + (k * TPR + lane) * V);
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
            st_vec<R, V>(static_cast<R *>(p.r_out) + t * p.ro_s + (k * TPR + lane) * V, o);
        }
    }
    if (!p.out) return;
    if (p.pre.kind != CSGMV_NORM_NONE) normalize<T, V, N, TPR>(v, p.pre, p.hidden, lane, red, round);
#pragma unroll
    for (int k = 0; k < N; ++k) {
        if ((k * TPR + lane) * V >= p.hidden) continue;
        Vec<T, V> o;
#pragma unroll
        for (int i = 0; i < V; ++i) o.e[i] = from_f32<T>(v[k][i]);
        st_vec<T, V>(static_cast<T *>(p.out) + t * p.o_s + (k * TPR + lane) * V, o);
    }
}

template <typename T, typename R, int V, int N, int TPR>
cudaError_t go(const AddNormParams &p, cudaStream_t stream) {
    const int rows = TPR > 32 ? 1 : 4;
    return launch_kernel(add_norm<T, R, V, N, TPR>, dim3((unsigned)((p.n + (int64_t)rows - 1) / rows)), TPR > 32 ? TPR : 128, 0,
                         stream, 0, true, p);
}

// Whether 16-byte (32 for f32) accesses of 8 elements reach every row.
bool vectors(const AddNormParams &p) {
    const uint64_t bits = reinterpret_cast<uintptr_t>(p.x) | reinterpret_cast<uintptr_t>(p.r) | reinterpret_cast<uintptr_t>(p.gate) |
                          reinterpret_cast<uintptr_t>(p.r_out) | reinterpret_cast<uintptr_t>(p.out) |
                          reinterpret_cast<uintptr_t>(p.post.w) | reinterpret_cast<uintptr_t>(p.post.b) |
                          reinterpret_cast<uintptr_t>(p.pre.w) | reinterpret_cast<uintptr_t>(p.pre.b);
    const int64_t strides = p.x_s | (p.r ? p.r_s : 0) | (p.gate ? p.g_s : 0) | (p.r_out ? p.ro_s : 0) | (p.out ? p.o_s : 0);
    return (bits & 15) == 0 && (strides & 7) == 0 && p.hidden % 8 == 0;
}

template <typename T, typename R>
cudaError_t pick(const AddNormParams &p, cudaStream_t stream) {
    const int D = p.hidden;
    if (vectors(p)) {
        if (D <= 256) return go<T, R, 8, 1, 32>(p, stream);
        if (D <= 1024) return go<T, R, 8, 1, 128>(p, stream);
        if (D <= 4096) return p.n <= 152 ? go<T, R, 8, 1, 512>(p, stream) : go<T, R, 8, 2, 256>(p, stream);
        if (D <= 8192) return go<T, R, 8, 4, 256>(p, stream);
        return go<T, R, 8, 4, 512>(p, stream);
    }
    if (D <= 256) return go<T, R, 1, 8, 32>(p, stream);
    if (D <= 4096) return go<T, R, 1, 16, 256>(p, stream);
    return go<T, R, 1, 16, 1024>(p, stream);
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
