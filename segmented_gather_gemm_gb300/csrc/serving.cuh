// Device and launch helpers shared by the serving step's kernels.
#pragma once
#include <cuda_runtime.h>
#include <cstdint>

#include "csgmv_internal.h"
#include "device_utils.cuh"
#include "serving.h"

namespace csgmv {

constexpr uint32_t kFullMask = 0xffffffffu;

__device__ __forceinline__ uint4 ldg16(const void *p) { return __ldg(reinterpret_cast<const uint4 *>(p)); }
// 16-byte load and store of data that is touched once.
__device__ __forceinline__ uint4 ld_stream16(const void *p) { return __ldcs(reinterpret_cast<const uint4 *>(p)); }
__device__ __forceinline__ void st_stream16(void *p, uint4 v) { __stcs(reinterpret_cast<uint4 *>(p), v); }

__device__ __forceinline__ void cluster_sync() {
    cluster_arrive();
    cluster_wait();
}
__device__ __forceinline__ int dsmem_ld_i32(uint32_t addr) {
    int v;
    asm volatile("ld.shared::cluster.s32 %0, [%1];\n" : "=r"(v) : "r"(addr) : "memory");
    return v;
}
__device__ __forceinline__ long long dsmem_ld_i64(uint32_t addr) {
    long long v;
    asm volatile("ld.shared::cluster.s64 %0, [%1];\n" : "=l"(v) : "r"(addr) : "memory");
    return v;
}

template <typename T>
__device__ __forceinline__ T warp_sum(T v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kFullMask, v, o);
    return v;
}
// Inclusive prefix sum over the warp.
template <typename T>
__device__ __forceinline__ T warp_scan(T v) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const T n = __shfl_up_sync(kFullMask, v, o);
        if (lane >= o) v += n;
    }
    return v;
}
// Exclusive prefix sum over the block (blockDim.x a multiple of 32, at most
// 1024; `ws` 33 entries of shared memory); the block's total in *total.
template <typename T>
__device__ __forceinline__ T block_scan_ex(T v, T *ws, T *total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
    const T inc = warp_scan(v);
    if (lane == 31) ws[warp] = inc;
    __syncthreads();
    if (warp == 0) {
        const T w = lane < nw ? ws[lane] : T(0);
        const T s = warp_scan(w);
        ws[lane] = s - w;
        if (lane == 31) ws[32] = s;
    }
    __syncthreads();
    const T pre = ws[warp] + inc - v;
    *total = ws[32];
    __syncthreads();
    return pre;
}

// Launch with an optional cluster and, with `dependent`, programmatic
// dependent launch: the kernel may be set up while the one before it in the
// stream still runs, and waits for it in griddep_wait().
template <typename... KArgs, typename... Args>
inline cudaError_t launch_kernel(void (*kernel)(KArgs...), dim3 grid, int block, size_t smem, cudaStream_t stream, int cluster,
                                 bool dependent, const Args &...args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3((unsigned)block);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute at[2];
    int n = 0;
    if (cluster > 1) {
        at[n].id = cudaLaunchAttributeClusterDimension;
        at[n].val.clusterDim.x = (unsigned)cluster;
        at[n].val.clusterDim.y = 1;
        at[n].val.clusterDim.z = 1;
        ++n;
    }
    if (dependent) {
        at[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        at[n].val.programmaticStreamSerializationAllowed = 1;
        ++n;
    }
    cfg.attrs = at;
    cfg.numAttrs = (unsigned)n;
    auto go = [&](const KArgs &...a) {  // arguments that have the parameters' types are not copied
        void *at[] = {const_cast<void *>(static_cast<const void *>(&a))...};
        return cudaLaunchKernelExC(&cfg, reinterpret_cast<const void *>(kernel), at);
    };
    return go(args...);
}

}  // namespace csgmv
