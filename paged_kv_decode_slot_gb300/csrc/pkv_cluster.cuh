// pkv_cluster.cuh - thread-block clusters: reads of each other's shared memory, and their launch.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include <utility>

namespace pkv {

// What lies at `at` (an address in this CTA's shared memory) in the shared memory of the cluster's CTA `rank`, 4 or 8
// bytes.  That CTA has started (a cluster barrier lies before) and has not left (another one follows).
template <typename T>
__device__ __forceinline__ T load_cluster(uint32_t at, int rank)
{
    uint32_t there;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(there) : "r"(at), "r"(rank));
    if constexpr (sizeof(T) == 4) {
        float v;
        asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(there) : "memory");
        return v;
    } else {
        long long v;
        asm volatile("ld.shared::cluster.b64 %0, [%1];" : "=l"(v) : "r"(there) : "memory");
        return v;
    }
}

// The cluster's barrier, in two halves: what its threads wrote before arriving is visible behind the wait.  Threads that
// have left do not count.
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_sync()
{
    cluster_arrive();
    cluster_wait();
}

// Clusters of more than 8 CTAs (16 at most) are the device's to allow.
template <typename... Params>
cudaError_t allow_wide_clusters(void (*kernel)(Params...))
{
    return cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
}

// A launch with early start (programmatic serialization), in clusters unless cluster is 1 x 1 x 1.
template <typename... Params, typename... Args>
cudaError_t launch_clusters(void (*kernel)(Params...), dim3 grid, dim3 block, dim3 cluster, size_t smem, cudaStream_t stream,
                            Args &&...args)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim = {cluster.x, cluster.y, cluster.z};
    cfg.attrs = attr;
    cfg.numAttrs = cluster.x * cluster.y * cluster.z > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kernel, std::forward<Args>(args)...);
}

}  // namespace pkv
