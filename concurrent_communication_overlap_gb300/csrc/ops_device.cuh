// ops_device.cuh -- what the routing and 4-bit kernels share beyond the device
// helpers of the GEMM: chained launches and the codes of their waits.
#pragma once

#include "c3_device.cuh"

namespace c3 {

// Waits that may give up, after those of WaitSite.
enum OpsWaitSite : int {
    kSiteFp4Producer = 8,
    kSiteFp4Mma = 9,
    kSiteFp4Epilogue = 10,
    kSiteFp4Drain = 11,
    kSiteFp4Scales = 12,
};

// ---------------------------------------------------------------- chained launches

// A kernel launched with launch_chained starts while the kernel before it on its
// stream still runs: its own set-up (barriers, TMEM, tensor maps) comes before
// chain_wait, every access to global memory after it, since chain_wait returns
// only when the kernel before has ended and its writes are visible.  It also lets
// the next chained kernel start.
__device__ __forceinline__ void chain_wait() {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
}

// cluster: CTAs of a cluster (1: none, or the kernel's own).
template <typename... Params, typename... Args>
inline cudaError_t launch_chained(void (*kernel)(Params...), dim3 grid, unsigned block, size_t smem, cudaStream_t s,
                                  unsigned cluster, Args&&... args) {
    cudaLaunchConfig_t c{};
    c.gridDim = grid;
    c.blockDim = dim3(block);
    c.dynamicSmemBytes = smem;
    c.stream = s;
    cudaLaunchAttribute attr[2] = {};
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = cluster;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    c.attrs = attr;
    c.numAttrs = cluster > 1 ? 2 : 1;
    cudaError_t e = cudaLaunchKernelEx(&c, kernel, static_cast<Params>(args)...);
    if (e != cudaSuccess) cudaGetLastError();
    return e;
}

}  // namespace c3
