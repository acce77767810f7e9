// ops_device.cuh -- what the operators' kernels share beyond the device helpers of the GEMM: chained
// launches, the codes of their waits, values by vectors, and two SMs on one tile.
#pragma once

#include "c3_device.cuh"

#include <cuda_bf16.h>

#include <mutex>

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
// the next chained kernel start (chain_next), which products under a budget of SMs
// leave out: what starts early waits on SMs that the budget leaves to others.  No
// wait with a time limit may begin before chain_ready.
__device__ __forceinline__ void chain_next() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void chain_ready() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void chain_wait() {
    chain_next();
    chain_ready();
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

// ---------------------------------------------------------------- values by vectors

// W consecutive values as fp32, whatever the type: 16 bytes at most at once.
template <int W>
__device__ __forceinline__ void load_w(const float* p, float (&v)[W]) {
    if constexpr (W == 8) {
        const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
        v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
    } else if constexpr (W == 2) {
        const float2 a = *reinterpret_cast<const float2*>(p);
        v[0] = a.x, v[1] = a.y;
    } else {
        v[0] = *p;
    }
}
template <int W>
__device__ __forceinline__ void load_w(const __nv_bfloat16* p, float (&v)[W]) {
    if constexpr (W == 1) {
        v[0] = __bfloat162float(*p);
    } else {
        uint32_t u[W / 2];
        if constexpr (W == 8) {
            const uint4 a = *reinterpret_cast<const uint4*>(p);
            u[0] = a.x, u[1] = a.y, u[2] = a.z, u[3] = a.w;
        } else {
            u[0] = *reinterpret_cast<const uint32_t*>(p);
        }
#pragma unroll
        for (int i = 0; i < W / 2; ++i) {
            v[2 * i] = __uint_as_float(u[i] << 16);
            v[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
        }
    }
}
template <int W>
__device__ __forceinline__ void store_w(float* p, const float (&v)[W]) {
    if constexpr (W == 8) {
        reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
        reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
    } else if constexpr (W == 2) {
        *reinterpret_cast<float2*>(p) = make_float2(v[0], v[1]);
    } else {
        *p = v[0];
    }
}
template <int W>
__device__ __forceinline__ void store_w(__nv_bfloat16* p, const float (&v)[W]) {
    if constexpr (W == 1) {
        *p = __float2bfloat16_rn(v[0]);
    } else {
        uint32_t u[W / 2];
#pragma unroll
        for (int i = 0; i < W / 2; ++i) {
            const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
            u[i] = *reinterpret_cast<const uint32_t*>(&h);
        }
        if constexpr (W == 8)
            *reinterpret_cast<uint4*>(p) = make_uint4(u[0], u[1], u[2], u[3]);
        else
            *reinterpret_cast<uint32_t*>(p) = u[0];
    }
}

// ---------------------------------------------------------------- clusters, and two SMs on one tile

// One lane of a converged warp.  The warps that issue tensor-core work stay
// together and predicate the instruction alone: their addresses and descriptors
// then live in uniform registers (one lane branching off to issue took 640
// cycles for a stage of four MMAs, 400 this way).
__device__ __forceinline__ uint32_t elect_lane() {
    uint32_t r;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
    return r;
}
// Arrive on this CTA's `bar` once all that the thread issued has completed.
template <int GROUP>
__device__ __forceinline__ void commit_local(uint32_t lead, uint32_t bar) {
#define C3_COMMIT(G_)                                                                                \
    asm volatile("{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %1, 0;\n\t@q tcgen05.commit.cta_group::" G_   \
                 ".mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(bar), "r"(lead) : "memory")
    if constexpr (GROUP == 2) C3_COMMIT("2");
    else C3_COMMIT("1");
#undef C3_COMMIT
}

__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ uint32_t leader_addr(uint32_t local) {
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(r) : "r"(local));
    return r;
}
__device__ __forceinline__ uint32_t peer_addr(uint32_t local, uint32_t rank) {
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(local), "r"(rank));
    return r;
}
__device__ __forceinline__ void mbar_arrive_cluster(uint32_t addr) {
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(addr) : "memory");
}
__device__ __forceinline__ void cluster_sync_all() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// The same without a fence: nothing that one CTA wrote is read by the other afterwards.
__device__ __forceinline__ void cluster_meet() {
    asm volatile("barrier.cluster.arrive.relaxed.aligned;\n\tbarrier.cluster.wait.aligned;" ::: "memory");
}
// A wait whose phase another CTA of the cluster may complete.
__device__ __forceinline__ bool mbar_try_wait_cluster(uint32_t bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    return ok != 0;
}
__device__ __forceinline__ bool mbar_wait_cluster(uint32_t bar, uint32_t parity, volatile int* abort) {
    if (mbar_try_wait_cluster(bar, parity)) return true;
    const unsigned long long t0 = globaltimer();
    for (uint32_t it = 1;; ++it) {
        if (mbar_try_wait_cluster(bar, parity)) return true;
        if ((it & 63u) == 0) {
            if (*abort) return false;
            if (globaltimer() - t0 > kWaitLimitNs) {
                *abort = 1;
                return false;
            }
        }
    }
}
__device__ __forceinline__ void tma_load_2d_pair(uint32_t dst, const CUtensorMap* map, uint32_t bar, int32_t x, int32_t y,
                                                 uint64_t policy) {
    asm volatile(
        "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint"
        " [%0], [%1, {%3, %4}], [%2], %5;" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(y), "l"(policy)
        : "memory");
}
__device__ __forceinline__ void commit_pair(uint32_t lead, uint32_t bar) {
    asm volatile(
        "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %2, 0;\n\t"
        "@q tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;\n\t}" ::"r"(bar),
        "h"((uint16_t)3), "r"(lead)
        : "memory");
}

__device__ __forceinline__ void ld_shared_v4(uint32_t addr, uint32_t* v) {
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3])
                 : "r"(addr)
                 : "memory");
}

// ---------------------------------------------------------------- accumulators to memory

// 64 bytes of each of the warp's 32 rows (16 fp32 or 32 bf16 values a lane, its
// row's) to C by way of shared memory, so that neighbouring lanes write neighbouring
// bytes, W at a time: 16 where rows of C are whole 16-byte units, else 4 or 2 (a lane
// writing its own row instead took 1485 us for 6978 x 23694 x 1942, 241 this way).
// Columns past N and rows past `rows` are left alone; ld is the distance between rows.  The 16-byte chunk j of row r
// lies at chunk j ^ ((r >> 1) & 3): no bank conflicts at 16 bytes either way.
template <typename TC, int W>
__device__ __forceinline__ void write_rows(uint32_t blk, int lane, TC* C, int64_t row0, int rows, int col0, int N, int64_t ld) {
    constexpr int kLanes = 64 / W, kAtOnce = 32 / kLanes;  // lanes a row, rows at once
    const int in = (lane % kLanes) * W, col = col0 + in / (int)sizeof(TC);
    if (col >= N) rows = 0;
    TC* c = C + (row0 + lane / kLanes) * ld + col;
#pragma unroll 4
    for (int r = lane / kLanes; r < 32; r += kAtOnce, c += kAtOnce * ld) {
        const uint32_t at = blk + (uint32_t)(r * 64 + (((in >> 4) ^ ((r >> 1) & 3)) << 4) + (in & 15));
        if (r >= rows) break;
        if constexpr (W == 16) {
            uint32_t u[4];
            ld_shared_v4(at, u);
            *reinterpret_cast<uint4*>(c) = make_uint4(u[0], u[1], u[2], u[3]);
        } else if constexpr (W == 4) {
            uint32_t u;
            asm volatile("ld.shared.b32 %0, [%1];" : "=r"(u) : "r"(at) : "memory");
            *reinterpret_cast<uint32_t*>(c) = u;
        } else {
            uint16_t u;
            asm volatile("ld.shared.b16 %0, [%1];" : "=h"(u) : "r"(at) : "memory");
            *reinterpret_cast<uint16_t*>(c) = u;
        }
    }
}

// A 32 x 32 piece, already rounded to TC.
template <typename TC>
__device__ __forceinline__ void store_piece(const uint32_t* v, uint32_t blk, int lane, int width, TC* C, int64_t row0,
                                            int rows, int col0, int N, int64_t ld) {
#pragma unroll
    for (int h = 0; h < (int)sizeof(TC) / 2; ++h) {
#pragma unroll
        for (int j = 0; j < 4; ++j)
            st_shared_v4(blk + (uint32_t)lane * 64u + (uint32_t)((j ^ ((lane >> 1) & 3)) << 4), v[16 * h + 4 * j],
                         v[16 * h + 4 * j + 1], v[16 * h + 4 * j + 2], v[16 * h + 4 * j + 3]);
        __syncwarp();
        const int col = col0 + 16 * h;
        if (width == 16) write_rows<TC, 16>(blk, lane, C, row0, rows, col, N, ld);
        else if (sizeof(TC) == 4 || width >= 4) write_rows<TC, 4>(blk, lane, C, row0, rows, col, N, ld);
        else write_rows<TC, 2>(blk, lane, C, row0, rows, col, N, ld);
        __syncwarp();
    }
}

// ---------------------------------------------------------------- tensor maps, host side

typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                  const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

inline EncodeTiledFn tensor_map_encode() {
    static EncodeTiledFn fn = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<EncodeTiledFn>(p);
    });
    return fn;
}

}  // namespace c3
