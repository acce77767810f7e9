// fp4_gemm.cu -- products of microscaled 4-bit matrices: C = A * B^T with both
// operands in 4-bit codes and block scales, accumulated in fp32 by the
// block-scaled tensor-core instruction (tcgen05.mma, kind mxf4 / mxf4nvf4), and
// the same for the experts of a sparse layer, whose rows of A lie one expert
// after the other.
//
// Layout (one CTA per SM, 192 threads), as in the bf16 kernel:
//   warp 0      producer: per stage 128 rows of A and BN rows of B, 256 columns
//               of 4 bits each (one 128-byte swizzle row), by TMA, and their
//               scales, which lie in memory as the tensor cores take them, by
//               plain bulk copies;
//   warp 1      TMEM owner and MMA issuer: the stage's scales go from shared
//               memory to TMEM (tcgen05.cp, 128 rows x 4 scales an instruction,
//               copied to all four lane quarters), then four MMAs of 64 columns;
//   warps 2..5  epilogue: accumulator to registers, times the matrices' fp32
//               scales, rounded once to the output type, to C.
#include "c3_device.cuh"
#include "c3_internal.h"

#include <cuda_bf16.h>

#include <mutex>

namespace c3 {

constexpr int kFM = 128;             // rows of A in a tile
constexpr int kFK = 256;             // columns of a stage: 128 bytes of codes
constexpr int kFThreads = 192;
constexpr int kFGroupM = 16;
constexpr int kFSmemLimit = 232448;  // 227 KiB
constexpr int kFMaxExperts = 1024;

template <bool NV, int BN>
struct Fp4Cfg {
    static constexpr int kKT = NV ? 4 : 2;                    // scale tiles along a stage's columns
    static constexpr uint32_t kABytes = kFM * 128;
    static constexpr uint32_t kBBytes = BN * 128;
    static constexpr uint32_t kSfa = kKT * 512;
    static constexpr uint32_t kSfb = kKT * 512 * (BN / 128);
    static constexpr uint32_t kStage = kABytes + kBBytes + (kSfa + kSfb + 1023) / 1024 * 1024;
    static constexpr int kExtra = 1024 + 512 + 4 * (kFMaxExperts + 1);
    static constexpr int kStages = (kFSmemLimit - kExtra) / (int)kStage > 8 ? 8 : (kFSmemLimit - kExtra) / (int)kStage;
    static constexpr int kAccBufs = 2;
    static constexpr int kSfCol = kAccBufs * BN;              // scales behind the accumulators
    static constexpr int kSmem = kStages * (int)kStage + kExtra;
    static_assert(kSfCol + kKT * 4 * (1 + BN / 128) <= 512, "TMEM");
};

struct Fp4GemmArgs {
    const uint8_t* sfa;
    const uint8_t* sfb;
    const float* ga;
    const float* gb;
    const int32_t* offsets;  // experts' rows of A, or NULL
    const int32_t* counts;
    void* C;
    int64_t M;
    int N, K;
    int experts;
    int k_tiles;             // scale tiles along K
    int b_row_tiles;         // scale tiles along one matrix of B
    int num_m, num_n, num_kb;
};

// A matrix descriptor without swizzle for the scales: 8 x 16-byte groups 128 bytes apart.
__device__ __forceinline__ uint64_t scale_desc(uint32_t saddr) {
    return (uint64_t)((saddr & 0x3FFFFu) >> 4) | ((uint64_t)(128 >> 4) << 32) | ((uint64_t)1 << 46);
}
// Codes: K-major, 128-byte swizzle, 1024 bytes between 8-row groups.
__device__ __forceinline__ uint64_t code_desc(uint32_t saddr) {
    return (uint64_t)((saddr & 0x3FFFFu) >> 4) | ((uint64_t)1 << 16) | ((uint64_t)(1024 >> 4) << 32) |
           ((uint64_t)1 << 46) | ((uint64_t)2 << 61);
}
__device__ __forceinline__ void tmem_copy_scales(uint32_t taddr, uint64_t sdesc) {
    asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(sdesc) : "memory");
}

// Instruction descriptor: E2M1 codes (bits 7-9, 10-11 = 1), both K-major, N >> 3
// at bits 17-22, power-of-two scales at bit 23, M >> 7 at bits 27-28; the scale
// factors' byte within their column (0 or 2) at bits 4-5 (B) and 29-30 (A).
template <bool NV, int BN>
__device__ __forceinline__ uint32_t fp4_idesc() {
    return (1u << 7) | (1u << 10) | ((uint32_t)(BN >> 3) << 17) | (NV ? 0u : 1u << 23) | (1u << 27);
}
template <bool NV>
__device__ __forceinline__ void mma_fp4(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sfa, uint32_t sfb,
                                        uint32_t accumulate) {
    if constexpr (NV)
        asm volatile(
            "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %6, 0;\n\t"
            "tcgen05.mma.cta_group::1.kind::mxf4nvf4.block_scale.scale_vec::4X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d),
            "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
            : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %6, 0;\n\t"
            "tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d),
            "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
            : "memory");
}

// One output tile: its expert, rows and columns.
struct Fp4Tile {
    int expert;       // matrix of B
    int64_t row0;     // first row of A and C
    int rows;         // rows of the tile that are the expert's (or the matrix's)
    int nb;
};

template <int BN>
__device__ __forceinline__ Fp4Tile fp4_tile(const Fp4GemmArgs& g, const int* prefix, int t) {
    Fp4Tile r;
    if (g.offsets == nullptr) {
        const int per = kFGroupM * g.num_n, grp = t / per, first = grp * kFGroupM;
        const int gm = min(g.num_m - first, kFGroupM), in = t - grp * per;
        const int mb = first + in % gm;
        r.expert = 0;
        r.row0 = (int64_t)mb * kFM;
        r.rows = (int)min((int64_t)kFM, g.M - r.row0);
        r.nb = in / gm;
        return r;
    }
    // the last expert whose first tile is not past t: prefix counts row tiles
    int lo = 0, hi = g.experts;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if ((int64_t)prefix[mid] * g.num_n <= t) lo = mid;
        else hi = mid;
    }
    const int in = t - prefix[lo] * g.num_n, mt = prefix[lo + 1] - prefix[lo];
    const int mb = in % mt;
    r.expert = lo;
    r.nb = in / mt;
    r.row0 = (int64_t)g.offsets[lo] + (int64_t)mb * kFM;
    r.rows = min(kFM, g.counts[lo] - mb * kFM);
    return r;
}

template <bool NV, int BN, typename TC>
__global__ void __launch_bounds__(kFThreads, 1)
    fp4_gemm_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB, Fp4GemmArgs g,
                    DevStatus* st) {
    using Cfg = Fp4Cfg<NV, BN>;
    constexpr int S = Cfg::kStages;
    constexpr int KT = Cfg::kKT;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    const uint32_t raw = smem_addr(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    uint8_t* gbase = smem_raw + (base - raw);
    uint64_t* bars = reinterpret_cast<uint64_t*>(gbase + S * Cfg::kStage);
    // full [0, S), empty [S, 2S), accumulator full [2S, 2S+2), empty [2S+2, 2S+4), drain 2S+4
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 2 * S + 5);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
    int* prefix = reinterpret_cast<int*>(gbase + S * Cfg::kStage + 512);
    auto bar = [&](int i) { return smem_addr(&bars[i]); };
    const int TFULL = 2 * S, TEMPTY = 2 * S + 2, DRAIN = 2 * S + 4;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        *abort_flag = 0;
        for (int i = 0; i < S; ++i) {
            mbar_init(bar(i), 1);
            mbar_init(bar(S + i), 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(bar(TFULL + b), 1);
            mbar_init(bar(TEMPTY + b), 4 * 32);
        }
        mbar_init(bar(DRAIN), 1);
        fence_barrier_init();
        prefetch_tensormap(&tmA);
        prefetch_tensormap(&tmB);
    }
    if (warp == 1) {
        tmem_alloc(smem_addr(tmem_slot), 512);
        tmem_relinquish();
    }
    if (g.offsets && warp == 2) {
        // Row tiles before each expert.  An expert whose rows do not lie in A, or
        // do not start at a whole tile, has none: nothing out of range is touched.
        int run = 0;
        for (int e0 = 0; e0 < g.experts; e0 += 32) {
            const int e = e0 + lane;
            int mt = 0;
            if (e < g.experts) {
                const int64_t off = g.offsets[e], c = g.counts[e];
                if (off >= 0 && c > 0 && off % kTileRows == 0 && off + c <= g.M) mt = (int)((c + kFM - 1) / kFM);
            }
            int incl = mt;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int v = __shfl_up_sync(0xffffffffu, incl, o);
                if (lane >= o) incl += v;
            }
            if (e < g.experts) prefix[e + 1] = run + incl;
            run += __shfl_sync(0xffffffffu, incl, 31);
        }
        if (lane == 0) prefix[0] = 0;
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    const int total = g.offsets ? prefix[g.experts] * g.num_n : g.num_m * g.num_n;

    if (warp == 0) {
        if (lane == 0) {
            int stage = 0;
            uint32_t phase = 0;
            bool ok = true;
            for (int t = blockIdx.x; ok && t < total; t += gridDim.x) {
                const Fp4Tile tile = fp4_tile<BN>(g, prefix, t);
                const uint8_t* sfa = g.sfa + (tile.row0 / kTileRows) * g.k_tiles * 512;
                const int rt0 = tile.nb * (BN / 128);
                const uint8_t* sfb = g.sfb + ((int64_t)tile.expert * g.b_row_tiles + rt0) * g.k_tiles * 512;
                const int nrt = min(BN / 128, g.b_row_tiles - rt0);
                const int arow = (int)tile.row0, brow = tile.expert * g.N + tile.nb * BN;
                for (int kb = 0; kb < g.num_kb; ++kb) {
                    if (!mbar_wait(bar(S + stage), phase ^ 1u, abort_flag)) {
                        report_error(st, -4, kSiteFp4Producer);
                        ok = false;
                        break;
                    }
                    const uint32_t sb = base + (uint32_t)stage * Cfg::kStage;
                    const uint32_t sf = sb + Cfg::kABytes + Cfg::kBBytes;
                    const uint32_t part = (uint32_t)min(KT, g.k_tiles - kb * KT) * 512u;
                    mbar_arrive_expect_tx(bar(stage), Cfg::kABytes + Cfg::kBBytes + part * (uint32_t)(1 + nrt));
                    tma_load_2d(sb, &tmA, bar(stage), kb * 128, arow, policy_evict_last());
                    tma_load_2d(sb + Cfg::kABytes, &tmB, bar(stage), kb * 128, brow, policy_evict_normal());
                    bulk_load(sf, sfa + (int64_t)kb * KT * 512, part, bar(stage));
                    for (int i = 0; i < nrt; ++i)
                        bulk_load(sf + Cfg::kSfa + (uint32_t)i * KT * 512u, sfb + ((int64_t)i * g.k_tiles + kb * KT) * 512,
                                  part, bar(stage));
                    if (++stage == S) {
                        stage = 0;
                        phase ^= 1u;
                    }
                }
            }
            // Every load must have landed before the CTA ends (see the bf16 kernel).
            volatile int no_abort = 0;
            for (int i = 0; i < S; ++i)
                if (!mbar_wait(bar(i), (i < stage) ? phase : (phase ^ 1u), &no_abort))
                    report_error(st, -4, kSiteFp4Drain);
        }
    } else if (warp == 1) {
        if (lane == 0) {
            const uint32_t idesc = fp4_idesc<NV, BN>();
            const uint32_t tsfa = tmem + (uint32_t)Cfg::kSfCol, tsfb = tsfa + KT * 4;
            int stage = 0, local = 0;
            uint32_t phase = 0;
            bool ok = true;
            for (int t = blockIdx.x; ok && t < total; t += gridDim.x, ++local) {
                const int buf = local & 1;
                if (!mbar_wait(bar(TEMPTY + buf), ((uint32_t)(local >> 1) & 1u) ^ 1u, abort_flag)) {
                    report_error(st, -4, kSiteFp4Mma);
                    break;
                }
                tc_fence_after();
                const uint32_t d = tmem + (uint32_t)(buf * BN);
                for (int kb = 0; kb < g.num_kb; ++kb) {
                    if (!mbar_wait(bar(stage), phase, abort_flag)) {
                        report_error(st, -4, kSiteFp4Mma);
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint32_t sb = base + (uint32_t)stage * Cfg::kStage;
                    const uint32_t sf = sb + Cfg::kABytes + Cfg::kBBytes;
                    const int steps = min(4, (g.K - kb * kFK + 63) / 64);
                    const int parts = min(KT, g.k_tiles - kb * KT);
                    for (int i = 0; i < parts; ++i) {
                        tmem_copy_scales(tsfa + (uint32_t)i * 4, scale_desc(sf + (uint32_t)i * 512u));
#pragma unroll
                        for (int j = 0; j < BN / 128; ++j)
                            tmem_copy_scales(tsfb + (uint32_t)(i * (BN / 128) + j) * 4,
                                             scale_desc(sf + Cfg::kSfa + (uint32_t)(j * KT + i) * 512u));
                    }
                    const uint64_t ad = code_desc(sb), bd = code_desc(sb + Cfg::kABytes);
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        if (k >= steps) break;
                        const int kt = NV ? k : k >> 1;
                        const uint32_t id = NV ? 0u : (uint32_t)(k & 1) * 2u;
                        mma_fp4<NV>(d, ad + (uint64_t)(2 * k), bd + (uint64_t)(2 * k), idesc | (id << 4) | (id << 29),
                                    tsfa + (uint32_t)kt * 4, tsfb + (uint32_t)(kt * (BN / 128)) * 4,
                                    (kb > 0 || k > 0) ? 1u : 0u);
                    }
                    tc_commit(bar(S + stage));
                    if (++stage == S) {
                        stage = 0;
                        phase ^= 1u;
                    }
                }
                if (ok) tc_commit(bar(TFULL + buf));
            }
            tc_commit(bar(DRAIN));
            volatile int no_abort = 0;
            if (!mbar_wait(bar(DRAIN), 0, &no_abort)) report_error(st, -4, kSiteFp4Drain);
        }
    } else {
        const int q = warp & 3;
        const bool vec = ((int64_t)g.N * (int)sizeof(TC)) % 16 == 0;
        const float ga = g.ga ? *g.ga : 1.0f;
        int local = 0;
        for (int t = blockIdx.x; t < total; t += gridDim.x, ++local) {
            const Fp4Tile tile = fp4_tile<BN>(g, prefix, t);
            const int buf = local & 1;
            const bool ready = mbar_wait(bar(TFULL + buf), (uint32_t)(local >> 1) & 1u, abort_flag);
            if (!__all_sync(0xffffffffu, ready)) {
                report_error(st, -4, kSiteFp4Epilogue);
                break;
            }
            tc_fence_after();
            const float alpha = ga * (g.gb ? g.gb[tile.expert] : 1.0f);
            const int row = q * 32 + lane;
            TC* crow = static_cast<TC*>(g.C) + (tile.row0 + row) * (int64_t)g.N;
            const uint32_t taddr = tmem + ((uint32_t)(q * 32) << 16) + (uint32_t)(buf * BN);
#pragma unroll 1
            for (int c = 0; c < BN / 32; ++c) {
                const int col0 = tile.nb * BN + c * 32;
                if (col0 >= g.N) break;
                uint32_t r[32];
                tmem_ld32(taddr + (uint32_t)(c * 32), r);
                tmem_ld_wait();
                if (row >= tile.rows) {
                    // not a row of this expert: left as it was
                } else if (vec && col0 + 32 <= g.N) {
                    if constexpr (sizeof(TC) == 4) {
#pragma unroll
                        for (int j = 0; j < 8; ++j)
                            reinterpret_cast<float4*>(crow + col0)[j] =
                                make_float4(alpha * __uint_as_float(r[4 * j]), alpha * __uint_as_float(r[4 * j + 1]),
                                            alpha * __uint_as_float(r[4 * j + 2]), alpha * __uint_as_float(r[4 * j + 3]));
                    } else {
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            uint32_t u[4];
#pragma unroll
                            for (int h = 0; h < 4; ++h) {
                                const __nv_bfloat162 b2 =
                                    __floats2bfloat162_rn(alpha * __uint_as_float(r[8 * j + 2 * h]),
                                                          alpha * __uint_as_float(r[8 * j + 2 * h + 1]));
                                u[h] = *reinterpret_cast<const uint32_t*>(&b2);
                            }
                            reinterpret_cast<uint4*>(crow + col0)[j] = make_uint4(u[0], u[1], u[2], u[3]);
                        }
                    }
                } else {
#pragma unroll
                    for (int j = 0; j < 32; ++j)
                        if (col0 + j < g.N) crow[col0 + j] = (TC)(alpha * __uint_as_float(r[j]));
                }
                __syncwarp();
            }
            tc_fence_before();
            mbar_arrive(bar(TEMPTY + buf));
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

// ---------------------------------------------------------------- host side

typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                  const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

static EncodeTiledFn fp4_encode_fn() {
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

// The codes of all `count` matrices as one byte matrix: box 128 bytes x box_rows.
// Bytes past the last column read as zeros.
static int code_map(CUtensorMap* map, const Fp4& q, int box_rows) {
    EncodeTiledFn fn = fp4_encode_fn();
    if (!fn) return set_error(-3, "cuTensorMapEncodeTiled entry point unavailable");
    cuuint64_t dims[2] = {(cuuint64_t)((q.cols + 1) / 2), (cuuint64_t)q.rows * (cuuint64_t)q.count};
    cuuint64_t strides[1] = {(cuuint64_t)q.pitch()};
    cuuint32_t box[2] = {128, (cuuint32_t)box_rows};
    cuuint32_t estr[2] = {1, 1};
    CUresult r = fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, q.codes, dims, strides, box, estr,
                    CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                    CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS) return set_error(-3, "cuTensorMapEncodeTiled (4-bit codes) failed");
    return 0;
}

template <bool NV, int BN, typename TC>
static cudaError_t fp4_attr() {
    return cudaFuncSetAttribute(fp4_gemm_kernel<NV, BN, TC>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                Fp4Cfg<NV, BN>::kSmem);
}

int fp4_gemm_init_device() {
    cudaError_t e = fp4_attr<false, 128, float>();
    if (e == cudaSuccess) e = fp4_attr<false, 128, __nv_bfloat16>();
    if (e == cudaSuccess) e = fp4_attr<true, 128, float>();
    if (e == cudaSuccess) e = fp4_attr<true, 128, __nv_bfloat16>();
    if (e != cudaSuccess) return set_cuda_error(e, "cudaFuncSetAttribute(4-bit gemm)");
    return 0;
}

int fp4_gemm_launch(const Fp4& a, const Fp4& b, const int32_t* offsets, const int32_t* counts, void* C, int bf16,
                    int sm_budget, cudaStream_t s, DevStatus* st) {
    DeviceState* ds = device_state();
    if (!ds) return -3;
    if (take_fault(kFaultGemmLaunch)) return set_error(-3, "injected failure: GEMM launch");
    const int cap = (sm_budget <= 0 || sm_budget > ds->sm_count) ? ds->sm_count : sm_budget;
    constexpr int BN = 128;
    Fp4GemmArgs g;
    g.sfa = a.scales;
    g.sfb = b.scales;
    g.ga = a.tensor_scale;
    g.gb = b.tensor_scale;
    g.offsets = offsets;
    g.counts = counts;
    g.C = C;
    g.M = a.rows;
    g.N = (int)b.rows;
    g.K = (int)a.cols;
    g.experts = b.count;
    g.k_tiles = (int)a.k_tiles();
    g.b_row_tiles = (int)b.row_tiles();
    g.num_m = (int)((a.rows + kFM - 1) / kFM);
    g.num_n = (int)((b.rows + BN - 1) / BN);
    g.num_kb = (int)((a.cols + kFK - 1) / kFK);
    const int64_t tiles = (int64_t)g.num_m * g.num_n;  // an upper bound for experts
    if (tiles > 0x7FFFFFFF) return set_error(-5, "4-bit product has more than 2^31 tiles");
    const int grid = (int)(tiles < cap ? tiles : cap);
    CUtensorMap ma, mb;
    int rc = code_map(&ma, a, kFM);
    if (rc) return rc;
    if ((rc = code_map(&mb, b, BN))) return rc;
#define C3_GO(NV_, T_) fp4_gemm_kernel<NV_, BN, T_><<<grid, kFThreads, Fp4Cfg<NV_, BN>::kSmem, s>>>(ma, mb, g, st)
    if (a.nv && bf16) C3_GO(true, __nv_bfloat16);
    else if (a.nv) C3_GO(true, float);
    else if (bf16) C3_GO(false, __nv_bfloat16);
    else C3_GO(false, float);
#undef C3_GO
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return set_cuda_error(e, "4-bit gemm kernel launch");
    count_launch();
    return 0;
}

}  // namespace c3
