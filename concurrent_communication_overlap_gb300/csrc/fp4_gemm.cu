// fp4_gemm.cu -- products of microscaled 4-bit matrices: C = A * B^T with both
// operands in 4-bit codes and block scales, accumulated in fp32 by the
// block-scaled tensor-core instruction (tcgen05.mma, kind mxf4 / mxf4nvf4), and
// the same for the experts of a sparse layer, whose rows of A lie one expert
// after the other.
//
// Two kernels: many rows, two SMs on a tile; few rows, the operands' roles swapped.
// fp4_plan (fp4_plan.h) picks.  Both have the same parts, warp by warp:
//   producer   per stage 256 columns of 4 bits (one 128-byte swizzle row) of A's and
//              B's rows and their scales, all by TMA; scales lie in memory as the
//              tensor cores take them;
//   MMA        four MMAs of 64 columns a stage and accumulator;
//   scales     128 rows x 4 scales at a time from shared memory to TMEM, copied to all
//              four lane quarters.  A warp of its own: copies that the MMA warp itself
//              issues run between its MMAs instead of beside them, however early they
//              are issued (8192 x 28672 x 8192: 886 us against 661, which is what it took
//              without any copies; by way of registers and tcgen05.st: 1012);
//   epilogue   accumulators to registers, times the matrices' fp32 scales, rounded
//              once to the output type, to C.
// Every wait is bounded, as in the bf16 kernel.
#include "ops_device.cuh"
#include "c3_internal.h"

#include <cuda_bf16.h>

namespace c3 {

constexpr int kFM = 128;             // rows of A in a tile
constexpr int kFGroupM = 16;
constexpr int kFSmemLimit = 232448;  // 227 KiB
constexpr int kFHalfSmem = 115712;   // two CTAs on an SM: half of 228 KiB less 1 KiB each
constexpr int kFMaxExperts = 1024;

struct Fp4GemmArgs {
    const float* ga;
    const float* gb;
    const int32_t* offsets;  // experts' rows of A, or NULL
    const int32_t* counts;
    void* C;
    int64_t M;
    int N, K;
    int experts;
    int b_row_tiles;         // scale tiles along one matrix of B
    int num_m, num_n, num_kb;
    int early;               // the next kernel may start beside this one
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
// GROUP: CTAs that share the tile (1 or 2).
template <int GROUP, bool NV>
__device__ __forceinline__ void mma_fp4(uint32_t lead, uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sfa,
                                        uint32_t sfb, uint32_t accumulate) {
#define C3_MMA(G_, KIND_, VEC_)                                                                                      \
    asm volatile("{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %6, 0;\n\tsetp.ne.b32 q, %7, 0;\n\t"                     \
                 "@q tcgen05.mma.cta_group::" G_ ".kind::" KIND_ ".block_scale.scale_vec::" VEC_                      \
                 " [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb),  \
                 "r"(accumulate), "r"(lead)                                                                          \
                 : "memory")
    if constexpr (GROUP == 2 && NV) C3_MMA("2", "mxf4nvf4", "4X");
    else if constexpr (GROUP == 2) C3_MMA("2", "mxf4", "2X");
    else if constexpr (NV) C3_MMA("1", "mxf4nvf4", "4X");
    else C3_MMA("1", "mxf4", "2X");
#undef C3_MMA
}
// 128 rows x 4 scales from shared memory to four TMEM columns, in every lane quarter.
template <int GROUP>
__device__ __forceinline__ void copy_scales(uint32_t lead, uint32_t taddr, uint64_t sdesc) {
#define C3_CP(G_)                                                                                    \
    asm volatile("{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %2, 0;\n\t@q tcgen05.cp.cta_group::" G_       \
                 ".32x128b.warpx4 [%0], %1;\n\t}" ::"r"(taddr), "l"(sdesc), "r"(lead) : "memory")
    if constexpr (GROUP == 2) C3_CP("2");
    else C3_CP("1");
#undef C3_CP
}
// One output tile: its expert, rows and columns.
struct Fp4Tile {
    int expert;       // matrix of B
    int64_t row0;     // first row of A and C
    int rows;         // rows of the tile that are the expert's (or the matrix's)
    int nb;
};

template <int ROWS>
__device__ __forceinline__ Fp4Tile fp4_tile(const Fp4GemmArgs& g, const int* prefix, int t) {
    Fp4Tile r;
    if (g.offsets == nullptr) {
        const int per = kFGroupM * g.num_n, grp = t / per, first = grp * kFGroupM;
        const int gm = min(g.num_m - first, kFGroupM), in = t - grp * per;
        const int mb = first + in % gm;
        r.expert = 0;
        r.row0 = (int64_t)mb * ROWS;
        r.rows = (int)min((int64_t)ROWS, g.M - r.row0);
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
    r.row0 = (int64_t)g.offsets[lo] + (int64_t)mb * ROWS;
    r.rows = min(ROWS, g.counts[lo] - mb * ROWS);
    return r;
}

// Row tiles before each expert, by one warp.  An expert whose rows do not lie in
// A, or do not start at a whole scale tile, has none: nothing out of range is touched.
template <int ROWS>
__device__ __forceinline__ void expert_tiles(const Fp4GemmArgs& g, int* prefix, int lane) {
    const int64_t limit = (int64_t)g.num_m + g.experts;
    int run = 0;
    for (int e0 = 0; e0 < g.experts; e0 += 32) {
        const int e = e0 + lane;
        int mt = 0;
        if (e < g.experts) {
            const int64_t off = g.offsets[e], c = g.counts[e];
            if (off >= 0 && c > 0 && off % kTileRows == 0 && off + c <= g.M) mt = (int)((c + ROWS - 1) / ROWS);
        }
        int incl = mt;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += v;
        }
        if (e < g.experts) prefix[e + 1] = tiles_up_to(run, incl, limit);
        run = tiles_up_to(run, __shfl_sync(0xffffffffu, incl, 31), limit);
    }
    if (lane == 0) prefix[0] = 0;
}

// ---------------------------------------------------------------- two SMs on one tile
//
// The form for many rows.  A cluster of two CTAs shares one tile (cta_group::2):
// each CTA brings in half of A's rows, half of B's and all of the tile's scales of
// B, and holds the accumulators of its own rows.  A 4-bit MMA at full rate eats
// its operands four times as fast as a bf16 one, so what an SM has to take in per
// MMA cycle decides: 128 x 128 tiles on one SM need 126 bytes a cycle, 256 x 192
// on two 78, 512 x 192 or 256 x 384 on two 61.  Accumulators are 192 columns,
// because a tile's scales have to begin at an even TMEM column (a multiple of 64
// rows of B) and 2 x 256 columns would leave TMEM no room for scales; there are
// two: one above the other (512 rows), side by side (384 columns), or in turn for
// tiles of 256 x 192, whose read-out then hides behind the next tile.
//
// The leader (rank 0) issues every MMA.  Its full barriers count the bytes of
// both CTAs' loads; a commit frees a stage, or publishes a tile, in both.  The
// epilogue's eight warps in each CTA read 32 x 32 pieces out of TMEM one ahead,
// turn them through 2 KB of shared memory each, and write whole 64-byte pieces
// of rows.
//
// 8192 x 28672 x 8192 MX takes 576 to 592 us, 6.5 to 6.7 PFLOP/s.  Copies with a part of the
// work left out put what bounds it side by side: loads alone 463, MMAs alone about 380, and
// the copies of scales another 70 beside them.  NV, with twice the scales, takes 8 to 15%
// more, 4096 x 7680 x 8192 101 us (MX) and 104.
//
// The bf16 epilogues of two accumulators spill 20 to 28 bytes a thread, once a tile.
constexpr int kPThreads = 352;  // producer, MMA, scales, and the epilogue's eight warps
constexpr int kPEpiWarps = 8;

template <bool NV, int MSUB, int NSUB, typename TC>
struct Fp4PairCfg {
    static constexpr int kKT = NV ? 4 : 2;
    static constexpr int kRows = MSUB * 256, kCols = NSUB * kPN;
    static constexpr int kBN2 = kPN / 2;
    static constexpr int kSfbTiles = NSUB + 1;  // scale tiles that the columns lie in
    static constexpr int kSub = MSUB * NSUB;    // accumulators of a tile
    static constexpr uint32_t kABytes = MSUB * kFM * 128;
    static constexpr uint32_t kBBytes = NSUB * kBN2 * 128;
    static constexpr uint32_t kSfa = MSUB * kKT * 512;
    static constexpr uint32_t kSfb = kSfbTiles * kKT * 512;
    static constexpr uint32_t kStage = kABytes + kBBytes + kSfa + kSfb;
    static constexpr uint32_t kStaging = kPEpiWarps * 2048;
    // 512 rows: one matrix only
    static constexpr int kExtra = 1024 + 512 + (MSUB == 1 ? 4 * (kFMaxExperts + 1) : 0) + (int)kStaging;
    static constexpr int kFit = (kFSmemLimit - kExtra) / (int)kStage;
    static constexpr int kStages = kFit > 8 ? 8 : kFit;
    static constexpr int kSmem = kStages * (int)kStage + kExtra;
    static constexpr int kAccBufs = kSub == 2 ? 1 : 2;
    static constexpr int kSetCols = (MSUB + kSfbTiles) * 4;   // TMEM columns of one k tile's scales
    static_assert(kStage % 1024 == 0, "the codes need 1024-byte alignment");
    static constexpr int kSets = NV ? 2 : 4;          // stages whose scales TMEM holds
    static_assert(kStages >= kSets && 2 * kPN + kSets * kKT * kSetCols <= 512, "pair configuration");
};

// tmA, tmB: codes; tmSA, tmSB: scales as [row tiles][k tiles * 64] 64-bit words.
template <bool NV, int MSUB, int NSUB, typename TC>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kPThreads, 1)
    fp4_gemm_pair_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                         const __grid_constant__ CUtensorMap tmSA, const __grid_constant__ CUtensorMap tmSB,
                         Fp4GemmArgs g, DevStatus* st) {
    using Cfg = Fp4PairCfg<NV, MSUB, NSUB, TC>;
    constexpr int S = Cfg::kStages, KT = Cfg::kKT, NB = Cfg::kAccBufs;
    constexpr int kRows = Cfg::kRows;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    const uint32_t raw = smem_addr(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    uint8_t* gbase = smem_raw + (base - raw);
    const uint32_t staging = base + S * Cfg::kStage;
    uint64_t* bars = reinterpret_cast<uint64_t*>(gbase + S * Cfg::kStage + Cfg::kStaging);
    // stage full [0, S), empty [S, 2S), its scales in TMEM too [2S, 3S), accumulator full 3S..,
    // empty 3S+2.., drain 3S+4
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 3 * S + 5);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
    int* prefix = reinterpret_cast<int*>(gbase + S * Cfg::kStage + Cfg::kStaging + 512);
    auto bar = [&](int i) { return smem_addr(&bars[i]); };
    const int SREADY = 2 * S, TFULL = 3 * S, TEMPTY = 3 * S + 2, DRAIN = 3 * S + 4;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = cluster_rank();

    if (threadIdx.x == 0) {
        *abort_flag = 0;
        for (int i = 0; i < S; ++i) {
            mbar_init(bar(i), 1);
            mbar_init(bar(S + i), 1);
            mbar_init(bar(SREADY + i), 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(bar(TFULL + b), 1);
            mbar_init(bar(TEMPTY + b), 2 * kPEpiWarps);
        }
        mbar_init(bar(DRAIN), 1);
        fence_barrier_init();
        prefetch_tensormap(&tmA);
        prefetch_tensormap(&tmB);
        prefetch_tensormap(&tmSA);
        prefetch_tensormap(&tmSB);
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_addr(tmem_slot))
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    }
    if (g.early) chain_next();
    chain_ready();
    if (MSUB == 1 && g.offsets && warp == 3) expert_tiles<kRows>(g, prefix, lane);
    tc_fence_before();
    __syncthreads();
    cluster_sync_all();  // both CTAs' barriers are ready before either signals the other's
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    const int total = MSUB == 1 && g.offsets ? prefix[g.experts] * g.num_n : g.num_m * g.num_n;
    const int first = blockIdx.x >> 1, step = gridDim.x >> 1;

    if (warp == 0) {
        if (lane == 0) {
            const uint64_t pol_a = policy_evict_last(), pol_b = policy_evict_normal();
            int stage = 0;
            uint32_t phase = 0;
            bool ok = true;
            for (int t = first; ok && t < total; t += step) {
                const Fp4Tile tile = fp4_tile<kRows>(g, prefix, t);
                const int arow = (int)tile.row0 + (int)rank * (kRows / 2);
                const int n0 = tile.nb * Cfg::kCols;
                const int brow = tile.expert * g.N + n0 + (int)rank * Cfg::kBN2;
                const int sbrow = tile.expert * g.b_row_tiles + n0 / 128;
                for (int kb = 0; kb < g.num_kb; ++kb) {
                    if (!mbar_wait_cluster(bar(S + stage), phase ^ 1u, abort_flag)) {
                        report_error(st, -4, kSiteFp4Producer);
                        ok = false;
                        break;
                    }
                    const uint32_t sb = base + (uint32_t)stage * Cfg::kStage;
                    const uint32_t full = leader_addr(bar(stage));
                    const uint32_t sf = sb + Cfg::kABytes + Cfg::kBBytes;
                    if (rank == 0) mbar_arrive_expect_tx(bar(stage), 2 * Cfg::kStage);
                    tma_load_2d_pair(sf, &tmSA, full, kb * KT * 64, arow / 128, pol_a);
                    tma_load_2d_pair(sf + Cfg::kSfa, &tmSB, full, kb * KT * 64, sbrow, pol_b);
                    tma_load_2d_pair(sb, &tmA, full, kb * 128, arow, pol_a);
#pragma unroll
                    for (int j = 0; j < NSUB; ++j)
                        tma_load_2d_pair(sb + Cfg::kABytes + (uint32_t)j * Cfg::kBN2 * 128u, &tmB, full, kb * 128, brow + j * kPN, pol_b);
                    if (++stage == S) {
                        stage = 0;
                        phase ^= 1u;
                    }
                }
            }
            // The pair's loads have all landed once every stage that was filled has been
            // freed (its MMAs follow its loads): wait for that before the CTA may end.
            // After a wait gave up, the leader's full barriers tell it instead.
            volatile int no_abort = 0;
            for (int i = 0; (ok || rank == 0) && i < S; ++i)
                if (!mbar_wait_cluster(bar(ok ? S + i : i), (i < stage) ? phase : (phase ^ 1u), &no_abort))
                    report_error(st, -4, kSiteFp4Drain);
        }
    } else if (warp == 1) {
        if (rank == 0) {
            const uint32_t lead = elect_lane();
            const uint32_t idesc = (1u << 7) | (1u << 10) | ((uint32_t)(kPN >> 3) << 17) | (NV ? 0u : 1u << 23) | (2u << 27);
            const uint64_t code0 = code_desc(base);
            int stage = 0, local = 0, set = 0;
            uint32_t phase = 0;
            bool ok = true;
            for (int t = first; ok && t < total; t += step, ++local) {
                // 192 columns: odd tiles begin at row 64 of a scale tile, two TMEM columns on
                const uint32_t shift = NSUB == 2 ? 0u : (uint32_t)(fp4_tile<kRows>(g, prefix, t).nb & 1) * 2u;
                const int buf = local % NB;
                if (!mbar_wait_cluster(bar(TEMPTY + buf), ((uint32_t)(local / NB) & 1u) ^ 1u, abort_flag)) {
                    report_error(st, -4, kSiteFp4Mma);
                    break;
                }
                tc_fence_after();
                const uint32_t d = tmem + (uint32_t)(buf * kPN);
                for (int kb = 0; kb < g.num_kb; ++kb) {
                    if (!mbar_wait_cluster(bar(SREADY + stage), phase, abort_flag)) {
                        report_error(st, -4, kSiteFp4Mma);
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint64_t ad = code0 + (uint64_t)((uint32_t)stage * (Cfg::kStage >> 4));
                    const uint64_t bd = ad + (Cfg::kABytes >> 4);
                    const int steps = min(4, (g.K - kb * kFK + 63) / 64);
                    const uint32_t tsf0 = tmem + 2u * kPN + (uint32_t)(set * KT * Cfg::kSetCols);
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const uint32_t go = k < steps ? lead : 0u;
                        const uint32_t tsf = tsf0 + (uint32_t)((NV ? k : k >> 1) * Cfg::kSetCols);
                        const uint32_t id = NV ? 0u : (uint32_t)(k & 1) * 2u;
#pragma unroll
                        for (int i = 0; i < MSUB; ++i)
#pragma unroll
                            for (int j = 0; j < NSUB; ++j)
                                mma_fp4<2, NV>(go, d + (uint32_t)((i + j) * kPN), ad + (uint64_t)(i * (kFM * 128 >> 4) + 2 * k),
                                               bd + (uint64_t)(j * (Cfg::kBN2 * 128 >> 4) + 2 * k), idesc | (id << 4) | (id << 29),
                                               tsf + (uint32_t)i * 4, tsf + (uint32_t)(MSUB * 4 + j * (kPN / 32)) + shift,
                                               k > 0 ? 1u : (uint32_t)(kb > 0));
                    }
                    commit_pair(lead, bar(S + stage));
                    set = set + 1 == Cfg::kSets ? 0 : set + 1;
                    if (++stage == S) {
                        stage = 0;
                        phase ^= 1u;
                    }
                }
                if (ok) commit_pair(lead, bar(TFULL + buf));
            }
            // no MMA may still run when TMEM is freed
            commit_local<2>(lead, bar(DRAIN));
            volatile int no_abort = 0;
            if (!mbar_wait(bar(DRAIN), 0, &no_abort)) report_error(st, -4, kSiteFp4Drain);
        }
    } else if (warp == 2) {
        if (rank == 0) {
            // ---------------- scales from shared memory to TMEM, in both CTAs
            const uint32_t lead = elect_lane();
            const uint64_t scale0 = scale_desc(base + Cfg::kABytes + Cfg::kBBytes);
            int stage = 0, set = 0, old_stage = 0;  // old_stage: the stage whose MMAs used this set last
            uint32_t phase = 0, old_phase = 0;
            int done = 0;
            bool ok = true;
            for (int t = first; ok && t < total; t += step)
                for (int kb = 0; kb < g.num_kb; ++kb) {
                    ok = mbar_wait_cluster(bar(stage), phase, abort_flag);
                    if (ok && done >= Cfg::kSets) ok = mbar_wait_cluster(bar(S + old_stage), old_phase, abort_flag);
                    if (!ok) {
                        report_error(st, -4, kSiteFp4Scales);
                        break;
                    }
                    tc_fence_after();
                    const uint64_t from = scale0 + (uint64_t)((uint32_t)stage * (Cfg::kStage >> 4));
                    const uint32_t to = tmem + 2u * kPN + (uint32_t)(set * KT * Cfg::kSetCols);
#pragma unroll
                    for (int kt = 0; kt < KT; ++kt)
#pragma unroll
                        for (int i = 0; i < MSUB + Cfg::kSfbTiles; ++i)
                            copy_scales<2>(lead, to + (uint32_t)(kt * Cfg::kSetCols + i * 4),
                                                  from + (uint64_t)((i * KT + kt) * (512 >> 4)));
                    commit_local<2>(lead, bar(SREADY + stage));
                    if (++done > Cfg::kSets && ++old_stage == S) {
                        old_stage = 0;
                        old_phase ^= 1u;
                    }
                    set = set + 1 == Cfg::kSets ? 0 : set + 1;
                    if (++stage == S) {
                        stage = 0;
                        phase ^= 1u;
                    }
                }
        }
    } else {
        const int q = warp & 3, half = (warp - 3) >> 2;
        const uint32_t blk = staging + (uint32_t)(warp - 3) * 2048u;
        // bytes that every row of C is aligned to, 16 at most
        const int row_bytes = g.N * (int)sizeof(TC), width = min(row_bytes & -row_bytes, 16);
        const float ga = g.ga ? *g.ga : 1.0f;
        int local = 0;
        for (int t = first; t < total; t += step, ++local) {
            const Fp4Tile tile = fp4_tile<kRows>(g, prefix, t);
            const int buf = local % NB;
            const bool ready = mbar_wait_cluster(bar(TFULL + buf), (uint32_t)(local / NB) & 1u, abort_flag);
            if (!__all_sync(0xffffffffu, ready)) {
                report_error(st, -4, kSiteFp4Epilogue);
                break;
            }
            tc_fence_after();
            const float alpha = ga * (g.gb ? g.gb[tile.expert] : 1.0f);
            // This warp's columns: all of one accumulator's where there are two, else half.
            constexpr int kPieces = kPN / 32 / (Cfg::kSub == 2 ? 1 : 2);
            constexpr int kWords = 8 * sizeof(TC);
            constexpr int kBatch = kPieces * kWords <= 96 ? kPieces : 96 / kWords;
            const int sub = Cfg::kSub == 2 ? half : 0;
            const int r0 = (int)rank * (kRows / 2) + (MSUB == 2 ? sub * 128 : 0) + q * 32;  // the warp's first row in the tile
            const int c0 = Cfg::kSub == 2 ? 0 : half * kPieces * 32;
            const int rows = tile.rows - r0, col0 = tile.nb * Cfg::kCols + (NSUB == 2 ? sub * kPN : 0) + c0;
            const uint32_t taddr = tmem + ((uint32_t)(q * 32) << 16) + (uint32_t)((buf + sub) * kPN + c0);
            // Read out and rounded first: the accumulator is free again before anything is stored.
#pragma unroll
            for (int b = 0; b < kPieces; b += kBatch) {
                uint32_t v[kBatch * kWords];
#pragma unroll
                for (int i = 0; i < kBatch; ++i) {
                    uint32_t r[32];
                    tmem_ld32(taddr + (uint32_t)((b + i) * 32), r);
                    tmem_ld_wait();
                    if constexpr (sizeof(TC) == 2) {
#pragma unroll
                        for (int j = 0; j < 16; ++j) {
                            const __nv_bfloat162 h = __floats2bfloat162_rn(alpha * __uint_as_float(r[2 * j]),
                                                                           alpha * __uint_as_float(r[2 * j + 1]));
                            v[i * kWords + j] = *reinterpret_cast<const uint32_t*>(&h);
                        }
                    } else {
#pragma unroll
                        for (int j = 0; j < 32; ++j) v[i * kWords + j] = __float_as_uint(alpha * __uint_as_float(r[j]));
                    }
                }
                if (b + kBatch >= kPieces) {
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive_cluster(leader_addr(bar(TEMPTY + buf)));
                }
#pragma unroll
                for (int i = 0; i < kBatch; ++i)
                    store_piece<TC>(&v[i * kWords], blk, lane, width, static_cast<TC*>(g.C), tile.row0 + r0, rows,
                                    col0 + (b + i) * 32, g.N, g.N);
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    cluster_sync_all();  // nothing of this CTA's is signalled or read by the other any more
    if (warp == 1) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
    }
}

// ---------------------------------------------------------------- few rows
//
// The form for few rows of A (a serving step's tokens, an expert's handful): the
// weights' bytes decide, so the roles are swapped.  B's rows (the output's
// columns) take the MMA's 128 rows and A's rows its columns, NT of them: nothing
// of a tile is padding that has to be brought in, and a warp stores 32
// neighbours of one row of C.
//
// Two CTAs fit an SM: one's start and end hide behind the other's stream (64
// experts of 2048 x 4096 with 192 rows: 45 us, 5.8 TB/s of weights).  Where
// there are fewer tiles than CTAs to fill the machine, a cluster of `split` CTAs
// takes a tile at a time, each a part of K; their fp32 parts meet in shared memory, each
// CTA adding up its share of A's rows in the order of the ranks.  13 x 8200 x 8072
// takes 12.3 us in a chain of calls, where its bytes need 5.5; the rest is set-up, the
// first loads' latency and the cluster's two meetings.
constexpr int kRThreads = 256;

template <bool NV, int NT>
struct Fp4RowsCfg {
    static constexpr int kKT = NV ? 4 : 2;
    static constexpr uint32_t kWBytes = 128 * 128;
    static constexpr uint32_t kTBytes = NT * 128;
    static constexpr uint32_t kSf = kKT * 512;
    static constexpr uint32_t kStage = kWBytes + kTBytes + 2 * kSf;
    static constexpr int kExtra = 1024 + 512 + (NT == 64 ? 4 * (kFMaxExperts + 1) : 0);  // experts: 64 rows
    static constexpr int kStages = (kFHalfSmem - kExtra) / (int)kStage;
    static constexpr int kSmem = kStages * (int)kStage + kExtra;
    static constexpr int kAccBufs = NT == 128 ? 1 : 2;
    static constexpr int kSetCols = 8;
    // Stages whose scales TMEM holds: no more than the ring's, since a set's last use is
    // told by that stage's empty barrier, which must not have come round twice.
    static constexpr int kSets = kStages < 4 ? kStages : 4;
    static_assert(kStage % 1024 == 0 && kStages >= 3 && kSets * kKT * kSetCols <= 128, "few-rows configuration");
    static_assert(kStages * kStage >= NT * 512, "the parts meet in the ring");
};

template <bool NV, int NT, typename TC>
__global__ void __launch_bounds__(kRThreads, 2)
    fp4_gemm_rows_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                         const __grid_constant__ CUtensorMap tmSA, const __grid_constant__ CUtensorMap tmSB,
                         Fp4GemmArgs g, int split, DevStatus* st) {
    using Cfg = Fp4RowsCfg<NV, NT>;
    constexpr int S = Cfg::kStages, KT = Cfg::kKT, NB = Cfg::kAccBufs;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    const uint32_t raw = smem_addr(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    uint8_t* gbase = smem_raw + (base - raw);
    uint64_t* bars = reinterpret_cast<uint64_t*>(gbase + S * Cfg::kStage);
    // stage full [0, S), empty [S, 2S), its scales in TMEM [2S, 3S), accumulator full 3S.., empty 3S+2.., drain 3S+4
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 3 * S + 5);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
    int* prefix = reinterpret_cast<int*>(gbase + S * Cfg::kStage + 512);
    auto bar = [&](int i) { return smem_addr(&bars[i]); };
    const int SREADY = 2 * S, TFULL = 3 * S, TEMPTY = 3 * S + 2, DRAIN = 3 * S + 4;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        *abort_flag = 0;
        for (int i = 0; i < S; ++i) {
            mbar_init(bar(i), 1);
            mbar_init(bar(S + i), 1);
            mbar_init(bar(SREADY + i), 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(bar(TFULL + b), 1);
            mbar_init(bar(TEMPTY + b), 4);
        }
        mbar_init(bar(DRAIN), 1);
        fence_barrier_init();
        prefetch_tensormap(&tmA);
        prefetch_tensormap(&tmB);
        prefetch_tensormap(&tmSA);
        prefetch_tensormap(&tmSB);
    }
    if (warp == 1) {
        tmem_alloc(smem_addr(tmem_slot), 256);
        tmem_relinquish();
    }
    if (g.early) chain_next();
    chain_ready();
    if (NT == 64 && g.offsets && warp == 2) expert_tiles<NT>(g, prefix, lane);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    const int total = NT == 64 && g.offsets ? prefix[g.experts] * g.num_n : g.num_m * g.num_n;
    const uint32_t rank = split > 1 ? cluster_rank() : 0u;
    const int first = split > 1 ? blockIdx.x / split : blockIdx.x;
    const int step = gridDim.x / split;
    const int kb0 = (int)((int64_t)g.num_kb * (int)rank / split), kb1 = (int)((int64_t)g.num_kb * ((int)rank + 1) / split);

    // The roles' places in the ring; a warp has one role.  A cluster does one tile after
    // the other, a CTA by itself all of its tiles in one go.
    int stage = 0, set = 0, old_stage = 0, done = 0;
    uint32_t phase = 0, old_phase = 0, turn = 0;
    bool ok = true;
    for (int t0 = first;; t0 += step, turn ^= 1u) {
        const int end = split > 1 ? min(t0 + 1, total) : total;
        if (warp == 0) {
            if (lane == 0) {
                // weights that one tile alone reads do not stay in L2
                const uint64_t pol_w = g.num_m > 1 ? policy_evict_normal() : policy_evict_first(), pol_t = policy_evict_last();
                for (int t = t0; ok && t < end; t += step) {
                    const Fp4Tile tile = fp4_tile<NT>(g, prefix, t);
                    const int trow = (int)tile.row0, wrow = tile.expert * g.N + tile.nb * 128;
                    const int swrow = tile.expert * g.b_row_tiles + tile.nb;
                    for (int kb = kb0; kb < kb1; ++kb) {
                        if (!mbar_wait(bar(S + stage), phase ^ 1u, abort_flag)) {
                            report_error(st, -4, kSiteFp4Producer);
                            ok = false;
                            break;
                        }
                        const uint32_t sb = base + (uint32_t)stage * Cfg::kStage;
                        const uint32_t sf = sb + Cfg::kWBytes + Cfg::kTBytes;
                        mbar_arrive_expect_tx(bar(stage), Cfg::kStage);
                        tma_load_2d(sb, &tmB, bar(stage), kb * 128, wrow, pol_w);
                        tma_load_2d(sb + Cfg::kWBytes, &tmA, bar(stage), kb * 128, trow, pol_t);
                        tma_load_2d(sf, &tmSB, bar(stage), kb * KT * 64, swrow, pol_w);
                        tma_load_2d(sf + Cfg::kSf, &tmSA, bar(stage), kb * KT * 64, trow / 128, pol_t);
                        if (++stage == S) {
                            stage = 0;
                            phase ^= 1u;
                        }
                    }
                }
            }
        } else if (warp == 1) {
            const uint32_t lead = elect_lane();
            const uint32_t idesc = (1u << 7) | (1u << 10) | ((uint32_t)(NT >> 3) << 17) | (NV ? 0u : 1u << 23) | (1u << 27);
            const uint64_t code0 = code_desc(base);
            int local = 0;
            for (int t = t0; ok && t < end; t += step, ++local) {
                const uint32_t shift = (uint32_t)(fp4_tile<NT>(g, prefix, t).row0 % 128) / 32;  // 0 or 2
                const int buf = local % NB;
                if (!mbar_wait(bar(TEMPTY + buf), ((uint32_t)(local / NB) & 1u) ^ 1u, abort_flag)) {
                    report_error(st, -4, kSiteFp4Mma);
                    ok = false;
                    break;
                }
                tc_fence_after();
                const uint32_t d = tmem + (uint32_t)(buf * NT);
                for (int kb = kb0; kb < kb1; ++kb) {
                    if (!mbar_wait(bar(SREADY + stage), phase, abort_flag)) {
                        report_error(st, -4, kSiteFp4Mma);
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint64_t wd = code0 + (uint64_t)((uint32_t)stage * (Cfg::kStage >> 4));
                    const uint64_t td = wd + (Cfg::kWBytes >> 4);
                    const int steps = min(4, (g.K - kb * kFK + 63) / 64);
                    const uint32_t tsf0 = tmem + 128u + (uint32_t)(set * KT * Cfg::kSetCols);
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const uint32_t tsf = tsf0 + (uint32_t)((NV ? k : k >> 1) * Cfg::kSetCols);
                        const uint32_t id = NV ? 0u : (uint32_t)(k & 1) * 2u;
                        mma_fp4<1, NV>(k < steps ? lead : 0u, d, wd + (uint64_t)(2 * k), td + (uint64_t)(2 * k),
                                       idesc | (id << 4) | (id << 29), tsf, tsf + 4u + shift, k > 0 ? 1u : (uint32_t)(kb > kb0));
                    }
                    commit_local<1>(lead, bar(S + stage));
                    set = set + 1 == Cfg::kSets ? 0 : set + 1;
                    if (++stage == S) {
                        stage = 0;
                        phase ^= 1u;
                    }
                }
                if (ok) commit_local<1>(lead, bar(TFULL + buf));
            }
        } else if (warp == 2) {
            // ---------------- scales from shared memory to TMEM (see the pair kernel)
            const uint32_t lead = elect_lane();
            const uint64_t scale0 = scale_desc(base + Cfg::kWBytes + Cfg::kTBytes);
            for (int t = t0; ok && t < end; t += step)
                for (int kb = kb0; kb < kb1; ++kb) {
                    ok = mbar_wait(bar(stage), phase, abort_flag);
                    if (ok && done >= Cfg::kSets) ok = mbar_wait(bar(S + old_stage), old_phase, abort_flag);
                    if (!ok) {
                        report_error(st, -4, kSiteFp4Scales);
                        break;
                    }
                    tc_fence_after();
                    const uint64_t from = scale0 + (uint64_t)((uint32_t)stage * (Cfg::kStage >> 4));
                    const uint32_t to = tmem + 128u + (uint32_t)(set * KT * Cfg::kSetCols);
#pragma unroll
                    for (int kt = 0; kt < KT; ++kt)
#pragma unroll
                        for (int i = 0; i < 2; ++i)
                            copy_scales<1>(lead, to + (uint32_t)(kt * Cfg::kSetCols + i * 4),
                                           from + (uint64_t)((i * KT + kt) * (512 >> 4)));
                    commit_local<1>(lead, bar(SREADY + stage));
                    if (++done > Cfg::kSets && ++old_stage == S) {
                        old_stage = 0;
                        old_phase ^= 1u;
                    }
                    set = set + 1 == Cfg::kSets ? 0 : set + 1;
                    if (++stage == S) {
                        stage = 0;
                        phase ^= 1u;
                    }
                }
        } else if (warp >= 4 && split == 1) {
            const int q = warp & 3;
            const float ga = g.ga ? *g.ga : 1.0f;
            int local = 0;
            for (int t = t0; t < end; t += step, ++local) {
                const Fp4Tile tile = fp4_tile<NT>(g, prefix, t);
                const int buf = local % NB;
                const bool go = mbar_wait(bar(TFULL + buf), (uint32_t)(local / NB) & 1u, abort_flag);
                if (!__all_sync(0xffffffffu, go)) {
                    report_error(st, -4, kSiteFp4Epilogue);
                    break;
                }
                tc_fence_after();
                const float alpha = ga * (g.gb ? g.gb[tile.expert] : 1.0f);
                const int n = tile.nb * 128 + q * 32 + lane;
                TC* c = static_cast<TC*>(g.C) + tile.row0 * (int64_t)g.N + n;
                const uint32_t taddr = tmem + ((uint32_t)(q * 32) << 16) + (uint32_t)(buf * NT);
#pragma unroll 1
                for (int j0 = 0; j0 < NT && j0 < tile.rows; j0 += 32) {
                    uint32_t r[32];
                    tmem_ld32(taddr + (uint32_t)j0, r);
                    tmem_ld_wait();
#pragma unroll
                    for (int j = 0; j < 32; ++j)
                        if (j0 + j < tile.rows && n < g.N) c[(int64_t)(j0 + j) * g.N] = (TC)(alpha * __uint_as_float(r[j]));
                    __syncwarp();
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(TEMPTY + buf));
            }
        }
        __syncwarp();
        if (split > 1) {
            // The parts of a tile: share s of A's rows (NT / split of them) is added up by
            // rank s, from the parts that every rank writes into its ring, which is idle:
            // all MMAs and loads of the cluster are done at the first barrier.
            // Four of A's rows make a piece: 16 bytes a lane, lane after lane, so that a warp
            // sends 512 bytes in one run (a lane's pieces together, 64 bytes apart from the next
            // lane's, took 22 us for 100 x 4096 x 4096 over 8 CTAs instead of 13).
            const int share = NT / split, shift = __ffs(share) - 1;  // powers of two, 4 at least
            const bool live = t0 < total;
            const int q = warp & 3;
            bool go = true;
            if (warp >= 4 && live) {
                go = mbar_wait(bar(TFULL), turn, abort_flag);
                go = __all_sync(0xffffffffu, go);
                if (!go) report_error(st, -4, kSiteFp4Epilogue);
            }
            cluster_sync_all();
            if (warp >= 4 && live && go) {
                tc_fence_after();
                const uint32_t taddr = tmem + ((uint32_t)(q * 32) << 16);
                const uint32_t mine = base + (uint32_t)(rank * (share / 4) * 128 + q * 32 + lane) * 16u;
#pragma unroll 1
                for (int j0 = 0; j0 < NT; j0 += 32) {
                    uint32_t r[32];
                    tmem_ld32(taddr + (uint32_t)j0, r);
                    tmem_ld_wait();
#pragma unroll
                    for (int j = 0; j < 32; j += 4) {
                        const int to = (j0 + j) >> shift, piece = ((j0 + j) & (share - 1)) >> 2;
                        asm volatile("st.shared::cluster.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(
                                         peer_addr(mine + (uint32_t)piece * 2048u, (uint32_t)to)),
                                     "r"(r[j]), "r"(r[j + 1]), "r"(r[j + 2]), "r"(r[j + 3])
                                     : "memory");
                    }
                }
                tc_fence_before();
            }
            cluster_sync_all();
            if (warp >= 4 && live && go) {
                const Fp4Tile tile = fp4_tile<NT>(g, prefix, t0);
                const float alpha = (g.ga ? *g.ga : 1.0f) * (g.gb ? g.gb[tile.expert] : 1.0f);
                const int n = tile.nb * 128 + q * 32 + lane;
                const float4* part = reinterpret_cast<const float4*>(gbase) + q * 32 + lane;
                const int mine = min(share, tile.rows - (int)rank * share);
                TC* c = static_cast<TC*>(g.C) + (tile.row0 + (int)rank * share) * (int64_t)g.N + n;
#pragma unroll 2
                for (int at = 0; at < mine; at += 4) {
                    float4 sum = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
                    for (int s = 0; s < 8; ++s)
                        if (s < split) {
                            const float4 v = part[(s * (share / 4) + (at >> 2)) * 128];
                            sum.x += v.x, sum.y += v.y, sum.z += v.z, sum.w += v.w;
                        }
                    const float out[4] = {sum.x, sum.y, sum.z, sum.w};
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if (n < g.N && at + i < mine) c[(int64_t)(at + i) * g.N] = (TC)(alpha * out[i]);
                }
            }
        }
        if (split == 1 || t0 + step >= total) break;
        // the next tile's loads (the other proxy) follow these reads of the parts, its MMAs those of TMEM
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        tc_fence_before();
        __syncthreads();
        tc_fence_after();
    }
    if (warp == 0 && lane == 0) {
        // Every load must have landed before the CTA ends.
        volatile int no_abort = 0;
        for (int i = 0; i < S; ++i)
            if (!mbar_wait(bar(i), (i < stage) ? phase : (phase ^ 1u), &no_abort))
                report_error(st, -4, kSiteFp4Drain);
    } else if (warp == 1) {
        // no MMA may still run when TMEM is freed
        commit_local<1>(elect_lane(), bar(DRAIN));
        volatile int no_abort = 0;
        if (!mbar_wait(bar(DRAIN), 0, &no_abort)) report_error(st, -4, kSiteFp4Drain);
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, 256);
    }
}

// ---------------------------------------------------------------- host side

// The codes of all `count` matrices as one byte matrix: box 128 bytes x box_rows.
// Bytes past the last column read as zeros.
static int code_map(CUtensorMap* map, const Fp4& q, int box_rows) {
    EncodeTiledFn fn = tensor_map_encode();
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

// The scales of all matrices as rows of 64-bit words, one row tile a row; what lies past the last k tile reads as zeros.
static int scale_map(CUtensorMap* map, const Fp4& q, int box_rows) {
    EncodeTiledFn fn = tensor_map_encode();
    if (!fn) return set_error(-3, "cuTensorMapEncodeTiled entry point unavailable");
    cuuint64_t dims[2] = {(cuuint64_t)q.k_tiles() * 64, (cuuint64_t)q.row_tiles() * (cuuint64_t)q.count};
    cuuint64_t strides[1] = {(cuuint64_t)q.k_tiles() * 512};
    cuuint32_t box[2] = {q.nv ? 256u : 128u, (cuuint32_t)box_rows};
    cuuint32_t estr[2] = {1, 1};
    CUresult r = fn(map, CU_TENSOR_MAP_DATA_TYPE_INT64, 2, q.scales, dims, strides, box, estr,
                    CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                    CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS) return set_error(-3, "cuTensorMapEncodeTiled (4-bit scales) failed");
    return 0;
}

template <typename K>
static cudaError_t allow_smem(K kernel, int bytes) {
    return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
}

template <bool NV, typename TC>
static cudaError_t fp4_attr() {
    cudaError_t e = allow_smem(fp4_gemm_pair_kernel<NV, 1, 1, TC>, Fp4PairCfg<NV, 1, 1, TC>::kSmem);
    if (e == cudaSuccess) e = allow_smem(fp4_gemm_pair_kernel<NV, 2, 1, TC>, Fp4PairCfg<NV, 2, 1, TC>::kSmem);
    if (e == cudaSuccess) e = allow_smem(fp4_gemm_pair_kernel<NV, 1, 2, TC>, Fp4PairCfg<NV, 1, 2, TC>::kSmem);
    if (e == cudaSuccess) e = allow_smem(fp4_gemm_rows_kernel<NV, 32, TC>, Fp4RowsCfg<NV, 32>::kSmem);
    if (e == cudaSuccess) e = allow_smem(fp4_gemm_rows_kernel<NV, 64, TC>, Fp4RowsCfg<NV, 64>::kSmem);
    if (e == cudaSuccess) e = allow_smem(fp4_gemm_rows_kernel<NV, 128, TC>, Fp4RowsCfg<NV, 128>::kSmem);
    return e;
}

int fp4_gemm_init_device() {
    cudaError_t e = fp4_attr<false, float>();
    if (e == cudaSuccess) e = fp4_attr<false, __nv_bfloat16>();
    if (e == cudaSuccess) e = fp4_attr<true, float>();
    if (e == cudaSuccess) e = fp4_attr<true, __nv_bfloat16>();
    if (e != cudaSuccess) return set_cuda_error(e, "cudaFuncSetAttribute(4-bit gemm)");
    return 0;
}

template <bool NV, int MSUB, int NSUB, typename TC>
static cudaError_t go_pair(const Fp4Plan& p, const CUtensorMap* m, const Fp4GemmArgs& g, cudaStream_t s, DevStatus* st) {
    return launch_chained(fp4_gemm_pair_kernel<NV, MSUB, NSUB, TC>, dim3(p.ctas), kPThreads,
                          Fp4PairCfg<NV, MSUB, NSUB, TC>::kSmem, s, 1, m[0], m[1], m[2], m[3], g, st);
}

template <bool NV, int NT, typename TC>
static cudaError_t go_rows(const Fp4Plan& p, const CUtensorMap* m, const Fp4GemmArgs& g, cudaStream_t s, DevStatus* st) {
    return launch_chained(fp4_gemm_rows_kernel<NV, NT, TC>, dim3(p.ctas), kRThreads, Fp4RowsCfg<NV, NT>::kSmem, s,
                          (unsigned)p.split, m[0], m[1], m[2], m[3], g, p.split, st);
}

template <bool NV, typename TC>
static cudaError_t go_any(const Fp4Plan& p, const CUtensorMap* m, const Fp4GemmArgs& g, cudaStream_t s, DevStatus* st) {
    switch (p.rows) {
        case 512: return go_pair<NV, 2, 1, TC>(p, m, g, s, st);
        case 256: return p.cols == kPN ? go_pair<NV, 1, 1, TC>(p, m, g, s, st) : go_pair<NV, 1, 2, TC>(p, m, g, s, st);
        case 128: return go_rows<NV, 128, TC>(p, m, g, s, st);
        case 64: return go_rows<NV, 64, TC>(p, m, g, s, st);
        default: return go_rows<NV, 32, TC>(p, m, g, s, st);
    }
}

int fp4_gemm_launch(const Fp4& a, const Fp4& b, const int32_t* offsets, const int32_t* counts, void* C, int bf16,
                    int sm_budget, cudaStream_t s, DevStatus* st) {
    DeviceState* ds = device_state();
    if (!ds) return -3;
    if (take_fault(kFaultGemmLaunch)) return set_error(-3, "injected failure: GEMM launch");
    const int cap = (sm_budget <= 0 || sm_budget > ds->sm_count) ? ds->sm_count : sm_budget;
    const Fp4Plan p = fp4_plan(a.rows, b.rows, a.cols, b.count, offsets != nullptr, cap, ds->sm_count);
    Fp4GemmArgs g;
    g.ga = a.tensor_scale;
    g.gb = b.tensor_scale;
    g.offsets = offsets;
    g.counts = counts;
    g.C = C;
    g.M = a.rows;
    g.N = (int)b.rows;
    g.K = (int)a.cols;
    g.experts = b.count;
    g.b_row_tiles = (int)b.row_tiles();
    g.num_m = (int)((a.rows + p.rows - 1) / p.rows);
    g.num_n = (int)((b.rows + p.cols - 1) / p.cols);
    g.num_kb = (int)((a.cols + kFK - 1) / kFK);
    // Under a budget the next kernel starts on no SM that is left to others: it would wait there for this one's end
    // (a chain of 8192^3 on 20 SMs: a product of 0.1 ms on the other 132 took 1.8 ms beside it).
    g.early = cap == ds->sm_count;
    // For experts a bound: each may end inside a tile.
    if (((int64_t)g.num_m + (offsets ? b.count : 0)) * g.num_n * p.split > 0x7FFFFFFF)
        return set_error(-5, "4-bit product has more than 2^31 tiles");
    const bool pair = p.rows > 128;
    CUtensorMap m[4];
    int rc = code_map(&m[0], a, pair ? p.rows / 2 : p.rows);
    if (rc || (rc = code_map(&m[1], b, pair ? kPN / 2 : 128)) || (rc = scale_map(&m[2], a, pair ? p.rows / 256 : 1)) ||
        (rc = scale_map(&m[3], b, pair ? p.cols / kPN + 1 : 1)))
        return rc;
    const cudaError_t e = a.nv ? (bf16 ? go_any<true, __nv_bfloat16>(p, m, g, s, st) : go_any<true, float>(p, m, g, s, st))
                               : (bf16 ? go_any<false, __nv_bfloat16>(p, m, g, s, st) : go_any<false, float>(p, m, g, s, st));
    if (e != cudaSuccess) return set_cuda_error(e, "4-bit gemm kernel launch");
    count_launch();
    return 0;
}

}  // namespace c3
