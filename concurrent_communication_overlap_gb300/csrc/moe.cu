// moe.cu -- what stands between a router and the experts' products: the rows
// of the tokens sorted by expert, and the experts' outputs put together again,
// forward and backward.
#include "ops_device.cuh"
#include "c3_internal.h"

#include <cuda_bf16.h>

namespace c3 {

constexpr unsigned kAll = 0xffffffffu;
constexpr int kMaxExperts = 1024;

// ---------------------------------------------------------------- order
//
// A stable counting sort of the choices by expert.  A choice's row is
//   start[e] + (choices of e before its CTA's) + (before its warp's) + (before it in its warp),
// whole-number sums, so that the rows do not depend on the order in which CTAs or
// atomics run.
//
// Up to kOneLaunch choices, one launch: every CTA counts all choices itself (64 a
// thread at most, from L2) and places 1024 of them, one a thread.  Above, counting
// again in every CTA would cost more than two small launches: one that counts each
// CTA's 4096 choices, one that adds the counts up along the CTAs.  Latency bounds
// all of it (us a call): 192 choices of 64 experts 4.3, 32768 of 32 8.7 (three
// launches: 14), 65536 of 256 13 (three: 19), 524288 of 256 21.
constexpr int kOrderThreads = 1024;
constexpr int kOrderWarps = kOrderThreads / 32;
constexpr int64_t kOneLaunch = 65536;

__device__ __forceinline__ int choice_expert(const int32_t* idx, int64_t i, int64_t n, int experts) {
    if (i >= n) return -1;
    const int e = idx[i];
    return (e >= 0 && e < experts) ? e : -1;
}

// Adds choices [from, to) to counts in shared memory; eight loads at a time, which the
// adds would otherwise keep apart.
__device__ __forceinline__ void count_choices(const int32_t* idx, int64_t from, int64_t to, int experts, int* counts) {
    for (int64_t i0 = from + threadIdx.x; i0 < to; i0 += 8 * kOrderThreads) {
        int e[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) e[j] = choice_expert(idx, i0 + j * kOrderThreads, to, experts);
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (e[j] >= 0) atomicAdd(&counts[e[j]], 1);
    }
}

// Counts of choices [first, first + per_cta) of each CTA.
__global__ void __launch_bounds__(kOrderThreads)
    order_count_kernel(const int32_t* __restrict__ idx, int64_t n, int experts, int per_cta, int* __restrict__ counts) {
    __shared__ int c[kMaxExperts];
    chain_wait();
    for (int e = threadIdx.x; e < experts; e += kOrderThreads) c[e] = 0;
    __syncthreads();
    const int64_t first = (int64_t)blockIdx.x * per_cta;
    count_choices(idx, first, min(n, first + per_cta), experts, c);
    __syncthreads();
    for (int e = threadIdx.x; e < experts; e += kOrderThreads) counts[(size_t)blockIdx.x * experts + e] = c[e];
}

// counts[cta][e] to the sum over the CTAs before, and the sum over all behind the last; a warp an expert.
__global__ void __launch_bounds__(256) order_sum_kernel(int* __restrict__ counts, int ctas, int experts) {
    const int e = blockIdx.x * 8 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
    chain_wait();
    if (e >= experts) return;
    int run = 0;
    for (int b0 = 0; b0 < ctas; b0 += 32) {
        const int c = b0 + lane < ctas ? counts[(size_t)(b0 + lane) * experts + e] : 0;
        int incl = c;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(kAll, incl, o);
            if (lane >= o) incl += v;
        }
        if (b0 + lane < ctas) counts[(size_t)(b0 + lane) * experts + e] = run + incl - c;
        run += __shfl_sync(kAll, incl, 31);
    }
    if (lane == 0) counts[(size_t)ctas * experts + e] = run;
}

// sums: order_sum_kernel's, or NULL where every CTA counts for itself.  1024 threads have 64
// registers each, of which the 32 warps' counts take half: 24 bytes spill.
__global__ void __launch_bounds__(kOrderThreads)
    order_place_kernel(const int32_t* __restrict__ idx, int64_t n, int topk, int experts, int per_cta, int place_ctas,
                       const int* __restrict__ sums, int32_t* __restrict__ slot, int32_t* __restrict__ row_of,
                       int64_t rows, int32_t* __restrict__ offsets, int32_t* __restrict__ counts) {
    extern __shared__ int shared[];
    int* total = shared;              // [experts] choices of each expert
    int* before = total + experts;    // [experts] those of the CTAs before
    int* start = before + experts;    // [experts + 1] first row
    int* hist = start + experts + 1;  // [warps][experts] of this CTA
    __shared__ int warp_sums[kOrderWarps];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t first = (int64_t)blockIdx.x * per_cta;
    const bool places = (int)blockIdx.x < place_ctas;
    chain_wait();
    for (int e = threadIdx.x; e < experts; e += kOrderThreads) {
        total[e] = sums ? sums[(size_t)place_ctas * experts + e] : 0;
        before[e] = sums && places ? sums[(size_t)blockIdx.x * experts + e] : 0;
    }
    if (places)
        for (int i = threadIdx.x; i < kOrderWarps * experts; i += kOrderThreads) hist[i] = 0;
    __syncthreads();
    if (!sums) {
        // the choices of the CTAs before, then this CTA's and those behind
        count_choices(idx, 0, min(first, n), experts, before);
        count_choices(idx, min(first, n), n, experts, total);
        __syncthreads();
        for (int e = threadIdx.x; e < experts; e += kOrderThreads) total[e] += before[e];
    }
    // A warp's choices are consecutive: counted first, so that each warp knows what lies before it.
    const int per_warp = per_cta / kOrderWarps;
    const int64_t mine = first + (int64_t)warp * per_warp;
    if (places)
        for (int j = 0; j < per_warp; j += 32) {
            const int e = choice_expert(idx, mine + j + lane, n, experts);
            const unsigned same = __match_any_sync(kAll, e);
            if (e >= 0 && (same & ((1u << lane) - 1)) == 0) hist[warp * experts + e] += __popc(same);
            __syncwarp();
        }
    __syncthreads();
    // Each expert's first row: an exclusive sum of the counts rounded up to whole tiles, a thread an expert.
    static_assert(kMaxExperts <= kOrderThreads, "a thread an expert");
    const int up = (int)threadIdx.x < experts ? (total[threadIdx.x] + kTileRows - 1) / kTileRows * kTileRows : 0;
    int incl = up;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(kAll, incl, o);
        if (lane >= o) incl += v;
    }
    if (lane == 31) warp_sums[warp] = incl;
    if (places && (int)threadIdx.x < experts) {
        int c[kOrderWarps], run = before[threadIdx.x];
#pragma unroll
        for (int w = 0; w < kOrderWarps; ++w) c[w] = hist[w * experts + threadIdx.x];
#pragma unroll
        for (int w = 0; w < kOrderWarps; ++w) {
            hist[w * experts + threadIdx.x] = run;
            run += c[w];
        }
    }
    __syncthreads();
    const int lower = lane < warp ? warp_sums[lane] : 0;
    const int base = __reduce_add_sync(kAll, lower) + incl - up;
    if ((int)threadIdx.x < experts) start[threadIdx.x] = base;
    if ((int)threadIdx.x == experts - 1) start[experts] = base + up;
    __syncthreads();
    if (blockIdx.x == 0 && (int)threadIdx.x < experts) {
        offsets[threadIdx.x] = base;
        counts[threadIdx.x] = total[threadIdx.x];
        if ((int)threadIdx.x == experts - 1) offsets[experts] = base + up;
    }
    if (places)
        for (int j = 0; j < per_warp; j += 32) {
            const int64_t i = mine + j + lane;
            const int e = choice_expert(idx, i, n, experts);
            const unsigned same = __match_any_sync(kAll, e);
            int row = -1;
            if (e >= 0) row = start[e] + hist[warp * experts + e] + __popc(same & ((1u << lane) - 1));
            __syncwarp();
            if (e >= 0 && (same & ((1u << lane) - 1)) == 0) hist[warp * experts + e] += __popc(same);
            __syncwarp();
            if (i < n) {
                slot[i] = row;
                if (row >= 0) row_of[row] = (int32_t)((unsigned)i / (unsigned)topk);
            }
        }
    // Rows that no choice takes: past an expert's count in its last tile, and past the last expert.
    for (int64_t r = (int64_t)blockIdx.x * kOrderThreads + threadIdx.x; r < rows; r += (int64_t)gridDim.x * kOrderThreads) {
        int lo = 0, hi = experts;  // the last expert that starts at r or before
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (start[mid] <= r) lo = mid;
            else hi = mid;
        }
        if (r >= start[lo] + (int64_t)total[lo]) row_of[r] = -1;
    }
}

int64_t order_rows(int64_t tokens, int topk, int experts) {
    const int64_t n = tokens * topk;
    const int64_t busy = n < experts ? n : experts;
    return (n + (kTileRows - 1) * busy) / kTileRows * kTileRows;
}

static int order_per_cta(int64_t n) { return n <= kOneLaunch ? kOrderThreads : 4 * kOrderThreads; }

size_t order_bytes(int64_t tokens, int topk, int experts) {
    const int64_t n = tokens * topk;
    if (n <= kOneLaunch) return sizeof(int);
    return (size_t)((n + order_per_cta(n) - 1) / order_per_cta(n) + 1) * (size_t)experts * sizeof(int);
}

int order_init_device() {
    cudaError_t e = cudaFuncSetAttribute(order_place_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         (int)sizeof(int) * ((kOrderWarps + 3) * kMaxExperts + 1));
    return e == cudaSuccess ? 0 : set_cuda_error(e, "cudaFuncSetAttribute(order)");
}

int order_launch(const int32_t* idx, int64_t tokens, int topk, int experts, int32_t* slot, int32_t* row_of,
                 int64_t rows, int32_t* offsets, int32_t* counts, void* work, cudaStream_t s) {
    DeviceState* ds = device_state();
    if (!ds) return -3;
    const int64_t n = tokens * topk;
    const int per = order_per_cta(n);
    const int place = (int)((n + per - 1) / per);
    int* sums = n <= kOneLaunch ? nullptr : static_cast<int*>(work);
    cudaError_t e;
    if (sums) {
        e = launch_chained(order_count_kernel, dim3(place), kOrderThreads, 0, s, 1, idx, n, experts, per, sums);
        if (e != cudaSuccess) return set_cuda_error(e, "order count kernel launch");
        count_launch();
        e = launch_chained(order_sum_kernel, dim3((experts + 7) / 8), 256, 0, s, 1, sums, place, experts);
        if (e != cudaSuccess) return set_cuda_error(e, "order sum kernel launch");
        count_launch();
    }
    // CTAs beyond those that place choices only help to mark unused rows
    const int64_t fill = (rows + kOrderThreads - 1) / kOrderThreads;
    const int64_t most = fill < 8 ? (fill > 0 ? fill : 1) : 8;
    const int grid = place > most ? place : (int)most;
    const size_t smem = sizeof(int) * ((size_t)(kOrderWarps + 3) * experts + 1);
    e = launch_chained(order_place_kernel, dim3(grid), kOrderThreads, smem, s, 1, idx, n, topk, experts, per, place, sums, slot,
                       row_of, rows, offsets, counts);
    if (e != cudaSuccess) return set_cuda_error(e, "order kernel launch");
    count_launch();
    return 0;
}

// ---------------------------------------------------------------- combine

constexpr int kCombineThreads = 256;
constexpr int kCombineWarps = kCombineThreads / 32;
constexpr int kSpan = 256;  // columns a warp takes at once: 8 a lane, W by W

// out[t] = sum_j w[t][j] y[slot[t][j]], in fp32, j ascending.  A warp takes one
// token and kSpan columns, so that each row is read in whole runs wherever it lies,
// and few or odd columns leave no CTA half empty; lane j fetches the j-th slot and
// weight for all.  Bytes bound it: 8192 tokens of 8 rows of 4096 bf16 take 102 us,
// 5.9 TB/s; 8192 of 4 rows of 2171, one value at a time, 63 us where the bytes need 26.
template <typename Ty, typename To, int W>
__global__ void __launch_bounds__(kCombineThreads)
    combine_kernel(const Ty* __restrict__ y, int64_t rows, int64_t cols, const int32_t* __restrict__ slot,
                   const float* __restrict__ weights, int64_t tokens, int topk, To* __restrict__ out) {
    const int lane = threadIdx.x & 31;
    constexpr int U = kSpan / (32 * W);
    const int64_t spans = (cols + kSpan - 1) / kSpan, jobs = tokens * spans;
    chain_wait();
    for (int64_t job = (int64_t)blockIdx.x * kCombineWarps + (threadIdx.x >> 5); job < jobs;
         job += (int64_t)gridDim.x * kCombineWarps) {
        const int64_t t = job / spans;
        const int64_t c0 = (job - t * spans) * kSpan + lane * W;
        int r = lane < topk ? slot[t * topk + lane] : -1;
        if (r >= rows) r = -1;
        const float w = lane < topk && weights ? weights[t * topk + lane] : 1.0f;
        float acc[U][W] = {};
#pragma unroll (W == 8 ? 4 : 2)
        for (int j = 0; j < topk; ++j) {
            const int rj = __shfl_sync(kAll, r, j);
            const float wj = __shfl_sync(kAll, w, j);
            if (rj < 0) continue;
            const Ty* yr = y + (int64_t)rj * cols;
            float v[U][W];
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (c0 + 32 * W * u < cols) load_w<W>(yr + c0 + 32 * W * u, v[u]);
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (c0 + 32 * W * u < cols) {
#pragma unroll
                    for (int i = 0; i < W; ++i) acc[u][i] = fmaf(wj, v[u][i], acc[u][i]);
                }
        }
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (c0 + 32 * W * u < cols) store_w<W>(out + t * cols + c0 + 32 * W * u, acc[u]);
    }
}

// dy[slot] = w dout[t] and dw = <dout[t], y[slot]>: one warp a choice, which reads
// its row of y and of dout once for both.  The same 8192 tokens take 170 us, 6.7 TB/s
// (with the loop unrolled 3 or 4 times 180: many warps with few loads each suit it).
template <typename Td, typename Ty, int W>
__global__ void __launch_bounds__(kCombineThreads)
    combine_backward_kernel(const Td* __restrict__ dout, const Ty* __restrict__ y, int64_t rows, int64_t cols,
                            const int32_t* __restrict__ slot, const float* __restrict__ weights, int64_t tokens,
                            int topk, Ty* __restrict__ dy, float* __restrict__ dweights) {
    constexpr int U = kSpan / (32 * W);
    const int lane = threadIdx.x & 31;
    chain_wait();
    for (int64_t job = (int64_t)blockIdx.x * kCombineWarps + (threadIdx.x >> 5); job < tokens * topk;
         job += (int64_t)gridDim.x * kCombineWarps) {
        const int r = slot[job];
        float dot = 0.0f;
        if (r >= 0 && r < rows) {
            const float w = weights ? weights[job] : 1.0f;
            const Td* dr = dout + job / topk * cols;
            const int64_t at = (int64_t)r * cols;
#pragma unroll (W == 8 ? 1 : 2)
            for (int64_t c0 = lane * W; c0 < cols; c0 += kSpan) {
                float d[U][W], v[U][W], eight = 0.0f;  // a sum of its own: fewer roundings of the long one
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const int64_t c = c0 + 32 * W * u;
                    if (U > 1 && c >= cols) continue;
                    load_w<W>(dr + c, d[u]);
                    if (dweights) load_w<W>(y + at + c, v[u]);
                }
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const int64_t c = c0 + 32 * W * u;
                    if (U > 1 && c >= cols) continue;
                    if (dweights) {
#pragma unroll
                        for (int i = 0; i < W; ++i) eight = fmaf(d[u][i], v[u][i], eight);
                    }
#pragma unroll
                    for (int i = 0; i < W; ++i) d[u][i] *= w;
                    store_w<W>(dy + at + c, d[u]);
                }
                dot += eight;
            }
        }
        if (dweights) {
#pragma unroll
            for (int o = 16; o; o >>= 1) dot += __shfl_xor_sync(kAll, dot, o);
            if (lane == 0) dweights[job] = dot;
        }
    }
}

static int combine_grid(int64_t jobs) {
    DeviceState* ds = device_state();
    if (!ds) return 0;
    const int64_t need = (jobs + kCombineWarps - 1) / kCombineWarps, most = (int64_t)ds->sm_count * 32;
    return (int)(need < most ? need : most);
}

// Values at once: 8 where rows are whole 16-byte units of both types, else 2 or 1.
static int rows_width(const void* p, int64_t cols, int bf16) {
    const size_t sz = bf16 ? 2 : 4;
    if ((uintptr_t)p % 16 == 0 && cols % 8 == 0) return 8;
    return (uintptr_t)p % (2 * sz) == 0 && cols % 2 == 0 ? 2 : 1;
}

// One of three instances by width.
template <typename K>
static K by_width(int w, K k8, K k2, K k1) {
    return w == 8 ? k8 : w == 2 ? k2 : k1;
}

template <typename Ty, typename To>
static int combine_go(const void* y, int64_t rows, int64_t cols, const int32_t* slot, const float* weights,
                      int64_t tokens, int topk, void* out, int width, cudaStream_t s) {
    const int grid = combine_grid(tokens * ((cols + kSpan - 1) / kSpan));
    if (grid == 0) return -3;
    const auto kernel = by_width(width, combine_kernel<Ty, To, 8>, combine_kernel<Ty, To, 2>, combine_kernel<Ty, To, 1>);
    const cudaError_t e = launch_chained(kernel, dim3(grid), kCombineThreads, 0, s, 1, static_cast<const Ty*>(y), rows, cols,
                                         slot, weights, tokens, topk, static_cast<To*>(out));
    if (e != cudaSuccess) return set_cuda_error(e, "combine kernel launch");
    count_launch();
    return 0;
}

int combine_launch(const void* y, int y_bf16, int64_t rows, int64_t cols, const int32_t* slot, const float* weights,
                   int64_t tokens, int topk, void* out, int out_bf16, cudaStream_t s) {
    const int w = rows_width(y, cols, y_bf16), wo = rows_width(out, cols, out_bf16), width = w < wo ? w : wo;
    if (y_bf16)
        return out_bf16 ? combine_go<__nv_bfloat16, __nv_bfloat16>(y, rows, cols, slot, weights, tokens, topk, out, width, s)
                        : combine_go<__nv_bfloat16, float>(y, rows, cols, slot, weights, tokens, topk, out, width, s);
    return out_bf16 ? combine_go<float, __nv_bfloat16>(y, rows, cols, slot, weights, tokens, topk, out, width, s)
                    : combine_go<float, float>(y, rows, cols, slot, weights, tokens, topk, out, width, s);
}

template <typename Td, typename Ty>
static int combine_back_go(const void* dout, const void* y, int64_t rows, int64_t cols, const int32_t* slot,
                           const float* weights, int64_t tokens, int topk, void* dy, float* dweights, int width,
                           cudaStream_t s) {
    const int grid = combine_grid(tokens * topk);
    if (grid == 0) return -3;
    const auto kernel = by_width(width, combine_backward_kernel<Td, Ty, 8>, combine_backward_kernel<Td, Ty, 2>,
                                 combine_backward_kernel<Td, Ty, 1>);
    const cudaError_t e = launch_chained(kernel, dim3(grid), kCombineThreads, 0, s, 1, static_cast<const Td*>(dout),
                                         static_cast<const Ty*>(y), rows, cols, slot, weights, tokens, topk,
                                         static_cast<Ty*>(dy), dweights);
    if (e != cudaSuccess) return set_cuda_error(e, "combine backward kernel launch");
    count_launch();
    return 0;
}

int combine_backward_launch(const void* dout, int dout_bf16, const void* y, int y_bf16, int64_t rows, int64_t cols,
                            const int32_t* slot, const float* weights, int64_t tokens, int topk, void* dy,
                            float* dweights, cudaStream_t s) {
    int w = rows_width(dout, cols, dout_bf16);
    const int wd = rows_width(dy, cols, y_bf16), wy = dweights ? rows_width(y, cols, y_bf16) : 8;
    w = w < wd ? w : wd;
    w = w < wy ? w : wy;
    if (dout_bf16)
        return y_bf16 ? combine_back_go<__nv_bfloat16, __nv_bfloat16>(dout, y, rows, cols, slot, weights, tokens, topk, dy, dweights, w, s)
                      : combine_back_go<__nv_bfloat16, float>(dout, y, rows, cols, slot, weights, tokens, topk, dy, dweights, w, s);
    return y_bf16 ? combine_back_go<float, __nv_bfloat16>(dout, y, rows, cols, slot, weights, tokens, topk, dy, dweights, w, s)
                  : combine_back_go<float, float>(dout, y, rows, cols, slot, weights, tokens, topk, dy, dweights, w, s);
}

}  // namespace c3
