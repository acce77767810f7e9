// embed.cu -- the lookup of embeddings with a scale, and the gradient of the table,
// whose rows are sums over the tokens that named them: the tokens are sorted by row
// first, so that every sum has one owner and a fixed order.
#include "ops_device.cuh"
#include "c3_internal.h"

namespace c3 {

constexpr unsigned kAll = 0xffffffffu;
constexpr int kEmbedThreads = 256;
constexpr int kEmbedWarps = kEmbedThreads / 32;
constexpr int kSpan = 256;  // columns a warp takes of a row at once: 8 a lane, W by W

// ---------------------------------------------------------------- lookup

// out[t] = scale * table[ids[t] - first], zeros where that is no row.  A warp takes one
// token and kSpan columns; each row is read and written once, in whole runs.
template <typename Tt, typename To, int W>
__global__ void __launch_bounds__(kEmbedThreads)
    embed_kernel(const Tt* __restrict__ table, int64_t rows, int64_t cols, int64_t ld, int64_t first,
                 const int32_t* __restrict__ ids, int64_t tokens, float scale, To* __restrict__ out, int64_t out_ld) {
    constexpr int U = kSpan / (32 * W);
    const int lane = threadIdx.x & 31;
    const int64_t spans = (cols + kSpan - 1) / kSpan, jobs = tokens * spans;
    chain_wait();
    for (int64_t job = (int64_t)blockIdx.x * kEmbedWarps + (threadIdx.x >> 5); job < jobs;
         job += (int64_t)gridDim.x * kEmbedWarps) {
        const int64_t t = job / spans, c0 = (job - t * spans) * kSpan + lane * W;
        const int64_t r = (int64_t)ids[t] - first;
        const bool have = r >= 0 && r < rows;
        float v[U][W] = {};
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (have && c0 + 32 * W * u < cols) load_w<W>(table + r * ld + c0 + 32 * W * u, v[u]);
#pragma unroll
        for (int u = 0; u < U; ++u) {
#pragma unroll
            for (int i = 0; i < W; ++i) v[u][i] = have ? v[u][i] * scale : 0.0f;
            if (c0 + 32 * W * u < cols) store_w<W>(out + t * out_ld + c0 + 32 * W * u, v[u]);
        }
    }
}

// ---------------------------------------------------------------- order of the tokens by row
//
// A stable radix sort of (row, token) by row, least digit first, by one cluster in one
// launch.  A token's place in a pass is
//   start[digit] + (of the CTAs before) + (of the warps before) + (before it in its warp),
// whole-number sums, so that the order does not depend on timing.  Tokens without a row
// in the table drop out in the first pass.
constexpr int kSortThreads = 1024;
constexpr int kSortWarps = kSortThreads / 32;
constexpr int kSortBits = 10;  // a digit at most: a thread a bin in the scans
constexpr int kSortCtas = 8;

// What the sort leaves for the sums.
struct EmbedOrder {
    int valid;  // tokens that have a row
    int joins;  // chunks whose last row goes on in the next
};

__device__ __forceinline__ int remote_int(uint32_t addr) {
    int v;
    asm volatile("ld.shared::cluster.b32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
    return v;
}

// pairs: where the sorted (row, token) end up; other: as much scratch.  joins: numbers of the chunks
// (of `chunk` places) whose last row goes on in the next.  touched: a bit a row of the table, or NULL.
__global__ void __launch_bounds__(kSortThreads, 1)
    embed_sort_kernel(const int32_t* __restrict__ ids, int64_t n, int64_t first, int64_t rows, int bits, int passes,
                      int2* pairs, int2* other, int chunk, EmbedOrder* order, int* joins, uint32_t* touched) {
    extern __shared__ int shared[];
    const int bins = 1 << bits;
    int* total = shared;                       // [bins] this CTA's, read by the others
    int* hist = shared + bins;                 // [warps][bins]
    __shared__ int warp_sums[kSortWarps];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const unsigned before_me = (1u << lane) - 1;
    const int ctas = (int)gridDim.x, rank = (int)blockIdx.x;
    chain_wait();
    if (touched)
        for (int64_t i = (int64_t)rank * kSortThreads + threadIdx.x; i < (rows + 31) / 32; i += (int64_t)ctas * kSortThreads)
            touched[i] = 0;
    if (rank == 0 && threadIdx.x == 0) order->joins = 0;
    int valid = 0;
    for (int pass = 0; pass < passes; ++pass) {
        int2* to = (passes - pass) & 1 ? pairs : other;
        const int2* from = (passes - pass) & 1 ? other : pairs;
        const int64_t count = pass ? valid : n;
        // A warp's places are consecutive, whole groups of 32.
        const int64_t per = (count + (int64_t)ctas * kSortThreads - 1) / ((int64_t)ctas * kSortThreads) * 32;
        const int64_t mine = ((int64_t)rank * kSortWarps + warp) * per;
        const int64_t end = mine + per < count ? mine + per : count;
        const int shift = pass * bits;
        auto fetch = [&](int64_t i) {
            if (i >= end) return make_int2(-1, 0);
            if (pass) return __ldcg(from + i);
            const int64_t r = (int64_t)ids[i] - first;
            return make_int2(r >= 0 && r < rows ? (int)r : -1, (int)i);
        };
        for (int d = lane; d < bins; d += 32) hist[warp * bins + d] = 0;
        __syncwarp();
        for (int64_t i0 = mine; i0 < end; i0 += 32) {
            const int2 p = fetch(i0 + lane);
            const int d = p.x < 0 ? -1 : (p.x >> shift) & (bins - 1);
            const unsigned same = __match_any_sync(kAll, d);
            if (d >= 0 && (same & before_me) == 0) hist[warp * bins + d] += __popc(same);
            __syncwarp();
        }
        __syncthreads();
        const int d = threadIdx.x;
        int sum = 0;
        if (d < bins) {
            for (int w = 0; w < kSortWarps; ++w) sum += hist[w * bins + d];
            total[d] = sum;
        }
        cluster_sync_all();
        int all = 0, before = 0;
        if (d < bins)
            for (int c = 0; c < ctas; ++c) {
                const int v = remote_int(peer_addr(smem_addr(&total[d]), (uint32_t)c));
                all += v;
                if (c < rank) before += v;
            }
        // exclusive sum over the bins
        int incl = all;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(kAll, incl, o);
            if (lane >= o) incl += v;
        }
        if (lane == 31) warp_sums[warp] = incl;
        __syncthreads();
        const int lower = __reduce_add_sync(kAll, lane < warp ? warp_sums[lane] : 0);
        valid = __reduce_add_sync(kAll, warp_sums[lane]);
        if (d < bins) {
            int run = lower + incl - all + before;
            for (int w = 0; w < kSortWarps; ++w) {
                const int c = hist[w * bins + d];
                hist[w * bins + d] = run;
                run += c;
            }
        }
        __syncthreads();
        for (int64_t i0 = mine; i0 < end; i0 += 32) {
            const int2 p = fetch(i0 + lane);
            const int dig = p.x < 0 ? -1 : (p.x >> shift) & (bins - 1);
            const unsigned same = __match_any_sync(kAll, dig);
            if (dig >= 0) to[hist[warp * bins + dig] + __popc(same & before_me)] = p;
            __syncwarp();
            if (dig >= 0 && (same & before_me) == 0) hist[warp * bins + dig] += __popc(same);
            __syncwarp();
        }
        cluster_sync_all();  // the pairs are where the next pass looks for them, and `total` has been read
    }
    if (rank == 0 && threadIdx.x == 0) order->valid = valid;
    for (int64_t p = (int64_t)rank * kSortThreads + threadIdx.x; p < valid; p += (int64_t)ctas * kSortThreads) {
        const int row = __ldcg(&pairs[p].x);
        if (p > 0 && __ldcg(&pairs[p - 1].x) == row) continue;
        if (touched) atomicOr(&touched[row >> 5], 1u << (row & 31));
        const int64_t next = (p / chunk + 1) * chunk;
        if (next < valid && __ldcg(&pairs[next].x) == row) joins[atomicAdd(&order->joins, 1)] = (int)(p / chunk);
    }
}

// ---------------------------------------------------------------- sums
//
// The sorted places are cut into chunks.  A warp adds up kSpan columns of a chunk's
// tokens, in order.  A row whose tokens all lie in the chunk is written at once; of a
// row that comes from the chunk before, the chunk's sum goes to heads[chunk], of one
// that begins here and goes on, to tails[chunk].  embed_join_kernel adds those up, in
// the order of the chunks.  Rows that no token names are written as zeros beside, by
// warps of their own.
struct EmbedSum {
    const int2* pairs;
    const EmbedOrder* order;
    const int* joins;
    const uint32_t* touched;  // NULL: rows without tokens are left as they are
    float* heads;             // [chunks][pitch]
    float* tails;
    int64_t rows, cols, ld, dout_ld, pitch;
    int chunk, chunks;
    int accumulate;
    float scale;
};

template <typename Tt, int W>
__device__ __forceinline__ void add_row(const EmbedSum& g, Tt* table, int row, int64_t c, const float (&v)[W]) {
    Tt* at = table + (int64_t)row * g.ld + c;
    float o[W] = {};
    if (g.accumulate) load_w<W>(at, o);
#pragma unroll
    for (int i = 0; i < W; ++i) o[i] = g.accumulate ? fmaf(g.scale, v[i], o[i]) : g.scale * v[i];
    store_w<W>(at, o);
}

template <typename Td, typename Tt, int W>
__global__ void __launch_bounds__(kEmbedThreads)
    embed_sum_kernel(const Td* __restrict__ dout, Tt* __restrict__ table, EmbedSum g) {
    constexpr int U = kSpan / (32 * W), B = W == 8 ? 8 : W == 2 ? 4 : 2;  // rows in flight
    const int lane = threadIdx.x & 31;
    const int64_t spans = (g.cols + kSpan - 1) / kSpan;
    const int64_t step = (int64_t)gridDim.x * kEmbedWarps;
    chain_wait();
    const int valid = g.order->valid;
    const int64_t chunks = ((int64_t)valid + g.chunk - 1) / g.chunk, jobs = chunks * spans;
    int64_t job = (int64_t)blockIdx.x * kEmbedWarps + (threadIdx.x >> 5);
    for (; job < jobs; job += step) {
        const int64_t ch = job / spans, c0 = (job - ch * spans) * kSpan + lane * W;
        const int64_t p0 = ch * g.chunk, p1 = p0 + g.chunk < valid ? p0 + g.chunk : valid;
        const int last = p0 > 0 ? g.pairs[p0 - 1].x : -1, next = p1 < valid ? g.pairs[p1].x : -1;
        float acc[U][W] = {};
        int row = -1;
        bool head = false;
        auto flush = [&](bool goes_on) {
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int64_t c = c0 + 32 * W * u;
                if (c >= g.cols) continue;
                if (head) store_w<W>(g.heads + ch * g.pitch + c, acc[u]);
                else if (goes_on) store_w<W>(g.tails + ch * g.pitch + c, acc[u]);
                else add_row<Tt, W>(g, table, row, c, acc[u]);
            }
        };
        for (int64_t q = p0; q < p1; q += 32) {
            const int2 mine = q + lane < p1 ? g.pairs[q + lane] : make_int2(-1, 0);
            const int here = (int)(p1 - q < 32 ? p1 - q : 32);
            for (int j0 = 0; j0 < here; j0 += B) {
                float v[B][U][W];
#pragma unroll
                for (int b = 0; b < B; ++b) {
                    const int64_t t = __shfl_sync(kAll, mine.y, (j0 + b) & 31);
#pragma unroll
                    for (int u = 0; u < U; ++u)
                        if (j0 + b < here && c0 + 32 * W * u < g.cols) load_w<W>(dout + t * g.dout_ld + c0 + 32 * W * u, v[b][u]);
                }
#pragma unroll
                for (int b = 0; b < B; ++b) {
                    const int r = __shfl_sync(kAll, mine.x, (j0 + b) & 31);
                    if (j0 + b >= here) break;
                    if (r != row) {
                        if (row >= 0) flush(false);
                        head = row < 0 && r == last;
                        row = r;
#pragma unroll
                        for (int u = 0; u < U; ++u)
#pragma unroll
                            for (int i = 0; i < W; ++i) acc[u][i] = 0.0f;
                    }
#pragma unroll
                    for (int u = 0; u < U; ++u)
#pragma unroll
                        for (int i = 0; i < W; ++i) acc[u][i] += v[b][u][i];
                }
            }
        }
        flush(row == next);
    }
    if (g.touched == nullptr) return;
    // rows without tokens, a warp four of them
    const int64_t groups = (g.rows + 3) / 4;
    for (job -= jobs; job < groups; job += step) {
        const uint32_t bits = g.touched[job >> 3] >> ((job & 7) * 4);
        for (int i = 0; i < 4; ++i) {
            const int64_t r = job * 4 + i;
            if (r >= g.rows || (bits >> i & 1)) continue;
            const float zero[W] = {};
            for (int64_t c = lane * W; c < g.cols; c += 32 * W) store_w<W>(table + r * g.ld + c, zero);
        }
    }
}

// The rows whose tokens lie in several chunks: tails[c] + heads[c + 1] + ... .  A CTA a row and kSpan columns;
// each warp adds up consecutive parts, and the warps' sums meet in shared memory, in order.
constexpr int kJoinThreads = 512;
constexpr int kJoinWarps = kJoinThreads / 32;

template <typename Tt, int W>
__global__ void __launch_bounds__(kJoinThreads) embed_join_kernel(Tt* __restrict__ table, EmbedSum g) {
    constexpr int U = kSpan / (32 * W);
    __shared__ float part[kJoinWarps][kSpan];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t spans = (g.cols + kSpan - 1) / kSpan;
    chain_wait();
    const int valid = g.order->valid;
    const int64_t jobs = g.order->joins * spans;
    for (int64_t job = blockIdx.x; job < jobs; job += gridDim.x) {
        const int64_t at = job / spans, c0 = (job - at * spans) * kSpan + lane * W;
        const int64_t ch = g.joins[at];
        const int row = g.pairs[(ch + 1) * g.chunk].x;
        // how many chunks begin with the row, every warp for itself
        int64_t more = 0;
        for (bool all = true; all; more += 32) {
            const int64_t p = (ch + 1 + more + lane) * g.chunk;
            const unsigned is = __ballot_sync(kAll, p < valid && g.pairs[p < valid ? p : 0].x == row);
            all = is == kAll;
            if (!all) {
                more += __ffs(~is) - 1;
                break;
            }
        }
        const int64_t per = (more + 1 + kJoinWarps - 1) / kJoinWarps;
        const int64_t from = warp * per, to = from + per < more + 1 ? from + per : more + 1;
        float acc[U][W] = {};
#pragma unroll 4
        for (int64_t k = from; k < to; ++k) {
            const float* src = (k ? g.heads : g.tails) + (ch + k) * g.pitch;
#pragma unroll
            for (int u = 0; u < U; ++u) {
                float v[W] = {};
                if (c0 + 32 * W * u < g.cols) load_w<W>(src + c0 + 32 * W * u, v);
#pragma unroll
                for (int i = 0; i < W; ++i) acc[u][i] += v[i];
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int i = 0; i < W; ++i) part[warp][(u * W + i) * 32 + lane] = acc[u][i];
        __syncthreads();
        if (warp == 0) {
#pragma unroll
            for (int u = 0; u < U; ++u)
#pragma unroll
                for (int i = 0; i < W; ++i) {
                    float sum = 0.0f;
                    for (int w = 0; w < kJoinWarps; ++w) sum += part[w][(u * W + i) * 32 + lane];
                    acc[u][i] = sum;
                }
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (c0 + 32 * W * u < g.cols) add_row<Tt, W>(g, table, row, c0 + 32 * W * u, acc[u]);
        }
        __syncthreads();
    }
}

// ---------------------------------------------------------------- host side

// Rows as they lie in memory: base, row distance, type.
struct Lines {
    const void* p;
    int64_t ld;
    int bf16;
    bool fits(int w) const {
        const uintptr_t size = bf16 ? 2 : 4, unit = w * size < 16 ? w * size : 16;
        return (uintptr_t)p % unit == 0 && (uintptr_t)ld * size % unit == 0;
    }
};
// Values a lane loads at once: 8 where every row begins at a multiple of 16 bytes and ends in whole
// vectors, 2 where pairs do, else 1.
static int width(int64_t cols, const Lines& x, const Lines& y) {
    for (int w : {8, 2})
        if (cols % w == 0 && x.fits(w) && y.fits(w)) return w;
    return 1;
}

int embed_init_device() {
    const int most = (int)sizeof(int) * (kSortWarps + 1) << kSortBits;
    cudaError_t e = cudaFuncSetAttribute(embed_sort_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, most);
    return e == cudaSuccess ? 0 : set_cuda_error(e, "cudaFuncSetAttribute(embedding order)");
}

template <typename Tt, typename To>
static cudaError_t go_lookup(int w, unsigned grid, cudaStream_t s, const void* table, const EmbedArgs& a, const int32_t* ids,
                             void* out) {
    auto go = [&](auto kernel) {
        return launch_chained(kernel, dim3(grid), kEmbedThreads, 0, s, 1, static_cast<const Tt*>(table), a.rows, a.cols, a.ld,
                              a.first, ids, a.tokens, a.scale, static_cast<To*>(out), a.out_ld);
    };
    return w == 8 ? go(embed_kernel<Tt, To, 8>) : w == 2 ? go(embed_kernel<Tt, To, 2>) : go(embed_kernel<Tt, To, 1>);
}

int embed_launch(const void* table, int bf16, const EmbedArgs& a, const int32_t* ids, void* out, int out_bf16,
                 cudaStream_t s) {
    DeviceState* ds = device_state();
    if (!ds) return -3;
    const int w = width(a.cols, Lines{table, a.ld, bf16}, Lines{out, a.out_ld, out_bf16});
    const int64_t ctas = (a.tokens * ((a.cols + kSpan - 1) / kSpan) + kEmbedWarps - 1) / kEmbedWarps;
    const int64_t most = (int64_t)ds->sm_count * 8;
    const unsigned grid = (unsigned)(ctas < most ? ctas : most);
    const cudaError_t e = bf16 ? (out_bf16 ? go_lookup<__nv_bfloat16, __nv_bfloat16>(w, grid, s, table, a, ids, out)
                                           : go_lookup<__nv_bfloat16, float>(w, grid, s, table, a, ids, out))
                               : (out_bf16 ? go_lookup<float, __nv_bfloat16>(w, grid, s, table, a, ids, out)
                                           : go_lookup<float, float>(w, grid, s, table, a, ids, out));
    if (e != cudaSuccess) return set_cuda_error(e, "embedding kernel launch");
    count_launch();
    return 0;
}

// The workspace: where each part begins, in bytes.
struct EmbedWork {
    int chunk, chunks;
    int64_t pitch;
    size_t pairs, other, joins, touched, heads, tails, bytes;
};

static EmbedWork embed_work(int64_t tokens, int64_t rows, int64_t cols) {
    EmbedWork w;
    const int64_t spans = (cols + kSpan - 1) / kSpan;
    w.chunk = 8;
    while ((tokens + w.chunk - 1) / w.chunk * spans > 16384 && w.chunk < (1 << 20)) w.chunk *= 2;
    w.chunks = (int)((tokens + w.chunk - 1) / w.chunk);
    w.pitch = (cols + 7) / 8 * 8;
    size_t at = 256;
    auto part = [&](size_t bytes) {
        const size_t from = at;
        at += (bytes + 255) / 256 * 256;
        return from;
    };
    w.pairs = part((size_t)tokens * sizeof(int2));
    w.other = part((size_t)tokens * sizeof(int2));
    w.joins = part((size_t)w.chunks * sizeof(int));
    w.touched = part((size_t)(rows + 31) / 32 * sizeof(uint32_t));
    w.heads = part((size_t)w.chunks * (size_t)w.pitch * sizeof(float));
    w.tails = part((size_t)w.chunks * (size_t)w.pitch * sizeof(float));
    w.bytes = at;
    return w;
}

size_t embed_backward_bytes(int64_t tokens, int64_t rows, int64_t cols) { return embed_work(tokens, rows, cols).bytes; }

template <typename Td, typename Tt>
static cudaError_t go_sums(int w, unsigned grid, unsigned join_grid, cudaStream_t s, const void* dout, void* table,
                           const EmbedSum& g) {
    auto go = [&](auto sum, auto join) {
        cudaError_t e = launch_chained(sum, dim3(grid), kEmbedThreads, 0, s, 1, static_cast<const Td*>(dout),
                                       static_cast<Tt*>(table), g);
        if (e != cudaSuccess || join_grid == 0) return e;
        count_launch();
        return launch_chained(join, dim3(join_grid), kJoinThreads, 0, s, 1, static_cast<Tt*>(table), g);
    };
    return w == 8   ? go(embed_sum_kernel<Td, Tt, 8>, embed_join_kernel<Tt, 8>)
           : w == 2 ? go(embed_sum_kernel<Td, Tt, 2>, embed_join_kernel<Tt, 2>)
                    : go(embed_sum_kernel<Td, Tt, 1>, embed_join_kernel<Tt, 1>);
}

int embed_backward_launch(const void* dout, int dout_bf16, const EmbedArgs& a, const int32_t* ids, int accumulate,
                          void* table, int bf16, void* work, cudaStream_t s) {
    DeviceState* ds = device_state();
    if (!ds) return -3;
    const EmbedWork w = embed_work(a.tokens, a.rows, a.cols);
    uint8_t* base = static_cast<uint8_t*>(work);
    EmbedSum g;
    g.pairs = reinterpret_cast<int2*>(base + w.pairs);
    g.order = reinterpret_cast<EmbedOrder*>(base);
    g.joins = reinterpret_cast<int*>(base + w.joins);
    g.touched = accumulate ? nullptr : reinterpret_cast<uint32_t*>(base + w.touched);
    g.heads = reinterpret_cast<float*>(base + w.heads);
    g.tails = reinterpret_cast<float*>(base + w.tails);
    g.rows = a.rows;
    g.cols = a.cols;
    g.ld = a.ld;
    g.dout_ld = a.out_ld;
    g.pitch = w.pitch;
    g.chunk = w.chunk;
    g.chunks = w.chunks;
    g.accumulate = accumulate;
    g.scale = a.scale;
    int bits = 1;
    while (bits < 31 && ((int64_t)1 << bits) < a.rows) ++bits;
    const int passes = (bits + kSortBits - 1) / kSortBits;
    bits = (bits + passes - 1) / passes;
    const int ctas = a.tokens <= 4 * kSortThreads ? 1 : kSortCtas;
    cudaError_t e = launch_chained(embed_sort_kernel, dim3(ctas), kSortThreads, sizeof(int) * (kSortWarps + 1) << bits, s,
                                   (unsigned)ctas, ids, a.tokens, a.first, a.rows, bits, passes, const_cast<int2*>(g.pairs),
                                   reinterpret_cast<int2*>(base + w.other), w.chunk, const_cast<EmbedOrder*>(g.order),
                                   const_cast<int*>(g.joins), const_cast<uint32_t*>(g.touched));
    if (e != cudaSuccess) return set_cuda_error(e, "embedding order kernel launch");
    count_launch();
    const int64_t spans = (a.cols + kSpan - 1) / kSpan;
    const int64_t jobs = w.chunks * spans + (accumulate ? 0 : (a.rows + 3) / 4), most = (int64_t)ds->sm_count * 8;
    const int64_t ctas_sum = (jobs + kEmbedWarps - 1) / kEmbedWarps;
    const unsigned grid = (unsigned)(ctas_sum < most ? ctas_sum : most);
    const int64_t joins = w.chunks > 1 ? (int64_t)(w.chunks - 1) * spans : 0, most_joins = (int64_t)ds->sm_count * 2;
    const unsigned join_grid = (unsigned)(joins < most_joins ? joins : most_joins);
    const int wide = width(a.cols, Lines{dout, a.out_ld, dout_bf16}, Lines{table, a.ld, bf16});
    e = dout_bf16 ? (bf16 ? go_sums<__nv_bfloat16, __nv_bfloat16>(wide, grid, join_grid, s, dout, table, g)
                          : go_sums<__nv_bfloat16, float>(wide, grid, join_grid, s, dout, table, g))
                  : (bf16 ? go_sums<float, __nv_bfloat16>(wide, grid, join_grid, s, dout, table, g)
                          : go_sums<float, float>(wide, grid, join_grid, s, dout, table, g));
    if (e != cudaSuccess) return set_cuda_error(e, "embedding gradient kernel launch");
    count_launch();
    return 0;
}

}  // namespace c3
