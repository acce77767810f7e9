// embed.cu -- the lookup of embeddings with a scale, and the gradient of the table,
// whose rows are sums over the tokens that named them: the tokens are sorted by row
// first, so that every sum has one owner and a fixed order.
#include "ops_device.cuh"
#include "c3_internal.h"

#include <type_traits>

namespace c3 {

constexpr unsigned kAll = 0xffffffffu;
constexpr int kEmbedThreads = 256;
constexpr int kEmbedWarps = kEmbedThreads / 32;
constexpr int kSpan = 256;  // columns a warp takes of a row at once, 8 a lane

// ---------------------------------------------------------------- rows wherever they begin
//
// A lane's 8 values of a row are 16 or 32 bytes.  Where every row begins at a multiple of 16 bytes
// and has whole vectors (SHIFT false) they are loaded and stored as they are.  Elsewhere a row's
// aligned 16-byte units are: loads take the units that hold a lane's values, one more than they
// fill, and shift them into place; stores shift the values on by what the row is off, the lane
// before lending its last ones, and write whole units but for the row's ends.  A unit is touched
// only where it holds a value of the row.

template <typename T, bool SHIFT>
struct Units {
    static constexpr int kCount = (int)sizeof(T) / 2 + (SHIFT ? 1 : 0);
    uint4 v[kCount];
};

// The units of the 8 values from p on, of a row that ends at `end`.
template <typename T, bool SHIFT>
__device__ __forceinline__ void load_units(const T* p, const T* end, Units<T, SHIFT>& r) {
    const uintptr_t at = SHIFT ? (uintptr_t)p & ~(uintptr_t)15 : (uintptr_t)p;
#pragma unroll
    for (int i = 0; i < Units<T, SHIFT>::kCount; ++i)
        r.v[i] = at + 16 * i < (uintptr_t)end ? *reinterpret_cast<const uint4*>(at + 16 * i) : make_uint4(0, 0, 0, 0);
}

// w moved down by `bytes` (whole values of T).
template <typename T, int N>
__device__ __forceinline__ void shift_words(uint32_t (&w)[N], int bytes) {
#pragma unroll
    for (int step = 16; step >= 4; step /= 2)
        if (bytes & step) {
#pragma unroll
            for (int i = 0; i + step / 4 < N; ++i) w[i] = w[i + step / 4];
        }
    if (sizeof(T) == 2 && (bytes & 2)) {
#pragma unroll
        for (int i = 0; i + 1 < N; ++i) w[i] = __funnelshift_r(w[i], w[i + 1], 16);
    }
}

template <typename T, bool SHIFT>
__device__ __forceinline__ void unit_values(const Units<T, SHIFT>& r, const T* p, float (&v)[8]) {
    uint32_t w[4 * Units<T, SHIFT>::kCount];
#pragma unroll
    for (int i = 0; i < Units<T, SHIFT>::kCount; ++i) w[4 * i] = r.v[i].x, w[4 * i + 1] = r.v[i].y, w[4 * i + 2] = r.v[i].z, w[4 * i + 3] = r.v[i].w;
    if constexpr (SHIFT) shift_words<T>(w, (int)((uintptr_t)p & 15));
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        if constexpr (sizeof(T) == 4) v[i] = __uint_as_float(w[i]);
        else v[i] = __uint_as_float(i & 1 ? w[i / 2] & 0xffff0000u : w[i / 2] << 16);
    }
}

// The warp's values of a row, n of them (kSpan at most); p: the place of this lane's first.
template <typename T, bool SHIFT>
__device__ __forceinline__ void store_values(T* p, const float (&v)[8], int n, int lane) {
    constexpr int NW = 2 * (int)sizeof(T), VB = 16 / (int)sizeof(T);
    uint32_t w[NW + 4];
#pragma unroll
    for (int i = 0; i < NW; ++i) {
        if constexpr (sizeof(T) == 4) {
            w[4 + i] = __float_as_uint(v[i]);
        } else {
            const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
            w[4 + i] = *reinterpret_cast<const uint32_t*>(&h);
        }
    }
    if constexpr (!SHIFT) {
        if (8 * lane >= n) return;
#pragma unroll
        for (int j = 0; j < NW / 4; ++j)
            reinterpret_cast<uint4*>(p)[j] = make_uint4(w[4 + 4 * j], w[5 + 4 * j], w[6 + 4 * j], w[7 + 4 * j]);
    } else {
        using Bits = std::conditional_t<sizeof(T) == 4, uint32_t, uint16_t>;
        const int off = (int)((uintptr_t)p & 15), k = off / (int)sizeof(T);
        auto value = [&](const uint32_t* x, int i) { return (Bits)(sizeof(T) == 4 ? x[i] : x[i / 2] >> (16 * (i & 1))); };
        if (lane == 31) {  // what is left behind the last whole unit
#pragma unroll
            for (int i = 8 - VB + 1; i < 8; ++i)
                if (i >= 8 - k && 248 + i < n) reinterpret_cast<Bits*>(p)[i] = value(w + 4, i);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = __shfl_up_sync(kAll, w[NW + i], 1);
        shift_words<T>(w, 16 - off);
#pragma unroll
        for (int j = 0; j < NW / 4; ++j) {
            const int first = 8 * lane - k + j * VB;
            Bits* at = reinterpret_cast<Bits*>(p) + (j * VB - k);
            if (first >= 0 && first + VB <= n) {
                *reinterpret_cast<uint4*>(at) = make_uint4(w[4 * j], w[4 * j + 1], w[4 * j + 2], w[4 * j + 3]);
            } else {
#pragma unroll
                for (int i = 0; i < VB; ++i)
                    if (first + i >= 0 && first + i < n) at[i] = value(w + 4 * j, i);
            }
        }
    }
}

// ---------------------------------------------------------------- lookup

// out[t] = scale * table[ids[t] - first], zeros where that is no row.  A warp takes kAhead pieces
// of kSpan columns, of one token or of several, whose loads are all in flight before the first is used.
constexpr int kAhead = 4;

template <typename Tt, typename To, bool SHIFT>
__global__ void __launch_bounds__(kEmbedThreads)
    embed_kernel(const Tt* __restrict__ table, int64_t rows, int64_t cols, int64_t ld, int64_t first,
                 const int32_t* __restrict__ ids, int64_t tokens, float scale, To* __restrict__ out, int64_t out_ld) {
    const int lane = threadIdx.x & 31;
    const int64_t spans = (cols + kSpan - 1) / kSpan, jobs = tokens * spans;
    chain_wait();
    for (int64_t job = ((int64_t)blockIdx.x * kEmbedWarps + (threadIdx.x >> 5)) * kAhead; job < jobs;
         job += (int64_t)gridDim.x * kEmbedWarps * kAhead) {
        Units<Tt, SHIFT> raw[kAhead];
        const Tt* from[kAhead];
        int64_t t[kAhead], c[kAhead];
        int id[kAhead];
        t[0] = job / spans;
        c[0] = job - t[0] * spans;
#pragma unroll
        for (int u = 1; u < kAhead; ++u) {
            const bool over = c[u - 1] + 1 == spans;
            t[u] = t[u - 1] + over;
            c[u] = over ? 0 : c[u - 1] + 1;
        }
#pragma unroll
        for (int u = 0; u < kAhead; ++u) id[u] = t[u] < tokens ? ids[t[u]] : -1;
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            const int64_t r = (int64_t)id[u] - first, col = c[u] * kSpan + lane * 8;
            from[u] = nullptr;
            if (r < 0 || r >= rows || col >= cols) continue;
            from[u] = table + r * ld + col;
            load_units<Tt, SHIFT>(from[u], table + r * ld + cols, raw[u]);
        }
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            if (t[u] >= tokens) break;
            float v[8] = {};
            if (from[u]) unit_values<Tt, SHIFT>(raw[u], from[u], v);
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = from[u] ? v[i] * scale : 0.0f;
            const int64_t left = cols - c[u] * kSpan;
            store_values<To, SHIFT>(out + t[u] * out_ld + c[u] * kSpan + lane * 8, v, (int)(left < kSpan ? left : kSpan), lane);
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
constexpr int kSortAhead = 8;  // pairs a lane holds: up to 65536 tokens are read once a pass

// What the sort leaves for the sums.
struct EmbedOrder {
    int valid;  // tokens that have a row
    int joins;  // chunks whose last row goes on in the next and is joined
};

__device__ __forceinline__ int remote_int(uint32_t addr) {
    int v;
    asm volatile("ld.shared::cluster.b32 %0, [%1];" : "=r"(v) : "r"(addr));
    return v;
}

// pairs: where the sorted (row, token) end up; other: as much scratch.  joins: numbers of the chunks
// (of `chunk` places) whose last row goes on in the next and has more than `few` tokens.
// touched: a bit a row of the table, or NULL.
__global__ void __launch_bounds__(kSortThreads, 1)
    embed_sort_kernel(const int32_t* __restrict__ ids, int64_t n, int64_t first, int64_t rows, int bits, int passes,
                      int2* pairs, int2* other, int chunk, int few, EmbedOrder* order, int* joins, uint32_t* touched) {
    extern __shared__ int shared[];
    const int bins = 1 << bits;
    int* total = shared;                       // [bins] this CTA's, read by the others
    int* hist = shared + bins;                 // [warps][bins]
    __shared__ int warp_sums[kSortWarps];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const unsigned before_me = (1u << lane) - 1;
    const int ctas = (int)gridDim.x, rank = (int)blockIdx.x;
    int* mine_hist = hist + warp * bins;
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
        int2 held[kSortAhead];
        auto fetch = [&](int64_t i0) {
#pragma unroll
            for (int j = 0; j < kSortAhead; ++j) {
                const int64_t i = i0 + 32 * j + lane;
                held[j] = make_int2(-1, 0);
                if (i < end) held[j] = pass ? __ldcg(from + i) : make_int2(ids[i], (int)i);
            }
            if (pass == 0) {
#pragma unroll
                for (int j = 0; j < kSortAhead; ++j) {
                    const int64_t r = (int64_t)held[j].x - first;
                    held[j].x = i0 + 32 * j + lane < end && r >= 0 && r < rows ? (int)r : -1;
                }
            }
        };
        auto digit = [&](int2 p) { return p.x < 0 ? -1 : (p.x >> shift) & (bins - 1); };
        for (int d = lane; d < bins; d += 32) mine_hist[d] = 0;
        __syncwarp();
        for (int64_t i0 = mine; i0 < end; i0 += 32 * kSortAhead) {
            fetch(i0);
#pragma unroll
            for (int j = 0; j < kSortAhead; ++j) {
                if (i0 + 32 * j >= end) break;
                const int d = digit(held[j]);
                const unsigned same = __match_any_sync(kAll, d);
                if (d >= 0 && (same & before_me) == 0) mine_hist[d] += __popc(same);
                __syncwarp();
            }
        }
        __syncthreads();
        const int d = threadIdx.x;
        int c[kSortWarps], sum = 0;
        if (d < bins) {
#pragma unroll
            for (int w = 0; w < kSortWarps; ++w) {
                c[w] = hist[w * bins + d];
                sum += c[w];
            }
            total[d] = sum;
        }
        cluster_sync_all();
        int all = sum, before = 0;
        if (ctas > 1 && d < bins) {
            int v[kSortCtas];
#pragma unroll
            for (int r = 0; r < kSortCtas; ++r) v[r] = remote_int(peer_addr(smem_addr(&total[d]), (uint32_t)r));
            all = 0;
#pragma unroll
            for (int r = 0; r < kSortCtas; ++r) {
                all += v[r];
                before += r < rank ? v[r] : 0;
            }
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
#pragma unroll
            for (int w = 0; w < kSortWarps; ++w) {
                hist[w * bins + d] = run;
                run += c[w];
            }
        }
        __syncthreads();
        for (int64_t i0 = mine; i0 < end; i0 += 32 * kSortAhead) {
            if (per > 32 * kSortAhead) fetch(i0);
#pragma unroll
            for (int j = 0; j < kSortAhead; ++j) {
                if (i0 + 32 * j >= end) break;
                const int dig = digit(held[j]);
                const unsigned same = __match_any_sync(kAll, dig);
                if (dig >= 0) to[mine_hist[dig] + __popc(same & before_me)] = held[j];
                __syncwarp();
                if (dig >= 0 && (same & before_me) == 0) mine_hist[dig] += __popc(same);
                __syncwarp();
            }
        }
        cluster_sync_all();  // the pairs are where the next pass looks for them, and `total` has been read
    }
    if (rank == 0 && threadIdx.x == 0) order->valid = valid;
    for (int64_t p = (int64_t)rank * kSortThreads + threadIdx.x; p < valid; p += (int64_t)ctas * kSortThreads) {
        const int64_t next = (p / chunk + 1) * chunk;
        const int row = __ldcg(&pairs[p].x);
        const int last = p > 0 ? __ldcg(&pairs[p - 1].x) : -1;
        const int cut = next < valid ? __ldcg(&pairs[next].x) : -1, far = p + few < valid ? __ldcg(&pairs[p + few].x) : -1;
        if (last == row) continue;
        if (touched) atomicOr(&touched[row >> 5], 1u << (row & 31));
        if (cut == row && far == row) joins[atomicAdd(&order->joins, 1)] = (int)(p / chunk);
    }
}

// ---------------------------------------------------------------- sums
//
// The sorted places are cut into chunks.  A warp adds up kSpan columns of a chunk's
// tokens, in order.  A row of at most `few` tokens (a chunk's length, 32 at most) is the
// business of the chunk that it begins in, wherever it ends; of a longer one that is cut,
// the part behind a cut goes to heads[chunk] and the part before the first to tails[chunk],
// and embed_join_kernel adds those up, in the order of the chunks.  Rows that no token
// names are written as zeros beside, by warps of their own.
struct EmbedSum {
    const int2* pairs;
    const EmbedOrder* order;
    const int* joins;
    const uint32_t* touched;  // NULL: rows without tokens are left as they are
    float* heads;             // [chunks][pitch]
    float* tails;
    int64_t rows, cols, ld, dout_ld, pitch;
    int chunk, few;
    int accumulate;
    float scale;
};

// table[row] (+)= scale * v: the warp's kSpan columns, of which n are there.
template <typename Tt, bool SHIFT>
__device__ __forceinline__ void add_row(const EmbedSum& g, Tt* table, int row, int64_t c0, int n, const float (&v)[8], int lane) {
    Tt* at = table + (int64_t)row * g.ld + c0 + lane * 8;
    float o[8];
    if (g.accumulate && 8 * lane < n) {
        Units<Tt, SHIFT> raw;
        load_units<Tt, SHIFT>(at, at - lane * 8 + n, raw);
        unit_values<Tt, SHIFT>(raw, at, o);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) o[i] = g.accumulate ? fmaf(g.scale, v[i], o[i]) : g.scale * v[i];
    // (neighbours' loads share units with this lane's stores)
    if (SHIFT) __syncwarp();
    store_values<Tt, SHIFT>(at, o, n, lane);
}

// A row of zeros, by a warp.
template <typename Tt, bool SHIFT>
__device__ __forceinline__ void zero_row(Tt* row, int64_t cols, int lane) {
    const float zero[8] = {};
    for (int64_t c = 0; c < cols; c += kSpan)
        store_values<Tt, SHIFT>(row + c + lane * 8, zero, (int)(cols - c < kSpan ? cols - c : kSpan), lane);
}

// Length of the run of ones from bit 0 on.
__device__ __forceinline__ int run_of(unsigned bits) { return bits == kAll ? 32 : __ffs(~bits) - 1; }

template <typename Td, typename Tt, bool SHIFT>
__global__ void __launch_bounds__(kEmbedThreads)
    embed_sum_kernel(const Td* __restrict__ dout, Tt* __restrict__ table, EmbedSum g) {
    constexpr int B = SHIFT && sizeof(Td) == 4 ? 4 : 8;  // rows in flight
    const int lane = threadIdx.x & 31;
    const int64_t spans = (g.cols + kSpan - 1) / kSpan;
    const int64_t step = (int64_t)gridDim.x * kEmbedWarps;
    chain_wait();
    const int64_t valid = g.order->valid;
    const int64_t chunks = (valid + g.chunk - 1) / g.chunk, jobs = chunks * spans;
    auto key = [&](int64_t p) { return p >= 0 && p < valid ? g.pairs[p].x : -1; };
    int64_t job = (int64_t)blockIdx.x * kEmbedWarps + (threadIdx.x >> 5);
    for (; job < jobs; job += step) {
        const int64_t ch = job / spans, c0 = (job - ch * spans) * kSpan;
        const int n = (int)(g.cols - c0 < kSpan ? g.cols - c0 : kSpan);
        int64_t p0 = ch * g.chunk, p1 = p0 + g.chunk < valid ? p0 + g.chunk : valid;
        // Keys on both sides of both cuts: the first row's tokens before and behind the first cut,
        // the last row's before and behind the second.
        const int b0 = key(p0 - 1 - lane), f0 = key(p0 + lane), b1 = key(p1 - 1 - lane), f1 = key(p1 + lane);
        const int row0 = __shfl_sync(kAll, f0, 0), row1 = __shfl_sync(kAll, b1, 0);
        const int before = run_of(__ballot_sync(kAll, b0 == row0)), here = run_of(__ballot_sync(kAll, f0 == row0));
        const int until = run_of(__ballot_sync(kAll, b1 == row1)), after = run_of(__ballot_sync(kAll, f1 == row1));
        bool head = before > 0, goes_on = after > 0;
        if (head && before + here <= g.few) {  // few: the chunk before has them
            p0 += here;
            head = false;
        }
        if (goes_on && until + after <= g.few) {
            p1 += after;
            goes_on = false;
        }
        if (p0 >= p1) continue;
        float acc[8] = {};
        int row = -1;
        auto flush = [&](bool more) {
            if (head) store_values<float, false>(g.heads + ch * g.pitch + c0 + lane * 8, acc, n, lane);
            else if (more) store_values<float, false>(g.tails + ch * g.pitch + c0 + lane * 8, acc, n, lane);
            else add_row<Tt, SHIFT>(g, table, row, c0, n, acc, lane);
            head = false;
        };
        for (int64_t q = p0; q < p1; q += 32) {
            const int2 mine = q + lane < p1 ? g.pairs[q + lane] : make_int2(-1, 0);
            const int many = (int)(p1 - q < 32 ? p1 - q : 32);
            for (int j0 = 0; j0 < many; j0 += B) {
                Units<Td, SHIFT> raw[B];
#pragma unroll
                for (int b = 0; b < B; ++b) {
                    const Td* from = dout + (int64_t)__shfl_sync(kAll, mine.y, (j0 + b) & 31) * g.dout_ld + c0;
                    if (j0 + b < many && 8 * lane < n) load_units<Td, SHIFT>(from + 8 * lane, from + n, raw[b]);
                }
#pragma unroll
                for (int b = 0; b < B; ++b) {
                    const int r = __shfl_sync(kAll, mine.x, (j0 + b) & 31);
                    const Td* from = dout + (int64_t)__shfl_sync(kAll, mine.y, (j0 + b) & 31) * g.dout_ld + c0;
                    if (j0 + b >= many) break;
                    if (r != row) {
                        if (row >= 0) flush(false);
                        row = r;
#pragma unroll
                        for (int i = 0; i < 8; ++i) acc[i] = 0.0f;
                    }
                    float v[8];
                    unit_values<Td, SHIFT>(raw[b], from, v);
#pragma unroll
                    for (int i = 0; i < 8; ++i) acc[i] += v[i];
                }
            }
        }
        flush(goes_on);
    }
    if (g.touched == nullptr) return;
    // rows without tokens, a warp four of them
    const int64_t groups = (g.rows + 3) / 4;
    for (job -= jobs; job < groups; job += step) {
        const uint32_t bits = g.touched[job >> 3] >> ((job & 7) * 4);
        for (int i = 0; i < 4; ++i) {
            const int64_t r = job * 4 + i;
            if (r < g.rows && !(bits >> i & 1)) zero_row<Tt, SHIFT>(table + r * g.ld, g.cols, lane);
        }
    }
}

// The rows that were cut: tails[c] + heads[c + 1] + ... , a warp a row and kSpan columns; of rows with
// more than kJoinAlone parts every warp of the CTA adds up consecutive ones, and the warps' sums meet
// in shared memory, in order.
constexpr int kJoinAlone = 64;

template <typename Tt, bool SHIFT>
__global__ void __launch_bounds__(kEmbedThreads) embed_join_kernel(Tt* __restrict__ table, EmbedSum g) {
    __shared__ float part[kEmbedWarps][8][32];
    __shared__ int parts_of[kEmbedWarps];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t spans = (g.cols + kSpan - 1) / kSpan;
    chain_wait();
    const int64_t valid = g.order->valid, jobs = g.order->joins * spans;
    for (int64_t job0 = (int64_t)blockIdx.x * kEmbedWarps; job0 < jobs; job0 += (int64_t)gridDim.x * kEmbedWarps) {
        // the sum of parts from..to-1 of a job's, this lane's columns
        auto add_up = [&](int64_t ch, int64_t c, int n, int from, int to, float (&acc)[8]) {
            if (8 * lane >= n) return;
#pragma unroll 8
            for (int k = from; k < to; ++k) {
                const float* src = (k ? g.heads : g.tails) + (ch + k) * g.pitch + c + 8 * lane;
                float v[8];
                load_w<8>(src, v);
#pragma unroll
                for (int i = 0; i < 8; ++i) acc[i] += v[i];
            }
        };
        const int64_t job = job0 + warp;
        int parts = 0;
        if (job < jobs) {
            const int64_t at = job / spans, c = (job - at * spans) * kSpan, ch = g.joins[at];
            const int n = (int)(g.cols - c < kSpan ? g.cols - c : kSpan);
            const int row = g.pairs[(ch + 1) * g.chunk].x;
            for (parts = 1;; parts += 32) {  // how many chunks begin with the row
                const int64_t p = (ch + parts + lane) * g.chunk;
                const int more = run_of(__ballot_sync(kAll, p < valid && g.pairs[p < valid ? p : 0].x == row));
                if (more < 32) {
                    parts += more;
                    break;
                }
            }
            if (parts <= kJoinAlone) {
                float acc[8] = {};
                add_up(ch, c, n, 0, parts, acc);
                add_row<Tt, SHIFT>(g, table, row, c, n, acc, lane);
            }
        }
        if (lane == 0) parts_of[warp] = parts;
        __syncthreads();
        for (int w = 0; w < kEmbedWarps; ++w) {
            const int many = parts_of[w];
            if (many <= kJoinAlone) continue;
            const int64_t at = (job0 + w) / spans, c = (job0 + w - at * spans) * kSpan, ch = g.joins[at];
            const int n = (int)(g.cols - c < kSpan ? g.cols - c : kSpan);
            const int per = (many + kEmbedWarps - 1) / kEmbedWarps;
            float acc[8] = {};
            add_up(ch, c, n, min(many, warp * per), min(many, (warp + 1) * per), acc);
#pragma unroll
            for (int i = 0; i < 8; ++i) part[warp][i][lane] = acc[i];
            __syncthreads();
            if (warp == 0) {
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    acc[i] = 0.0f;
                    for (int x = 0; x < kEmbedWarps; ++x) acc[i] += part[x][i][lane];
                }
                add_row<Tt, SHIFT>(g, table, g.pairs[(ch + 1) * g.chunk].x, c, n, acc, lane);
            }
            __syncthreads();
        }
        __syncthreads();
    }
}

// Few tokens: one launch.  Every CTA has all ids in shared memory; a warp takes a token and kSpan
// columns, adds up all tokens of its row if it is the first of them, and warps left over write the
// rows that no id names.
constexpr int kFewTokens = 256;

template <typename Td, typename Tt, bool SHIFT>
__global__ void __launch_bounds__(kEmbedThreads)
    embed_few_kernel(const Td* __restrict__ dout, const int32_t* __restrict__ ids, int tokens, int64_t first,
                     Tt* __restrict__ table, EmbedSum g) {
    __shared__ int keys[kFewTokens];
    constexpr int B = 4;
    const int lane = threadIdx.x & 31;
    const int64_t spans = (g.cols + kSpan - 1) / kSpan, jobs = tokens * spans;
    const int64_t step = (int64_t)gridDim.x * kEmbedWarps;
    static_assert(kFewTokens <= kEmbedThreads, "a thread a token");
    chain_wait();
    {
        int k = -1;
        if ((int)threadIdx.x < tokens) {
            const int64_t r = (int64_t)ids[threadIdx.x] - first;
            if (r >= 0 && r < g.rows) k = (int)r;
        }
        keys[threadIdx.x] = k;
    }
    __syncthreads();
    int64_t job = (int64_t)blockIdx.x * kEmbedWarps + (threadIdx.x >> 5);
    for (; job < jobs; job += step) {
        const int t = (int)(job / spans);
        const int64_t c0 = (job - t * spans) * kSpan;
        const int n = (int)(g.cols - c0 < kSpan ? g.cols - c0 : kSpan);
        const int row = keys[t];
        if (row < 0) continue;
        bool earlier = false;
        for (int j = lane; j < t; j += 32) earlier |= keys[j] == row;
        if (__any_sync(kAll, earlier)) continue;
        float acc[8] = {};
        for (int j0 = t & ~31; j0 < tokens; j0 += 32) {
            unsigned same = __ballot_sync(kAll, j0 + lane < tokens && keys[(j0 + lane) & (kFewTokens - 1)] == row);
            while (same) {
                Units<Td, SHIFT> raw[B];
                const Td* from[B];
                unsigned left = same;
#pragma unroll
                for (int b = 0; b < B; ++b) {
                    from[b] = nullptr;
                    if (!left) continue;
                    from[b] = dout + (int64_t)(j0 + __ffs(left) - 1) * g.dout_ld + c0;
                    left &= left - 1;
                    if (8 * lane < n) load_units<Td, SHIFT>(from[b] + 8 * lane, from[b] + n, raw[b]);
                }
                same = left;
#pragma unroll
                for (int b = 0; b < B; ++b) {
                    if (!from[b]) break;
                    float v[8];
                    unit_values<Td, SHIFT>(raw[b], from[b], v);
#pragma unroll
                    for (int i = 0; i < 8; ++i) acc[i] += v[i];
                }
            }
        }
        add_row<Tt, SHIFT>(g, table, row, c0, n, acc, lane);
    }
    if (g.accumulate) return;
    const int64_t groups = (g.rows + 3) / 4;
    for (job -= jobs; job < groups; job += step) {
        unsigned bits = 0;
        for (int j = lane; j < tokens; j += 32)
            if (keys[j] >> 2 == job) bits |= 1u << (keys[j] & 3);
        bits = __reduce_or_sync(kAll, bits);
        for (int i = 0; i < 4; ++i) {
            const int64_t r = job * 4 + i;
            if (r < g.rows && !(bits >> i & 1)) zero_row<Tt, SHIFT>(table + r * g.ld, g.cols, lane);
        }
    }
}

// ---------------------------------------------------------------- host side

// Every row begins at a multiple of 16 bytes and has whole vectors of 8 values.
static bool whole(const void* p, int64_t ld, int64_t cols, int bf16) {
    return cols % 8 == 0 && (uintptr_t)p % 16 == 0 && (uintptr_t)ld * (bf16 ? 2 : 4) % 16 == 0;
}

int embed_init_device() {
    const int most = (int)sizeof(int) * (kSortWarps + 1) << kSortBits;
    cudaError_t e = cudaFuncSetAttribute(embed_sort_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, most);
    return e == cudaSuccess ? 0 : set_cuda_error(e, "cudaFuncSetAttribute(embedding order)");
}

static unsigned up_to(int64_t jobs, int per_cta, int64_t most) {
    const int64_t ctas = (jobs + per_cta - 1) / per_cta;
    return (unsigned)(ctas < most ? ctas : most);
}

// f(Ta, Tb, SHIFT) as values of types.
template <typename F>
static cudaError_t by_types(int a_bf16, int b_bf16, bool shift, F f) {
    auto second = [&](auto a) {
        auto third = [&](auto b) { return shift ? f(a, b, std::true_type()) : f(a, b, std::false_type()); };
        return b_bf16 ? third(__nv_bfloat16()) : third(float());
    };
    return a_bf16 ? second(__nv_bfloat16()) : second(float());
}

int embed_launch(const void* table, int bf16, const EmbedArgs& a, const int32_t* ids, void* out, int out_bf16,
                 cudaStream_t s) {
    DeviceState* ds = device_state();
    if (!ds) return -3;
    const bool shift = !(whole(table, a.ld, a.cols, bf16) && whole(out, a.out_ld, a.cols, out_bf16));
    const int64_t jobs = a.tokens * ((a.cols + kSpan - 1) / kSpan);
    // Few pieces are spread over the warps of more CTAs than they fill: each takes kAhead all the same.
    const unsigned grid = up_to(jobs, kEmbedWarps * kAhead, (int64_t)ds->sm_count * 8);
    const cudaError_t e = by_types(bf16, out_bf16, shift, [&](auto t, auto o, auto sh) {
        using Tt = decltype(t);
        using To = decltype(o);
        return launch_chained(embed_kernel<Tt, To, decltype(sh)::value>, dim3(grid), kEmbedThreads, 0, s, 1,
                              static_cast<const Tt*>(table), a.rows, a.cols, a.ld, a.first, ids, a.tokens, a.scale,
                              static_cast<To*>(out), a.out_ld);
    });
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

int embed_backward_launch(const void* dout, int dout_bf16, const EmbedArgs& a, const int32_t* ids, int accumulate,
                          void* table, int bf16, void* work, cudaStream_t s) {
    DeviceState* ds = device_state();
    if (!ds) return -3;
    const EmbedWork w = embed_work(a.tokens, a.rows, a.cols);
    uint8_t* base = static_cast<uint8_t*>(work);
    int2* pairs = reinterpret_cast<int2*>(base + w.pairs);
    EmbedOrder* order = reinterpret_cast<EmbedOrder*>(base);
    int* joins = reinterpret_cast<int*>(base + w.joins);
    uint32_t* touched = accumulate ? nullptr : reinterpret_cast<uint32_t*>(base + w.touched);
    EmbedSum g;
    g.pairs = pairs;
    g.order = order;
    g.joins = joins;
    g.touched = touched;
    g.heads = reinterpret_cast<float*>(base + w.heads);
    g.tails = reinterpret_cast<float*>(base + w.tails);
    g.rows = a.rows;
    g.cols = a.cols;
    g.ld = a.ld;
    g.dout_ld = a.out_ld;
    g.pitch = w.pitch;
    g.chunk = w.chunk;
    g.few = w.chunk < 32 ? w.chunk : 32;
    g.accumulate = accumulate;
    g.scale = a.scale;
    const int64_t spans = (a.cols + kSpan - 1) / kSpan, zeros = accumulate ? 0 : (a.rows + 3) / 4;
    const int64_t most = (int64_t)ds->sm_count * 8;
    const bool shift = !(whole(dout, a.out_ld, a.cols, dout_bf16) && whole(table, a.ld, a.cols, bf16));
    if (a.tokens <= kFewTokens) {
        const unsigned grid = up_to(a.tokens * spans + zeros, kEmbedWarps, most);
        const cudaError_t e = by_types(dout_bf16, bf16, shift, [&](auto d, auto t, auto sh) {
            using Td = decltype(d);
            using Tt = decltype(t);
            return launch_chained(embed_few_kernel<Td, Tt, decltype(sh)::value>, dim3(grid), kEmbedThreads, 0, s, 1,
                                  static_cast<const Td*>(dout), ids, a.tokens, a.first, static_cast<Tt*>(table), g);
        });
        if (e != cudaSuccess) return set_cuda_error(e, "embedding gradient kernel launch");
        count_launch();
        return 0;
    }
    int bits = 1;
    while (bits < 31 && ((int64_t)1 << bits) < a.rows) ++bits;
    const int passes = (bits + kSortBits - 1) / kSortBits;
    bits = (bits + passes - 1) / passes;
    const int ctas = a.tokens <= 4 * kSortThreads ? 1 : kSortCtas;
    cudaError_t e = launch_chained(embed_sort_kernel, dim3(ctas), kSortThreads, sizeof(int) * (kSortWarps + 1) << bits, s,
                                   (unsigned)ctas, ids, a.tokens, a.first, a.rows, bits, passes, pairs,
                                   reinterpret_cast<int2*>(base + w.other), w.chunk, g.few, order, joins, touched);
    if (e != cudaSuccess) return set_cuda_error(e, "embedding order kernel launch");
    count_launch();
    const unsigned grid = up_to(w.chunks * spans + zeros, kEmbedWarps, most);
    const unsigned join_grid = w.chunks > 1 ? up_to((int64_t)(w.chunks - 1) * spans, kEmbedWarps, most) : 0;
    e = by_types(dout_bf16, bf16, shift, [&](auto d, auto t, auto sh) {
        using Td = decltype(d);
        using Tt = decltype(t);
        constexpr bool kShift = decltype(sh)::value;
        cudaError_t err = launch_chained(embed_sum_kernel<Td, Tt, kShift>, dim3(grid), kEmbedThreads, 0, s, 1,
                                         static_cast<const Td*>(dout), static_cast<Tt*>(table), g);
        if (err != cudaSuccess || join_grid == 0) return err;
        count_launch();
        return launch_chained(embed_join_kernel<Tt, kShift>, dim3(join_grid), kEmbedThreads, 0, s, 1, static_cast<Tt*>(table), g);
    });
    if (e != cudaSuccess) return set_cuda_error(e, "embedding gradient kernel launch");
    count_launch();
    return 0;
}

}  // namespace c3
