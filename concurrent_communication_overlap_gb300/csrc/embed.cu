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

// ---------------------------------------------------------------- a warp's part of a row
//
// A warp holds kSpan consecutive values of a row, 8 a lane: W neighbours of them, and again 32 W
// further on, so that every load and store of the warp is one run of W * 32 values.  W is what
// every row's beginning, and its length, are a multiple of: 16 bytes at most.

template <int BYTES>
struct WordOf;
template <>
struct WordOf<2> { using type = uint16_t; };
template <>
struct WordOf<4> { using type = uint32_t; };
template <>
struct WordOf<8> { using type = uint2; };
template <>
struct WordOf<16> { using type = uint4; };

template <typename T, int W>
struct Part {
    using Word = typename WordOf<W * (int)sizeof(T)>::type;
    Word w[8 / W];

    // from p, the place of this lane's first value; n: the row's values from there on.  FULL: all are there.
    template <bool FULL>
    __device__ __forceinline__ void load(const T* p, int n) {
#pragma unroll
        for (int q = 0; q < 8 / W; ++q)
            if (FULL || q * 32 * W < n) w[q] = *reinterpret_cast<const Word*>(p + q * 32 * W);
    }
    __device__ __forceinline__ void values(float (&v)[8]) const {
#pragma unroll
        for (int q = 0; q < 8 / W; ++q) {
            if constexpr (W * sizeof(T) == 2) {
                v[q] = __uint_as_float((uint32_t)w[q] << 16);
            } else {
                uint32_t u[4];
                if constexpr (W * sizeof(T) == 4) u[0] = w[q];
                else u[0] = w[q].x, u[1] = w[q].y;
                if constexpr (W * sizeof(T) == 16) u[2] = w[q].z, u[3] = w[q].w;
#pragma unroll
                for (int i = 0; i < W; ++i) {
                    if constexpr (sizeof(T) == 4) v[q * W + i] = __uint_as_float(u[i]);
                    else v[q * W + i] = __uint_as_float(i & 1 ? u[i / 2] & 0xffff0000u : u[i / 2] << 16);
                }
            }
        }
    }
    template <bool FULL>
    __device__ __forceinline__ static void store(T* p, int n, const float (&v)[8]) {
#pragma unroll
        for (int q = 0; q < 8 / W; ++q) {
            if (!FULL && q * 32 * W >= n) continue;
            if constexpr (W * sizeof(T) == 2) {
                p[q * 32] = __float2bfloat16_rn(v[q]);
            } else {
                uint32_t u[4];
#pragma unroll
                for (int i = 0; i < W * (int)sizeof(T) / 4; ++i) {
                    if constexpr (sizeof(T) == 4) {
                        u[i] = __float_as_uint(v[q * W + i]);
                    } else {
                        const __nv_bfloat162 h = __floats2bfloat162_rn(v[q * W + 2 * i], v[q * W + 2 * i + 1]);
                        u[i] = *reinterpret_cast<const uint32_t*>(&h);
                    }
                }
                Word x;
                if constexpr (W * sizeof(T) == 4) x = u[0];
                else x.x = u[0], x.y = u[1];
                if constexpr (W * sizeof(T) == 16) x.z = u[2], x.w = u[3];
                *reinterpret_cast<Word*>(p + q * 32 * W) = x;
            }
        }
    }
};

// Single bf16 values, stored in pairs: lane l has values 32 i + l, i < 8, of the piece from column c0 on of a row of
// `cols`; row + c0 is aligned to 4 bytes.  Lanes of a pair trade half their values.  ZERO: all are 0.
template <bool ZERO>
__device__ __forceinline__ void store_pairs(__nv_bfloat16* row, int64_t c0, int64_t cols, const float (&v)[8], int lane) {
    const bool odd = lane & 1;
    __nv_bfloat162 h[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (ZERO) {
            h[i] = __floats2bfloat162_rn(0.0f, 0.0f);
        } else {
            const float got = __shfl_xor_sync(kAll, odd ? v[2 * i] : v[2 * i + 1], 1);
            h[i] = __floats2bfloat162_rn(odd ? got : v[2 * i], odd ? v[2 * i + 1] : got);
        }
    }
    const int64_t c = c0 + (odd ? 32 : 0) + (lane & ~1);
    if (c0 >= 0 && c0 + kSpan <= cols) {
        __nv_bfloat162* at = reinterpret_cast<__nv_bfloat162*>(row + c);
#pragma unroll
        for (int i = 0; i < 4; ++i) at[32 * i] = h[i];
        return;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int64_t at = c + 64 * i;
        if (at >= 0 && at + 1 < cols) *reinterpret_cast<__nv_bfloat162*>(row + at) = h[i];
        else if (at >= 0 && at < cols) row[at] = h[i].x;
        else if (at + 1 >= 0 && at + 1 < cols) row[at + 1] = h[i].y;
    }
}

// ---------------------------------------------------------------- lookup

// out[t] = scale * table[ids[t] - first], zeros where that is no row.  A warp takes kAhead pieces
// of kSpan columns, of one token or of several, whose loads are all in flight before the first is used.
//
// Bytes bound it: 65536 tokens x 8192 bf16 take 261 us, 5.4 TB/s of what has to be read and written; tokens
// of a power law name a row again after more than L2 holds, so that memory gives more.  10007 x 2051
// fp32 to bf16, most tokens another shard's, take 14.5 us (floor 6.7): nine rows of ten are zeros, which go by 4-byte
// stores and with the address arithmetic of rows that hold something.
//
// Rows of bf16 of odd length: pieces of a row that begins at no multiple of 4 bytes begin one column
// before, so that pairs of values are aligned where they are stored.
constexpr int kAhead = 2;  // 4 (100 registers): 10007 x 2051 fp32 to bf16 18.4 us, 2: 14.9

template <typename Tt, typename To, int W>
__global__ void __launch_bounds__(kEmbedThreads)
    embed_kernel(const Tt* __restrict__ table, int64_t rows, int64_t cols, int64_t ld, int64_t first,
                 const int32_t* __restrict__ ids, int64_t tokens, float scale, To* __restrict__ out, int64_t out_ld) {
    constexpr bool kPairs = W == 1 && sizeof(To) == 2;
    const int lane = threadIdx.x & 31;
    const int64_t spans = (cols + (kPairs ? 1 : 0) + kSpan - 1) / kSpan, jobs = tokens * spans;
    chain_wait();
    for (int64_t job = ((int64_t)blockIdx.x * kEmbedWarps + (threadIdx.x >> 5)) * kAhead; job < jobs;
         job += (int64_t)gridDim.x * kEmbedWarps * kAhead) {
        Part<Tt, W> part[kAhead];
        int t[kAhead], span[kAhead], id[kAhead];
        bool have[kAhead];
        t[0] = (int)(job / spans);
        span[0] = (int)(job - t[0] * spans);
#pragma unroll
        for (int u = 1; u < kAhead; ++u) {
            const bool over = span[u - 1] + 1 == spans;
            t[u] = t[u - 1] + over;
            span[u] = over ? 0 : span[u - 1] + 1;
        }
        // the piece's first column
        auto column = [&](int u) {
            const int64_t c = (int64_t)span[u] * kSpan;
            return kPairs && ((uintptr_t)(out + t[u] * out_ld) & 2) ? c - 1 : c;
        };
#pragma unroll
        for (int u = 0; u < kAhead; ++u) id[u] = t[u] < tokens ? ids[t[u]] : -1;
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            const int64_t r = (int64_t)id[u] - first;
            have[u] = r >= 0 && r < rows;
            if constexpr (kPairs) {
                const int64_t c0 = column(u), at = c0 + lane;
                const Tt* from = table + r * ld + at;
                if (have[u] && c0 >= 0 && c0 + kSpan <= cols) {
                    part[u].template load<true>(from, 0);
                } else if (have[u]) {
#pragma unroll
                    for (int q = 0; q < 8; ++q)
                        if (at + 32 * q >= 0 && at + 32 * q < cols)
                            part[u].w[q] = *reinterpret_cast<const typename Part<Tt, 1>::Word*>(from + 32 * q);
                }
            } else {
                const int64_t left = cols - column(u);
                const Tt* from = table + r * ld + column(u) + lane * W;
                if (have[u] && left >= kSpan) part[u].template load<true>(from, 0);
                else if (have[u]) part[u].template load<false>(from, (int)left - lane * W);
            }
        }
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            if (t[u] >= tokens) break;
            float v[8] = {};
            if (have[u]) {
                part[u].values(v);
#pragma unroll
                for (int i = 0; i < 8; ++i) v[i] *= scale;
            }
            if constexpr (kPairs) {
                if (have[u]) store_pairs<false>(out + t[u] * out_ld, column(u), cols, v, lane);
                else store_pairs<true>(out + t[u] * out_ld, column(u), cols, v, lane);
            } else {
                const int64_t left = cols - column(u);
                To* to = out + t[u] * out_ld + column(u) + lane * W;
                if (left >= kSpan) Part<To, W>::template store<true>(to, 0, v);
                else Part<To, W>::template store<false>(to, (int)left - lane * W, v);
            }
        }
    }
}

// A row of zeros, by a warp.
template <typename Tt, int W>
__device__ __forceinline__ void zero_row(Tt* row, int64_t cols, int lane) {
    const float zero[8] = {};
    if constexpr (W == 1 && sizeof(Tt) == 2) {
        for (int64_t c = (uintptr_t)row & 2 ? -1 : 0; c < cols; c += kSpan) store_pairs<true>(row, c, cols, zero, lane);
    } else {
        int64_t c = 0;
        for (; c + kSpan <= cols; c += kSpan) Part<Tt, W>::template store<true>(row + c + lane * W, 0, zero);
        if (c < cols) Part<Tt, W>::template store<false>(row + c + lane * W, (int)(cols - c) - lane * W, zero);
    }
}

// What a warp clears at once: up to four rows' kZeroBytes.
constexpr int kZeroBytes = 4096;
template <typename Tt>
struct ZeroPieces {
    int64_t blocks;  // pieces of a row
    __device__ __forceinline__ explicit ZeroPieces(int64_t cols) : blocks((cols + kCols - 1) / kCols) {}
    static constexpr int kCols = kZeroBytes / (int)sizeof(Tt);
    // rows 4 group .. 4 group + 3 but for those whose bit is set in `skip`
    template <int W>
    __device__ __forceinline__ void clear(Tt* table, int64_t rows, int64_t cols, int64_t ld, int64_t group, int64_t block, uint32_t skip,
                                          int lane) const {
        const int64_t c = block * kCols, n = cols - c < kCols ? cols - c : kCols;
#pragma unroll 1
        for (int i = 0; i < 4; ++i)
            if (group * 4 + i < rows && !(skip >> i & 1)) zero_row<Tt, W>(table + (group * 4 + i) * ld + c, n, lane);
    }
};

// ---------------------------------------------------------------- order of the tokens by row
//
// A stable radix sort of (row, token) by row, least digit first, by one cluster in one
// launch.  A token's place in a pass is
//   start[digit] + (of the CTAs before) + (of the warps before) + (before it in its warp),
// whole-number sums, so that the order does not depend on timing.  Tokens without a row
// in the table drop out in the first pass.
//
// Latency bounds it, a step after the other: 16384 tokens of 131072 rows take 14 us in two passes of
// 512 bins, of which loads, votes and counts are 2.6 a pass, the meeting of the CTAs and the sums over
// the bins 2.6, and placing them, with the fence behind it, 2.
constexpr int kSortThreads = 1024;
constexpr int kSortWarps = kSortThreads / 32;
constexpr int kSortBits = 10;  // a digit at most: a thread a bin in the scans
constexpr int kSortCtas = 8;
constexpr int kFew = 32;       // tokens of a row that is never cut: a warp's lanes
constexpr int kSortHeld = 256;  // pairs a warp holds in shared memory: up to 65536 tokens are read once a pass

// What the sort leaves for the sums.
struct EmbedOrder {
    int valid;  // tokens that have a row
    int joins;  // rows that are cut, counted by the sums
};

__device__ __forceinline__ int remote_int(uint32_t addr) {
    int v;
    asm volatile("ld.shared::cluster.b32 %0, [%1];" : "=r"(v) : "r"(addr));
    return v;
}

// pairs: where the sorted (row, token) end up; other: as much scratch.
__device__ __forceinline__ void sort_by_row(const int32_t* __restrict__ ids, int64_t n, int64_t first, int64_t rows, int bits,
                                            int passes, int2* pairs, int2* other, EmbedOrder* order) {
    extern __shared__ int shared[];
    const int bins = 1 << bits;
    int* total = shared;                       // [bins] this CTA's, read by the others
    int* hist = shared + bins;                 // [warps][bins]
    int2* held = reinterpret_cast<int2*>(hist + kSortWarps * bins);  // [warps][kSortHeld] pairs
    uint16_t* places = reinterpret_cast<uint16_t*>(held + kSortWarps * kSortHeld);
    __shared__ int warp_sums[kSortWarps];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const unsigned before_me = (1u << lane) - 1;
    constexpr int ctas = kSortCtas;
    const int rank = (int)cluster_rank();
    int* mine_hist = hist + warp * bins;
    int2* mine_held = held + warp * kSortHeld;
    uint16_t* mine_place = places + warp * kSortHeld;
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
        // kSortHeld pairs from i0 on to shared memory, all loads in flight at once; rows that are none: -1
        auto fetch = [&](int64_t i0) {
            int2 p[kSortHeld / 32];
#pragma unroll
            for (int j = 0; j < kSortHeld / 32; ++j) {
                const int64_t i = i0 + 32 * j + lane;
                p[j] = make_int2(-1, 0);
                if (i < end) p[j] = pass ? __ldcg(from + i) : make_int2(ids[i], (int)i);
            }
#pragma unroll
            for (int j = 0; j < kSortHeld / 32; ++j) {
                if (pass == 0) {
                    const int64_t r = (int64_t)p[j].x - first;
                    p[j].x = i0 + 32 * j + lane < end && r >= 0 && r < rows ? (int)r : -1;
                }
                mine_held[32 * j + lane] = p[j];
            }
            __syncwarp();
        };
        // A lane's place among those of its digit that the warp has seen, which `mine_hist` counts.  The lanes
        // of the same digit are found by a vote a bit.
        auto place = [&](int d) {
            unsigned same = __ballot_sync(kAll, d >= 0);
#pragma unroll
            for (int b = 0; b < kSortBits; ++b) {
                const bool bit = (d >> b) & 1;
                const unsigned one = __ballot_sync(kAll, bit);
                same &= bit ? one : ~one;
            }
            int at = 0;
            if (d >= 0) at = mine_hist[d];
            __syncwarp();
            if (d >= 0 && (same & before_me) == 0) mine_hist[d] = at + __popc(same);
            __syncwarp();
            return at + __popc(same & before_me);
        };
        auto digit = [&](int2 p) { return p.x < 0 ? -1 : (p.x >> shift) & (bins - 1); };
        auto groups = [&](int64_t i0) { return (int)((end - i0 + 31) / 32 < kSortHeld / 32 ? (end - i0 + 31) / 32 : kSortHeld / 32); };
        const bool again = per > kSortHeld;
        for (int d = lane; d < bins; d += 32) mine_hist[d] = 0;
        __syncwarp();
        // (Loops are left rolled: the kernel runs each instruction a few times, and fetching them counts.)
#pragma unroll 1
        for (int64_t i0 = mine; i0 < end; i0 += kSortHeld) {
            fetch(i0);
            const int many = groups(i0);
#pragma unroll 1
            for (int j = 0; j < many; ++j) {
                const int at = place(digit(mine_held[32 * j + lane]));
                if (!again) mine_place[32 * j + lane] = (uint16_t)at;
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
        if (d < bins) {
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
#pragma unroll 1
        for (int64_t i0 = mine; i0 < end; i0 += kSortHeld) {
            if (again) fetch(i0);
            const int many = groups(i0);
#pragma unroll 1
            for (int j = 0; j < many; ++j) {
                const int2 p = mine_held[32 * j + lane];
                const int dig = digit(p);
                const int at = again ? place(dig) : dig >= 0 ? mine_hist[dig] + mine_place[32 * j + lane] : 0;
                if (dig < 0) continue;
                to[at] = p;
            }
            __syncwarp();
        }
        cluster_sync_all();  // the pairs are where the next pass looks for them, and `total` has been read
    }
    if (rank == 0 && threadIdx.x == 0) order->valid = valid;
}

// By clusters 1.. of the sort's launch, while latency bounds the sort: which rows no id names, a bit a row for the
// sums, and zeros into the first of them.  Each cluster has a run of rows; its CTAs mark what an eighth of the ids
// name each, in shared memory, and put an eighth of the words together.  Rows of the first `fill` words of a CTA get
// their zeros here, and bits that say so.  kFillBits rows at a time.
constexpr int kFillBits = 1 << 18;  // 32 KB of bits

template <typename Tt, int W>
__device__ __forceinline__ void mark_and_fill(const int32_t* __restrict__ ids, int64_t n, int64_t first, Tt* table, int64_t rows,
                                              int64_t cols, int64_t ld, int fill, uint32_t* named) {
    extern __shared__ int shared[];
    unsigned* marks = reinterpret_cast<unsigned*>(shared);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, rank = (int)cluster_rank();
    const int64_t clusters = gridDim.x / kSortCtas - 1, mine = blockIdx.x / kSortCtas - 1;
    const int64_t per = ((rows + 31) / 32 + clusters - 1) / clusters * 32, last = (mine + 1) * per < rows ? (mine + 1) * per : rows;
    for (int64_t r0 = mine * per; r0 < last; r0 += kFillBits) {
        const int many = (int)(last - r0 < kFillBits ? last - r0 : kFillBits), words = (many + 31) / 32;
        for (int i = threadIdx.x; i < words; i += kSortThreads) marks[i] = 0;
        __syncthreads();
        const int64_t base = first + r0, step = (int64_t)kSortCtas * kSortThreads;
        for (int64_t i0 = (int64_t)rank * kSortThreads + threadIdx.x; i0 < n; i0 += 8 * step) {
            int64_t r[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) r[j] = i0 + j * step < n ? (int64_t)ids[i0 + j * step] - base : -1;
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (r[j] >= 0 && r[j] < many) atomicOr(&marks[r[j] >> 5], 1u << (r[j] & 31));
        }
        cluster_sync_all();
        // this CTA's words, of all eight CTAs' marks
        const int share = (words + kSortCtas - 1) / kSortCtas, from = rank * share, end = min(words, from + share);
        for (int w = from + warp; w < end; w += kSortWarps) {
            const unsigned some = lane < kSortCtas ? (unsigned)remote_int(peer_addr(smem_addr(&marks[w]), (uint32_t)lane)) : 0u;
            const unsigned bits = __reduce_or_sync(kAll, some);
            if (lane == 0) named[(r0 >> 5) + w] = w - from < fill ? kAll : bits;
        }
        __syncwarp();
        // zeros: the rows of the first words, a warp a row
        for (int i = warp; i < 32 * min(fill, end - from); i += kSortWarps) {
            const int w = from + (i >> 5), row = w * 32 + (i & 31);
            const unsigned some = lane < kSortCtas ? (unsigned)remote_int(peer_addr(smem_addr(&marks[w]), (uint32_t)lane)) : 0u;
            const unsigned bits = __reduce_or_sync(kAll, some);
            if (row < many && !(bits >> (i & 31) & 1)) zero_row<Tt, W>(table + (r0 + row) * ld, cols, lane);
        }
        cluster_sync_all();  // the marks have been read
    }
}

template <typename Tt, int W>
__global__ void __launch_bounds__(kSortThreads, 1)
    embed_sort_kernel(const int32_t* __restrict__ ids, int64_t n, int64_t first, int64_t rows, int bits, int passes,
                      int2* pairs, int2* other, EmbedOrder* order, Tt* table, int64_t cols, int64_t ld, int fill, uint32_t* named) {
    chain_wait();
    if (blockIdx.x < kSortCtas) sort_by_row(ids, n, first, rows, bits, passes, pairs, other, order);
    else mark_and_fill<Tt, W>(ids, n, first, table, rows, cols, ld, fill, named);
}

// ---------------------------------------------------------------- order of some thousands of tokens
//
// Up to kRankTokens tokens every SM has all rows in shared memory and counts: a token's place is the number of tokens
// of lower rows, and of its own row before it.  That is n^2 comparisons in place of the sort's chain of latencies: gradients
// of 4096 tokens into 30000 x 100 bf16 take 22.5 us this way and 26.1 sorted, of 2048 19.1 and 23.6, but of 8192 29.9
// and 26.0.  Each CTA then finds which of its share of the rows are named, and clears some, as the sort's clusters do.
constexpr int kRankTokens = 4096;
constexpr int kRankRows = 1 << 16;  // of a CTA's rows at a time: 8 KB of bits

template <typename Tt, int W>
__global__ void __launch_bounds__(kSortThreads, 1)
    embed_rank_kernel(const int32_t* __restrict__ ids, int n, int64_t first, int64_t rows, int2* pairs, EmbedOrder* order,
                      Tt* table, int64_t cols, int64_t ld, int fill, uint32_t* named) {
    __shared__ __align__(16) int keys[kRankTokens];
    __shared__ unsigned marks[kRankRows / 32];
    constexpr int kNone = 0x7FFFFFFF;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int chunks = (n + 127) / 128;
    chain_wait();
    for (int i = threadIdx.x; i < chunks * 128; i += kSortThreads) {
        const int64_t r = i < n ? (int64_t)ids[i] - first : -1;
        keys[i] = r >= 0 && r < rows ? (int)r : kNone;
    }
    __syncthreads();
    if (blockIdx.x == 0 && warp == 0) {
        int valid = 0;
        for (int i = lane; i < n; i += 32) valid += keys[i] != kNone;
        valid = __reduce_add_sync(kAll, valid);
        if (lane == 0) {
            order->valid = valid;
            order->joins = 0;
        }
    }
    for (int i = (int)blockIdx.x * kSortWarps + warp; i < n; i += (int)gridDim.x * kSortWarps) {
        const int key = keys[i];
        if (key == kNone) continue;
        int below = 0;
        const int4* k4 = reinterpret_cast<const int4*>(keys) + lane;
        int c = 0;
#pragma unroll 4
        for (; c < i / 128; ++c) {
            const int4 k = k4[c * 32];
            below += (k.x <= key) + (k.y <= key) + (k.z <= key) + (k.w <= key);
        }
        {
            const int4 k = k4[c * 32];
            const int j = c * 128 + lane * 4;
            below += (k.x < key + (j < i)) + (k.y < key + (j + 1 < i)) + (k.z < key + (j + 2 < i)) + (k.w < key + (j + 3 < i));
        }
#pragma unroll 4
        for (++c; c < chunks; ++c) {
            const int4 k = k4[c * 32];
            below += (k.x < key) + (k.y < key) + (k.z < key) + (k.w < key);
        }
        below = __reduce_add_sync(kAll, below);
        if (lane == 0) pairs[below] = make_int2(key, i);
    }
    if (!named) return;
    const int64_t words = (rows + 31) / 32, share = (words + gridDim.x - 1) / gridDim.x;
    const int64_t last = (blockIdx.x + 1) * share < words ? (blockIdx.x + 1) * share : words;
    for (int64_t w0 = blockIdx.x * share; w0 < last; w0 += kRankRows / 32) {
        const int many = (int)(last - w0 < kRankRows / 32 ? last - w0 : kRankRows / 32);
        for (int w = threadIdx.x; w < many; w += kSortThreads) marks[w] = 0;
        __syncthreads();
        for (int i = threadIdx.x; i < n; i += kSortThreads) {
            const int64_t r = (int64_t)keys[i] - w0 * 32;
            if (keys[i] != kNone && r >= 0 && r < many * 32) atomicOr(&marks[r >> 5], 1u << (r & 31));
        }
        __syncthreads();
        const int clear = min(fill, many);
        for (int w = threadIdx.x; w < many; w += kSortThreads) named[w0 + w] = w < clear ? kAll : marks[w];
        for (int i = warp; i < 32 * clear; i += kSortWarps) {
            const int64_t row = w0 * 32 + i;
            if (row < rows && !(marks[i >> 5] >> (i & 31) & 1)) zero_row<Tt, W>(table + row * ld, cols, lane);
        }
        __syncthreads();
    }
}

// ---------------------------------------------------------------- sums
//
// The sorted places are cut into chunks.  A warp adds up kSpan columns of a chunk's
// tokens, in order.  A row of at most kFew tokens is the business of the chunk that it begins
// in, wherever it ends; of a longer one that is cut, the part behind a cut goes to
// heads[chunk] and the part before the first to tails[chunk], and embed_join_kernel adds
// those up, in the order of the chunks.  (With every row cut at chunks of 16 the joins of 40009
// tokens of a power law took 48 us, these 7.)  Eight tokens' rows are in flight a warp, four and
// the table's where it is added to, whose loads one after the other took 28 us of 53.
//
// Bytes bound it: 16384 x 8192 bf16 into 131072 rows 376 us at 6.3 TB/s, of 397 in all.
struct EmbedSum {
    const int2* pairs;
    EmbedOrder* order;
    int* joins;               // the chunks that such rows begin in
    float* heads;             // [chunks][pitch]
    float* tails;
    int64_t rows, cols, ld, dout_ld, pitch;
    const uint32_t* named;    // a bit a row that needs no zeros (any more)
    int chunk;
    int accumulate;
    float scale;
};

// Partial sums in fp32: as the lanes hold them, W neighbours in units of 16 bytes at most.
template <int W>
struct Parked {
    static constexpr int V = W < 4 ? W : 4;
    __device__ __forceinline__ static void store(float* p, int n, const float (&v)[8]) {
#pragma unroll
        for (int q = 0; q < 8 / W; ++q) {
            if (q * 32 * W >= n) continue;
#pragma unroll
            for (int i = 0; i < W; i += V) {
                if constexpr (V == 4) *reinterpret_cast<float4*>(p + q * 32 * W + i) = make_float4(v[q * W + i], v[q * W + i + 1], v[q * W + i + 2], v[q * W + i + 3]);
                else if constexpr (V == 2) *reinterpret_cast<float2*>(p + q * 32 * W + i) = make_float2(v[q * W + i], v[q * W + i + 1]);
                else p[q * 32 * W + i] = v[q * W + i];
            }
        }
    }
    __device__ __forceinline__ static void load(const float* p, int n, float (&v)[8]) {
#pragma unroll
        for (int q = 0; q < 8 / W; ++q) {
            const bool have = q * 32 * W < n;
#pragma unroll
            for (int i = 0; i < W; i += V) {
                if constexpr (V == 4) {
                    const float4 x = have ? *reinterpret_cast<const float4*>(p + q * 32 * W + i) : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                    v[q * W + i] = x.x, v[q * W + i + 1] = x.y, v[q * W + i + 2] = x.z, v[q * W + i + 3] = x.w;
                } else if constexpr (V == 2) {
                    const float2 x = have ? *reinterpret_cast<const float2*>(p + q * 32 * W + i) : make_float2(0.0f, 0.0f);
                    v[q * W + i] = x.x, v[q * W + i + 1] = x.y;
                } else {
                    v[q * W + i] = have ? p[q * 32 * W + i] : 0.0f;
                }
            }
        }
    }
};

// table[row] (+)= scale * v: the warp's kSpan columns, of which n are there.
template <typename Tt, int W>
__device__ __forceinline__ void add_row(const EmbedSum& g, Tt* table, int row, int64_t c0, int n, const float (&v)[8], int lane) {
    Tt* at = table + (int64_t)row * g.ld + c0 + lane * W;
    float o[8];
    if (g.accumulate) {
        Part<Tt, W> old;
        old.template load<false>(at, n - lane * W);
        old.values(o);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) o[i] = g.accumulate ? fmaf(g.scale, v[i], o[i]) : g.scale * v[i];
    Part<Tt, W>::template store<false>(at, n - lane * W, o);
}

// Length of the run of ones from bit 0 on.
__device__ __forceinline__ int run_of(unsigned bits) { return bits == kAll ? 32 : __ffs(~bits) - 1; }

template <typename Td, typename Tt, int W, bool ACCUMULATE>
__global__ void __launch_bounds__(kEmbedThreads, 2)
    embed_sum_kernel(const Td* __restrict__ dout, Tt* __restrict__ table, EmbedSum g) {
    // rows in flight; of a table that is added to, its rows too
    constexpr int B = ACCUMULATE ? 4 : 8;
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
        if (head && before + here <= kFew) {  // few: the chunk before has them
            p0 += here;
            head = false;
        }
        if (goes_on && until + after <= kFew) {
            p1 += after;
            goes_on = false;
        }
        float acc[8] = {};
        for (int64_t q = p0; q < p1; q += 32) {
            const int2 mine = q + lane < p1 ? g.pairs[q + lane] : make_int2(-1, 0);
            const int many = (int)(p1 - q < 32 ? p1 - q : 32);
            // tokens that are the last of their row here
            const unsigned ends = __ballot_sync(kAll, q + lane + 1 >= p1 || g.pairs[q + lane + 1].x != mine.x);
            for (int j0 = 0; j0 < many; j0 += B) {
                Part<Td, W> held[B];
                Part<Tt, W> old[ACCUMULATE ? B : 1];
#pragma unroll
                for (int b = 0; b < B; ++b) {
                    const int64_t t = __shfl_sync(kAll, mine.y, (j0 + b) & 31), r = __shfl_sync(kAll, mine.x, (j0 + b) & 31);
                    if (j0 + b >= many) continue;
                    const Td* from = dout + t * g.dout_ld + c0 + lane * W;
                    if (n == kSpan) held[b].template load<true>(from, 0);
                    else held[b].template load<false>(from, n - lane * W);
                    if (ACCUMULATE && (ends >> (j0 + b) & 1)) old[b].template load<false>(table + r * g.ld + c0 + lane * W, n - lane * W);
                }
#pragma unroll
                for (int b = 0; b < B; ++b) {
                    const int64_t r = __shfl_sync(kAll, mine.x, (j0 + b) & 31);
                    if (j0 + b >= many) break;
                    float v[8];
                    held[b].values(v);
#pragma unroll
                    for (int i = 0; i < 8; ++i) acc[i] += v[i];
                    if (!(ends >> (j0 + b) & 1)) continue;
                    const bool tail = goes_on && q + j0 + b + 1 == p1;
                    if (head || tail) {
                        if (!head && c0 == 0 && lane == 0) g.joins[atomicAdd(&g.order->joins, 1)] = (int)ch;
                        Parked<W>::store((head ? g.heads : g.tails) + ch * g.pitch + c0 + lane * W, n - lane * W, acc);
                    } else {
                        if (ACCUMULATE) old[b].values(v);
#pragma unroll
                        for (int i = 0; i < 8; ++i) v[i] = ACCUMULATE ? fmaf(g.scale, acc[i], v[i]) : g.scale * acc[i];
                        Part<Tt, W>::template store<false>(table + r * g.ld + c0 + lane * W, n - lane * W, v);
                    }
                    head = false;
#pragma unroll
                    for (int i = 0; i < 8; ++i) acc[i] = 0.0f;
                }
            }
        }
    }
    // rows without tokens that the sort's launch has left, a warp four of them
    if (ACCUMULATE) return;
    const ZeroPieces<Tt> zero(g.cols);
    const int64_t pieces = (g.rows + 3) / 4 * zero.blocks;
    for (job -= jobs; job < pieces; job += step) {
        const int64_t group = job / zero.blocks;
        zero.template clear<W>(table, g.rows, g.cols, g.ld, group, job - group * zero.blocks, g.named[group >> 3] >> ((group & 7) * 4), lane);
    }
}

// The rows that were cut: tails[c] + heads[c + 1] + ... .  A CTA takes a row and kSpan columns; its warps
// add up consecutive parts, and the warps' sums meet in shared memory, in order.
//
// Latency bounds it.  Rows of up to kJoinSpans spans: 16 warps a row and four parts in flight each, since few rows make few
// CTAs (32768 tokens of a power law, 256 columns: 36 us in all, and 43 with 8 warps; one row for all of them 67 and
// 170).  Longer rows: 8 warps and eight parts, of which more rows run at once (16384 x 8192 bf16 9 us less in all than with 16
// warps; 32768 x 4096 129 and 136; 1024 columns 55 and 54, 2048 81 either way).  Told to leave room for a second CTA or none, the
// compiler took 120 registers in place of 48 to 73 for the latter, and 32768 x 4096 133 us.
constexpr int kJoinSpans = 4;
template <typename Tt, int W, int WARPS>
__global__ void __launch_bounds__(WARPS * 32, WARPS == 16 ? 2 : 0) embed_join_kernel(Tt* __restrict__ table, EmbedSum g) {
    constexpr int B = WARPS == 16 ? 4 : 8;  // parts in flight
    __shared__ float part[WARPS][8][32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t spans = (g.cols + kSpan - 1) / kSpan;
    chain_wait();
    const int64_t valid = g.order->valid, jobs = g.order->joins * spans;
    for (int64_t job = blockIdx.x; job < jobs; job += gridDim.x) {
        const int64_t at = job / spans, c = (job - at * spans) * kSpan, ch = g.joins[at];
        const int n = (int)(g.cols - c < kSpan ? g.cols - c : kSpan);
        const int row = g.pairs[(ch + 1) * g.chunk].x;
        // how many chunks begin with the row: the next 32 first, then by steps that bring what is left down to a 32nd
        auto begins = [&](int64_t k) {
            const int64_t p = (ch + k) * g.chunk;
            return p < valid && g.pairs[p].x == row;
        };
        int more = run_of(__ballot_sync(kAll, begins(1 + lane))), parts = 1 + more;
        if (more == 32) {
            int left = (int)((valid - 1) / g.chunk - ch) - 32;  // chunks behind those
            while (left > 0) {
                const int apart = (left + 31) / 32, probe = (lane + 1) * apart;
                more = run_of(__ballot_sync(kAll, probe <= left && begins(parts - 1 + probe)));
                parts += more * apart;
                left = min(left - more * apart, apart - 1);
            }
        }
        const int per = (parts + WARPS - 1) / WARPS, to = min(parts, (warp + 1) * per);
        float acc[8] = {};
#pragma unroll 1
        for (int k0 = warp * per; k0 < to; k0 += B) {
            float v[B][8];
#pragma unroll
            for (int j = 0; j < B; ++j)
                Parked<W>::load((k0 + j ? g.heads : g.tails) + (ch + k0 + j) * g.pitch + c + lane * W, k0 + j < to ? n - lane * W : 0, v[j]);
#pragma unroll
            for (int j = 0; j < B; ++j)
#pragma unroll
                for (int i = 0; i < 8; ++i) acc[i] += v[j][i];
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) part[warp][i][lane] = acc[i];
        __syncthreads();
        if (warp == 0) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                acc[i] = 0.0f;
#pragma unroll
                for (int x = 0; x < WARPS; ++x) acc[i] += part[x][i][lane];
            }
            add_row<Tt, W>(g, table, row, c, n, acc, lane);
        }
        __syncthreads();
    }
}

// Few tokens: one launch.  Every CTA has all ids in shared memory; a warp takes a token and kSpan
// columns and adds up all tokens of its row, if it is the first of them.  A row of more than kAlone tokens
// (padding that has an id, say) is left for all the CTA's warps, which add up an eighth of the tokens each; the eighths
// meet in shared memory, in order.  Rows that no id names are cleared by what follows.
//
// The more tokens and spans, the longer the warps look for their rows'.  This way and ordered first: 512 tokens into
// 9000 x 1001 bf16 9.6 us and 11.2, 768 12.5 and 11.5; into 6250 x 4096 fp32, 16 spans, 256 18.3 and 19.8, 512 23.5 and 20.4.
constexpr int kFewTokens = 512, kFewJobs = 4096;
constexpr int kAlone = 32;

template <typename Td, typename Tt, int W>
__global__ void __launch_bounds__(kEmbedThreads)
    embed_few_kernel(const Td* __restrict__ dout, const int32_t* __restrict__ ids, int tokens, int64_t first,
                     Tt* __restrict__ table, EmbedSum g) {
    __shared__ int keys[kFewTokens];
    __shared__ float part[kEmbedWarps][8][32];
    __shared__ int crowd[kEmbedWarps];  // each warp's token whose row has many, or -1
    constexpr int B = 4;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t spans = (g.cols + kSpan - 1) / kSpan, jobs = tokens * spans;
    const int64_t step = (int64_t)gridDim.x * kEmbedWarps;
    chain_wait();
    for (int i = threadIdx.x; i < tokens; i += kEmbedThreads) {
        const int64_t r = (int64_t)ids[i] - first;
        keys[i] = r >= 0 && r < g.rows ? (int)r : -1;
    }
    __syncthreads();
    int64_t job0 = (int64_t)blockIdx.x * kEmbedWarps;
    for (; job0 < jobs; job0 += step) {
        auto token = [&](int w) { return (int)((job0 + w) / spans); };
        const int t = job0 + warp < jobs ? token(warp) : 0;
        int row = job0 + warp < jobs ? keys[t] : -1, many = 0;
        for (int j0 = 0; row >= 0 && j0 < tokens; j0 += 32) {
            const unsigned same = __ballot_sync(kAll, j0 + lane < tokens && keys[(j0 + lane) & (kFewTokens - 1)] == row);
            const unsigned earlier = j0 + 32 <= t ? kAll : j0 <= t ? (1u << (t - j0)) - 1 : 0u;
            if (same & earlier) row = -1;  // not the first
            many += __popc(same);
        }
        const bool alone = row >= 0 && many <= kAlone;
        if (lane == 0) crowd[warp] = row >= 0 && !alone ? t : -1;
        // turn 0: a warp's own; then the crowds of all warps, one after the other
#pragma unroll 1
        for (int turn = 0; turn <= kEmbedWarps; ++turn) {
            const int per = (tokens + kEmbedWarps - 1) / kEmbedWarps;
            int from = t, to = alone ? tokens : 0, w = warp;
            if (turn > 0) {
                if (turn == 1) __syncthreads();
                w = turn - 1;
                if (crowd[w] < 0) continue;
                row = keys[crowd[w]];
                from = warp * per;
                to = min(tokens, from + per);
            }
            const int64_t c0 = (job0 + w - token(w) * spans) * kSpan;
            const int n = (int)(g.cols - c0 < kSpan ? g.cols - c0 : kSpan);
            float acc[8] = {};
            for (int j0 = from; j0 < to; j0 += 32) {
                unsigned same = __ballot_sync(kAll, j0 + lane < to && keys[(j0 + lane) & (kFewTokens - 1)] == row);
                while (same) {
                    Part<Td, W> raw[B];
                    const Td* at[B];
                    unsigned left = same;
#pragma unroll
                    for (int b = 0; b < B; ++b) {
                        at[b] = nullptr;
                        if (!left) continue;
                        at[b] = dout + (int64_t)(j0 + __ffs(left) - 1) * g.dout_ld + c0;
                        left &= left - 1;
                        raw[b].template load<false>(at[b] + lane * W, n - lane * W);
                    }
                    same = left;
#pragma unroll
                    for (int b = 0; b < B; ++b) {
                        if (!at[b]) break;
                        float v[8];
                        raw[b].values(v);
#pragma unroll
                        for (int i = 0; i < 8; ++i) acc[i] += v[i];
                    }
                }
            }
            if (turn > 0) {
#pragma unroll
                for (int i = 0; i < 8; ++i) part[warp][i][lane] = acc[i];
                __syncthreads();
                if (warp == 0) {
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        acc[i] = 0.0f;
#pragma unroll
                        for (int x = 0; x < kEmbedWarps; ++x) acc[i] += part[x][i][lane];
                    }
                }
            }
            if (turn == 0 ? alone : warp == 0) add_row<Tt, W>(g, table, row, c0, n, acc, lane);
            if (turn > 0) __syncthreads();
        }
        __syncthreads();  // `crowd` has been read
    }
    int64_t job = job0 + warp;  // past the sums' jobs, whose number is made up to whole CTAs
    if (g.accumulate) return;
    const ZeroPieces<Tt> zero(g.cols);
    const int64_t pieces = (g.rows + 3) / 4 * zero.blocks;
    for (job -= (jobs + kEmbedWarps - 1) / kEmbedWarps * kEmbedWarps; job < pieces; job += step) {
        const int64_t group = job / zero.blocks;
        unsigned bits = 0;
        for (int j = lane; j < tokens; j += 32)
            if (keys[j] >> 2 == group) bits |= 1u << (keys[j] & 3);
        zero.template clear<W>(table, g.rows, g.cols, g.ld, group, job - group * zero.blocks, __reduce_or_sync(kAll, bits), lane);
    }
}

// ---------------------------------------------------------------- host side

// Rows as they lie in memory: base, row distance, type.
struct Lines {
    const void* p;
    int64_t ld;
    int bf16;
    bool fits(int w) const {
        const uintptr_t unit = (uintptr_t)w * (bf16 ? 2 : 4);
        return unit <= 16 && (uintptr_t)p % unit == 0 && ld % w == 0;
    }
};
// Neighbouring values that a lane loads at once: 16 bytes of the wider type, less where rows do not
// begin at, or are not whole, units of so many.
static int width(int64_t cols, const Lines& x, const Lines& y) {
    int w = 8;
    while (w > 1 && (cols % w || !x.fits(w) || !y.fits(w))) w /= 2;
    return w;
}

static size_t sort_smem(int bits) {
    return (sizeof(int) * (kSortWarps + 1) << bits) + (size_t)kSortWarps * kSortHeld * (sizeof(int2) + sizeof(uint16_t));
}

template <typename Tt, int W>
static cudaError_t sort_attr(int* clusters) {
    const size_t most = sort_smem(kSortBits);
    cudaError_t e = cudaFuncSetAttribute(embed_sort_kernel<Tt, W>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)most);
    if (e != cudaSuccess || !clusters) return e;
    cudaLaunchConfig_t c{};
    c.gridDim = dim3(kSortCtas);
    c.blockDim = dim3(kSortThreads);
    c.dynamicSmemBytes = most;
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = kSortCtas;
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    c.attrs = &attr;
    c.numAttrs = 1;
    return cudaOccupancyMaxActiveClusters(clusters, embed_sort_kernel<Tt, W>, &c);
}

int embed_init_device(int* clusters) {
    cudaError_t e = sort_attr<float, 1>(clusters);
    if (e == cudaSuccess) e = sort_attr<float, 2>(nullptr);
    if (e == cudaSuccess) e = sort_attr<float, 4>(nullptr);
    if (e == cudaSuccess) e = sort_attr<__nv_bfloat16, 1>(nullptr);
    if (e == cudaSuccess) e = sort_attr<__nv_bfloat16, 2>(nullptr);
    if (e == cudaSuccess) e = sort_attr<__nv_bfloat16, 4>(nullptr);
    if (e == cudaSuccess) e = sort_attr<__nv_bfloat16, 8>(nullptr);
    return e == cudaSuccess ? 0 : set_cuda_error(e, "cudaFuncSetAttribute(embedding order)");
}

static unsigned up_to(int64_t jobs, int per_cta, int64_t most) {
    const int64_t ctas = (jobs + per_cta - 1) / per_cta;
    return (unsigned)(ctas < most ? ctas : most);
}

// f(Ta, Tb, W) as values of types.
template <typename F>
static cudaError_t by_types(int a_bf16, int b_bf16, int w, F f) {
    auto second = [&](auto a) {
        auto third = [&](auto b) {
            switch (w) {
                case 8:
                    if constexpr (sizeof(a) == 2 && sizeof(b) == 2) return f(a, b, std::integral_constant<int, 8>());
                    [[fallthrough]];
                case 4: return f(a, b, std::integral_constant<int, 4>());
                case 2: return f(a, b, std::integral_constant<int, 2>());
                default: return f(a, b, std::integral_constant<int, 1>());
            }
        };
        return b_bf16 ? third(__nv_bfloat16()) : third(float());
    };
    return a_bf16 ? second(__nv_bfloat16()) : second(float());
}

int embed_launch(const void* table, int bf16, const EmbedArgs& a, const int32_t* ids, void* out, int out_bf16,
                 cudaStream_t s) {
    DeviceState* ds = device_state();
    if (!ds) return -3;
    const int w = width(a.cols, {table, a.ld, bf16}, {out, a.out_ld, out_bf16});
    const int64_t jobs = a.tokens * ((a.cols + 1 + kSpan - 1) / kSpan);  // (one more column where pairs begin before a row)
    // A dozen turns a warp where there are enough: 65536 x 8192 bf16 takes 282 us with as many CTAs as run at
    // once, 261 with ten times as many, whose runs in memory are nearer together, and 320 with one for each turn.
    const int64_t some = (int64_t)ds->sm_count * 8, dozen = jobs / (12 * kEmbedWarps * kAhead);
    const unsigned grid = up_to(jobs, kEmbedWarps * kAhead, dozen > some ? dozen < (1 << 30) ? dozen : 1 << 30 : some);
    const cudaError_t e = by_types(bf16, out_bf16, w, [&](auto t, auto o, auto wide_of) {
        using Tt = decltype(t);
        using To = decltype(o);
        return launch_chained(embed_kernel<Tt, To, decltype(wide_of)::value>, dim3(grid), kEmbedThreads, 0, s, 1,
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
    size_t pairs, other, joins, named, heads, tails, bytes;
};

static EmbedWork embed_work(int64_t tokens, int64_t rows, int64_t cols) {
    EmbedWork w;
    const int64_t spans = (cols + kSpan - 1) / kSpan;
    // Enough for every warp that runs at once to have two, down to 8 tokens: a chunk's rows are written one after the
    // other (2048 tokens into 9000 x 1001 bf16: chunks of 32 20.8 us in all).  Above 32 tokens more of them cost less.
    constexpr int64_t kEnough = 32 * 152, kMost = 16384;  // 152 SMs of two CTAs of eight warps
    w.chunk = 8;
    while ((tokens + w.chunk - 1) / w.chunk * spans > (w.chunk < 32 ? kEnough : kMost) && w.chunk < (1 << 20)) w.chunk *= 2;
    static_assert(kFew == 32, "a warp's votes find a short row's ends");
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
    w.named = part((size_t)(rows + 31) / 32 * sizeof(uint32_t));
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
    EmbedSum g;
    g.pairs = pairs;
    g.order = order;
    g.joins = joins;
    g.heads = reinterpret_cast<float*>(base + w.heads);
    g.tails = reinterpret_cast<float*>(base + w.tails);
    g.rows = a.rows;
    g.cols = a.cols;
    g.ld = a.ld;
    g.dout_ld = a.out_ld;
    g.pitch = w.pitch;
    g.chunk = w.chunk;
    g.accumulate = accumulate;
    g.scale = a.scale;
    const int64_t spans = (a.cols + kSpan - 1) / kSpan, zeros = accumulate ? 0 : (a.rows + 3) / 4 * ((a.cols * (bf16 ? 2 : 4) + kZeroBytes - 1) / kZeroBytes);
    const int64_t most = (int64_t)ds->sm_count * 8;
    const int wide = width(a.cols, {dout, a.out_ld, dout_bf16}, {table, a.ld, bf16});
    if (a.tokens <= kFewTokens && a.tokens * spans <= kFewJobs) {
        const unsigned grid = up_to((a.tokens * spans + kEmbedWarps - 1) / kEmbedWarps * kEmbedWarps + zeros, kEmbedWarps, most);
        const cudaError_t e = by_types(dout_bf16, bf16, wide, [&](auto d, auto t, auto wide_of) {
            using Td = decltype(d);
            using Tt = decltype(t);
            return launch_chained(embed_few_kernel<Td, Tt, decltype(wide_of)::value>, dim3(grid), kEmbedThreads, 0, s, 1,
                                  static_cast<const Td*>(dout), ids, a.tokens, a.first, static_cast<Tt*>(table), g);
        });
        if (e != cudaSuccess) return set_cuda_error(e, "embedding gradient kernel launch");
        count_launch();
        return 0;
    }
    // Beside the tokens' order the first launch finds the rows without tokens, and writes zeros into as many of them,
    // by words of 32 rows a CTA, as the order leaves time for, at 4.5 TB/s (40009 tokens of 50021 x 1347 fp32:
    // 104 us with none, 98 this way; all of them there, 104, and 29 us more for 16384 x 8192 bf16, whose reads
    // then come after the zeros and not beside them).
    const bool rank = a.tokens <= kRankTokens;
    const int64_t words = (a.rows + 31) / 32, room = rank ? ds->sm_count : ds->embed_clusters > 1 ? ds->embed_clusters - 1 : 1;
    const int64_t clusters = accumulate || rank ? 0 : words < room ? words : room;
    const double order_us = rank ? 2.0 + 4e-4 * (double)a.tokens : 10.0 + 2.5e-4 * (double)a.tokens;
    const double word_bytes = 32.0 * (double)a.cols * (bf16 ? 2 : 4), beside = (double)(rank ? room : room * kSortCtas);
    const double clear = order_us * 4.5e6 / word_bytes / beside + 0.5;
    const int fill = clear < kFillBits ? (int)clear : kFillBits;
    uint32_t* named = accumulate ? nullptr : reinterpret_cast<uint32_t*>(base + w.named);
    g.named = named;
    int bits = 1;
    while (bits < 31 && ((int64_t)1 << bits) < a.rows) ++bits;
    const int passes = (bits + kSortBits - 1) / kSortBits;
    bits = (bits + passes - 1) / passes;
    cudaError_t e = by_types(bf16, bf16, wide, [&](auto t, auto, auto wide_of) {
        using Tt = decltype(t);
        constexpr int W = decltype(wide_of)::value;
        Tt* to = static_cast<Tt*>(table);
        if (rank)
            return launch_chained(embed_rank_kernel<Tt, W>, dim3((unsigned)room), kSortThreads, 0, s, 1, ids, a.tokens, a.first, a.rows, pairs,
                                  order, to, a.cols, a.ld, fill, named);
        return launch_chained(embed_sort_kernel<Tt, W>, dim3((unsigned)(kSortCtas * (1 + clusters))), kSortThreads, sort_smem(bits), s,
                              kSortCtas, ids, a.tokens, a.first, a.rows, bits, passes, pairs, reinterpret_cast<int2*>(base + w.other),
                              order, to, a.cols, a.ld, fill, named);
    });
    if (e != cudaSuccess) return set_cuda_error(e, "embedding order kernel launch");
    count_launch();
    const unsigned grid = up_to(w.chunks * spans + zeros, kEmbedWarps, most);
    const unsigned join_grid = w.chunks > 1 ? up_to((int64_t)(w.chunks - 1) * spans, 1, most) : 0;
    e = by_types(dout_bf16, bf16, wide, [&](auto d, auto t, auto wide_of) {
        using Td = decltype(d);
        using Tt = decltype(t);
        constexpr int W = decltype(wide_of)::value;
        auto sum = [&](auto kernel) {
            return launch_chained(kernel, dim3(grid), kEmbedThreads, 0, s, 1, static_cast<const Td*>(dout), static_cast<Tt*>(table), g);
        };
        const cudaError_t err = accumulate ? sum(embed_sum_kernel<Td, Tt, W, true>) : sum(embed_sum_kernel<Td, Tt, W, false>);
        if (err != cudaSuccess || join_grid == 0) return err;
        count_launch();
        if (spans <= kJoinSpans) return launch_chained(embed_join_kernel<Tt, W, 16>, dim3(join_grid), 512, 0, s, 1, static_cast<Tt*>(table), g);
        return launch_chained(embed_join_kernel<Tt, W, 8>, dim3(join_grid), 256, 0, s, 1, static_cast<Tt*>(table), g);
    });
    if (e != cudaSuccess) return set_cuda_error(e, "embedding gradient kernel launch");
    count_launch();
    return 0;
}

}  // namespace c3
