// ortho.cu -- orthogonalises an update by Newton-Schulz products:
//   X = U / (|U|_F + eps);   X <- (a I + b X X^T + c (X X^T)^2) X, some times;   out = scale X
// (the transposed products where U is tall, so that the square matrices have the short side).
//
// Iterates are fp16 times powers of two (ortho_plan.h): the tensor cores' bf16 rate with 11 bits instead
// of 8.  Five steps end 0.8e-3 to 2.4e-3 off (2-norm, relative; sides of 16 to 5003, random and with strong directions,
// fp32 and bf16), about a bf16 output's own rounding, 1.7e-3; eight times that, as bf16 would have it, is far above.  In
// directions that a matrix hardly has, roundings count for more: each step multiplies them by a, as it does singular
// values near 0.  Of rank 1 to 30, fp32 matrices came out 3 to 15% off and bf16 ones 2 to 4% (bf16 iterates: 30 to 190%).
// The polynomial is one matrix, its multiple of I included: a X and (b A + c A^2) X, which nearly cancel, are never
// rounded apart.
//
// The norm and the conversion are two passes over U; a step is three products by one kernel:
//   A = X X^T and P = a I + b A + c A A   symmetric: tiles on and above the diagonal alone;
//   X <- P X.
// Operands lie in memory as they are, along K or across it; the tensor cores take either.
#include "ops_device.cuh"
#include "c3_internal.h"
#include "ortho_plan.h"

#include <cuda_fp16.h>

#include <type_traits>

namespace c3 {

constexpr unsigned kAll = 0xffffffffu;

// ---------------------------------------------------------------- norm and conversion

constexpr int kOrthoThreads = 512;  // two CTAs an SM
constexpr int kOrthoWarps = kOrthoThreads / 32;
constexpr int kOrthoSpan = 256;

// Sums of squares are fp32 within a CTA, where their total is far from both ends of fp32's range, and fp64 between
// CTAs.  A CTA whose total is not (or is no number) adds its squares up again times 2^-180 or 2^180: 2^38 values below 2^128
// stay below 2^114 that way, squares of 2^-149 are 2^-118, and what a sum of 1e36 or 1e-18 consists of lies between.
constexpr float kTiny = 8.077935669463161e-28f, kHuge = 1.2379400392853803e27f;  // 2^-90, 2^90
constexpr double kTwo180 = (double)kHuge * (double)kHuge;

struct OrthoIn {
    const void* x;
    int64_t rows, cols, ld;
    int count, parts;
    double eps;
    int power;  // 2^power: X's first scale
    int early;  // the next kernel may start beside this one
    double* sums;
    float* scale;
    int* counts;  // of the products' parts, to be zero before the first
    __half* out;
    int64_t pitch;
};

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kAll, v, o);
    return v;
}

// A warp's pieces of kOrthoSpan columns, `step` apart, as rows and spans.
struct OrthoWalk {
    int64_t row;
    int span, spans, span_step;
    int64_t row_step;
    __device__ __forceinline__ OrthoWalk(int64_t at, int64_t step, int64_t width) {
        spans = (int)((width + kOrthoSpan - 1) / kOrthoSpan);
        row = at / spans;
        span = (int)(at - row * spans);
        row_step = step / spans;
        span_step = (int)(step - row_step * spans);
    }
    __device__ __forceinline__ void next() {
        row += row_step;
        span += span_step;
        if (span >= spans) span -= spans, ++row;
    }
};
constexpr int kOrthoAhead = 4;  // pieces of which a warp has the loads in flight

// A lane's eight values of a piece, as they are loaded and not looked at: many are in flight at once.
//   kWhole    rows are whole, aligned units of eight neighbours;
//   kShifted  bf16: the two aligned units that a lane's eight neighbours lie in, shifted when they are there, and at a
//             row's ends, where a unit has other values too, one by one;
//   kSingles  fp32: one by one, 32 apart (shifted, 5003 x 1347 took 268 us in all, this way 260).
// (35 M bf16 in rows of 4321: norm and conversion 62 and 65 us with loads and stores of single values, 29 and 43 this way.)
enum { kWhole = 0, kShifted = 1, kSingles = 2 };
template <typename T, int FORM>
struct OrthoPiece {
    static_assert(FORM == kWhole || (sizeof(T) == 2) == (FORM == kShifted), "form");
    uint32_t w[FORM == kWhole && sizeof(T) == 2 ? 4 : 8];
    int shift;  // kShifted: by how many values, or -1: one in each word

    __device__ __forceinline__ void load(const OrthoIn& g, const T* x, const OrthoWalk& at, int lane) {
        const int64_t c = (int64_t)at.span * kOrthoSpan + lane * (FORM == kSingles ? 1 : 8);
        const T* from = x + at.row * g.ld + c;
        const bool there = at.row < g.rows && c < g.cols;
        if constexpr (FORM == kSingles) {
#pragma unroll
            for (int i = 0; i < 8; ++i) w[i] = there && c + 32 * i < g.cols ? __float_as_uint(from[32 * i]) : 0;
            return;
        }
        shift = FORM == kWhole ? 0 : (int)((uintptr_t)from % 16 / sizeof(T));
        if constexpr (FORM == kShifted) {
            if (c < shift || c - shift + (shift ? 16 : 8) > g.cols) {
                shift = -1;
#pragma unroll
                for (int i = 0; i < 8; ++i) w[i] = there && c + i < g.cols ? reinterpret_cast<const uint16_t*>(from)[i] : 0;
                return;
            }
        }
        const uint4* unit = reinterpret_cast<const uint4*>(from - shift);
#pragma unroll
        for (int k = 0; k < (int)(sizeof(w) / 16); ++k) {
            uint4 u = make_uint4(0, 0, 0, 0);
            if (there && (FORM == kWhole || k == 0 || shift)) u = unit[k];
            w[4 * k] = u.x, w[4 * k + 1] = u.y, w[4 * k + 2] = u.z, w[4 * k + 3] = u.w;
        }
    }
    __device__ __forceinline__ void values(float (&v)[8]) {
        if constexpr (sizeof(T) == 4) {
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(w[i]);
            return;
        } else {
            if constexpr (FORM == kShifted) {
                if (shift < 0) {
#pragma unroll
                    for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(w[i] << 16);
                    return;
                }
#pragma unroll
                for (int by = 2; by > 0; by /= 2)
                    if (shift & (2 * by)) {
#pragma unroll
                        for (int i = 0; i + by < 8; ++i) w[i] = w[i + by];
                    }
#pragma unroll
                for (int i = 0; i < 4; ++i) w[i] = __funnelshift_r(w[i], w[i + 1], (shift & 1) * 16);
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(i & 1 ? w[i / 2] & 0xffff0000u : w[i / 2] << 16);
        }
    }
};

template <typename T, int FORM>
__global__ void __launch_bounds__(kOrthoThreads, 2) ortho_norm_kernel(OrthoIn g) {
    __shared__ float part[kOrthoWarps];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    if (g.early) chain_next();
    chain_ready();
    if (blockIdx.x == 0)
        for (int i = threadIdx.x; i < kOrthoRuns * 16; i += kOrthoThreads) g.counts[i] = 0;
    for (int64_t i = blockIdx.x; i < (int64_t)g.count * g.parts; i += gridDim.x) {
        const int64_t m = i / g.parts, p = i - m * g.parts;
        const T* x = static_cast<const T*>(g.x) + m * g.rows * g.ld;
        // the CTA's sum of squares of what `scaled` makes of the values
        auto squares = [&](auto scaled) {
            float sum = 0.0f;
            OrthoWalk at(p * kOrthoWarps + warp, (int64_t)g.parts * kOrthoWarps, g.cols);
            while (at.row < g.rows) {
                OrthoPiece<T, FORM> piece[kOrthoAhead];
#pragma unroll
                for (int a = 0; a < kOrthoAhead; ++a, at.next()) piece[a].load(g, x, at, lane);
#pragma unroll
                for (int a = 0; a < kOrthoAhead; ++a) {
                    float v[8];
                    piece[a].values(v);
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        const float t = scaled(v[k]);
                        sum = fmaf(t, t, sum);
                    }
                }
            }
            sum = warp_sum(sum);
            if (lane == 0) part[warp] = sum;
            __syncthreads();
            sum = warp_sum(lane < kOrthoWarps ? part[lane] : 0.0f);
            __syncthreads();
            return sum;
        };
        const float sum = squares([](float v) { return v; });
        double total = sum;
        if (!(sum < 1e36f)) total = (double)squares([](float v) { return v * kTiny; }) * kTwo180;
        else if (sum < 1e-18f) total = (double)squares([](float v) { return v * kHuge; }) / kTwo180;
        if (threadIdx.x == 0) g.sums[m * g.parts + p] = total;
    }
}

// X = U 2^-e in fp16, where 2^e is the power of two above |U| + eps: exact for bf16.  What is left of the
// division, 2^e / (|U| + eps) in (1, 2], goes to scale[m] and into the first step's products.  A NaN or an
// infinity makes the whole matrix NaN.
template <typename T, int FORM>
__global__ void __launch_bounds__(kOrthoThreads, 2) ortho_convert_kernel(OrthoIn g) {
    __shared__ float factors[2];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    if (g.early) chain_next();
    chain_ready();
    for (int64_t i = blockIdx.x; i < (int64_t)g.count * g.parts; i += gridDim.x) {
        const int64_t m = i / g.parts, p = i - m * g.parts;
        if (warp == 0) {
            double sum = 0.0;
            for (int j = lane; j < g.parts; j += 32) sum += g.sums[m * g.parts + j];
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(kAll, sum, o);
            if (lane == 0) {
                const double r = sqrt(sum) + g.eps;
                int e = 0;
                const double f = frexp(r, &e);
                const bool fine = isfinite(r);
                // two factors where one alone may leave fp32's range
                const int half = !fine ? 0 : abs(g.power - e) < 120 ? g.power - e : (g.power - e) / 2;
                factors[0] = fine ? (r > 0 ? (float)ldexp(1.0, half) : 0.0f) : __int_as_float(0x7fc00000);
                factors[1] = fine ? (float)ldexp(1.0, g.power - e - half) : 0.0f;
                if (p == 0) g.scale[m] = fine && r > 0 ? (float)(1.0 / f) : 1.0f;
            }
        }
        __syncthreads();
        const float f0 = factors[0], f1 = factors[1];
        const T* x = static_cast<const T*>(g.x) + m * g.rows * g.ld;
        __half* out = g.out + m * g.rows * g.pitch;
        OrthoWalk at(p * kOrthoWarps + warp, (int64_t)g.parts * kOrthoWarps, g.pitch);
        while (at.row < g.rows) {
            OrthoPiece<T, FORM> piece[2];
            OrthoWalk to = at;
#pragma unroll
            for (int a = 0; a < 2; ++a, at.next()) piece[a].load(g, x, at, lane);
#pragma unroll
            for (int a = 0; a < 2; ++a, to.next()) {
                if (to.row >= g.rows) break;
                float v[8];
                piece[a].values(v);
                if (f1 != 1.0f) {
#pragma unroll
                    for (int k = 0; k < 8; ++k) v[k] *= f1;
                }
                // kSingles: lanes of a pair trade half their values, so that each has pairs of neighbours
                const bool odd = lane & 1;
                uint32_t w[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    float lo = v[2 * k] * f0, hi = v[2 * k + 1] * f0;
                    if constexpr (FORM == kSingles) {
                        const float got = __shfl_xor_sync(kAll, odd ? lo : hi, 1);
                        (odd ? lo : hi) = got;
                    }
                    const __half2 t = __floats2half2_rn(lo, hi);
                    w[k] = *reinterpret_cast<const uint32_t*>(&t);
                }
                const int64_t c = (int64_t)to.span * kOrthoSpan + (FORM == kSingles ? (odd ? 32 : 0) + (lane & ~1) : lane * 8);
                __half* h = out + to.row * g.pitch + c;
                if constexpr (FORM == kSingles) {
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        if (c + 64 * k < g.pitch) *reinterpret_cast<uint32_t*>(h + 64 * k) = w[k];
                } else {
                    if (c < g.pitch) *reinterpret_cast<uint4*>(h) = make_uint4(w[0], w[1], w[2], w[3]);
                }
            }
        }
        __syncthreads();
    }
}

// ---------------------------------------------------------------- products
//
// A cluster of two CTAs shares a tile of 256 x NT (tcgen05.mma, cta_group::2): each brings in half of
// A's rows and half of B's and holds the accumulators of its own 128 rows, two sets of them, so that
// the read-out of a tile hides behind the next.  How an operand lies, A_IS and B_IS:
//   kAlong   K along memory;
//   kAcross  its rows (the output's rows or columns) along memory and K across it;
//   kUpper   symmetric, K along memory, and only blocks of 256 x 256 on and above the diagonal are there:
//            those below are read across, from their mirror image.
// So a symmetric product writes each of its tiles once.  (Written twice, turned over by way of shared
// memory, which the tensor cores need, 16 matrices of 1024 x 2048 took 830 us, and 684 turned over by
// 2-byte stores.)
//
// Results leave by TMA, boxes of 32 rows x 64 columns, and what is added to them comes in the same way into
// the same boxes: lanes that stored whole 32-byte sectors of their own rows kept the load and store units
// busy for longer than the products (648 us against 618).
//
// What bounds it: the tensor cores, and power, where matrices are large (4096 x 4096, under ncu: tensor pipe
// 80, 75 and 84% of the cycles in a step's three products; 8192 x 28672: 1.6 PFLOP/s of those that have
// to be done, 20.0 to 20.8 ms); what one SM can bring in, 60 bytes a cycle, for one tile, 0.27 us a K block of
// 256 x 256; and a launch's way from the last store before it to its own first one, 4.6 us, for
// matrices of one tile (256 x 640: 79 us for 17 launches).
constexpr int kGThreads = 320;  // producer, MMA, and the epilogue's eight warps
constexpr int kGEpiWarps = 8;
constexpr int kGK = 64;         // K of a stage: 128 bytes
constexpr int kGSmemLimit = 232448;
constexpr int kGGroupM = 16;

enum { kAlong = 0, kAcross = 1, kUpper = 2 };

enum OrthoWaitSite : int {
    kSiteOrthoProducer = 16,
    kSiteOrthoMma = 17,
    kSiteOrthoEpilogue = 18,
    kSiteOrthoDrain = 19,
};

// out = alpha A B^T (times scale[m] `times` times), rounded to fp16, or times scale_out to bf16; of two operands that are kUpper
// + beta mat + diag I, mat fp16 of the output's shape.
struct OrthoProduct {
    void* out;           // NULL: it has a tensor map, of boxes of 32 rows x 64 columns
    const float* scale;
    int64_t ld, stride;  // of out, and from one matrix to the next (no tensor map)
    int M, N, num_kb, count;
    int bf16, times;
    int early;           // the next kernel may start beside this one
    int width;           // bytes that rows of out are aligned to (no tensor map)
    float alpha, beta, diag;
    float scale_out;     // of the bf16 output, besides alpha
    OrthoTiles tiles;    // symmetric: tiles above the diagonal
    int per_matrix;      // tiles of one matrix
    OrthoSplit cut;
    float* parts;        // [runs][2][2 CTAs][8 warps][pieces][8][32 lanes] float4: sums of parts of tiles
    int* counts;         // [split][16]: parts that are there, by CTA and warp; all zero between products
};

template <int NT>
struct OrthoCfg {
    static constexpr uint32_t kABytes = 128 * 128;
    static constexpr uint32_t kBBytes = NT / 2 * 128;
    static constexpr uint32_t kStage = kABytes + kBBytes;
    // Boxes of 32 rows x 64 columns a warp, all of a tile's.  (One, and a sixth stage in its place: 5 x 1605 x 4321 922 us
    // against 889, 16 x 1024 x 2048 540 against 558.)
    static constexpr int kBoxes = NT / 128;
    static constexpr uint32_t kStaging = kGEpiWarps * kBoxes * 4096;
    static constexpr int kExtra = 1024 + 512 + (int)kStaging;
    static constexpr int kFit = (kGSmemLimit - kExtra) / (int)kStage;
    static constexpr int kStages = kFit > 8 ? 8 : kFit;
    static constexpr int kSmem = kStages * (int)kStage + kExtra;
};

__device__ __forceinline__ uint64_t along_desc(uint32_t saddr) {
    return (uint64_t)((saddr & 0x3FFFFu) >> 4) | ((uint64_t)1 << 16) | ((uint64_t)(1024 >> 4) << 32) | ((uint64_t)1 << 46) |
           ((uint64_t)2 << 61);
}
// Rows along memory: 64 of them and one K a 128-byte line, 8 K a swizzle atom of 1024 bytes, 64 K a box
// of 8 KB; leading offset from one box to the next 64 rows, stride offset from atom to atom.
__device__ __forceinline__ uint64_t across_desc(uint32_t saddr) {
    return (uint64_t)((saddr & 0x3FFFFu) >> 4) | ((uint64_t)(8192 >> 4) << 16) | ((uint64_t)(1024 >> 4) << 32) |
           ((uint64_t)1 << 46) | ((uint64_t)2 << 61);
}
__device__ __forceinline__ void mma_pair(uint32_t lead, uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 q, %5, 0;\n\t"
        "@q tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(accumulate),
        "r"(lead)
        : "memory");
}
__device__ __forceinline__ void tma_load_3d_pair(uint32_t dst, const CUtensorMap* map, uint32_t bar, int32_t x, int32_t y, int32_t z,
                                                 uint64_t policy) {
    asm volatile(
        "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint"
        " [%0], [%1, {%3, %4, %5}], [%2], %6;" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(y), "r"(z), "l"(policy)
        : "memory");
}

struct OrthoTile {
    int m, row, col;  // matrix, first row and column
};

template <int NT>
__device__ __forceinline__ OrthoTile ortho_tile(const OrthoProduct& g, int t) {
    OrthoTile r;
    r.m = g.count == 1 ? 0 : t / g.per_matrix;
    const int in = t - r.m * g.per_matrix;
    if (g.tiles.skip) {
        int i = 0;
        while (i + 1 < g.tiles.rows && g.tiles.before(i + 1) <= in) ++i;
        r.row = i * 256;
        r.col = (in - g.tiles.before(i) + g.tiles.skip * i) * NT;
        return r;
    }
    if (g.tiles.rows <= kGGroupM) {
        r.col = in / g.tiles.rows;
        r.row = (in - r.col * g.tiles.rows) * 256;
        r.col *= NT;
        return r;
    }
    const int per = kGGroupM * g.tiles.cols;
    const int grp = in / per, first = grp * kGGroupM;
    const int gm = min(g.tiles.rows - first, kGGroupM);
    const int at = in - grp * per;
    r.row = (first + at % gm) * 256;
    r.col = at / gm * NT;
    return r;
}

// Whether a K block of a symmetric operand's rows, which begin at `row` of a tile, lies below the diagonal's blocks.
__device__ __forceinline__ bool mirrored(int kb, int row) { return kb * kGK / 256 < row / 256; }

// A pair's i-th piece of work: the parts of tiles of its run, then whole tiles.
struct OrthoWorkItem {
    int tile;  // -1: no more
    int kb0, kb1;
};
template <bool CUT>
__device__ __forceinline__ OrthoWorkItem ortho_item(const OrthoSplit& s, int pair, int pairs, int i) {
    OrthoWorkItem w;
    const int whole = s.tiles - s.split;
    if (CUT && pair < s.runs) {
        const unsigned b0 = s.begin(pair), b1 = s.begin(pair + 1), t0 = b0 / (unsigned)s.num_kb;
        const int parts = (t0 + 1) * (unsigned)s.num_kb < b1 ? 2 : 1;  // a run is no longer than a tile
        if (i < parts) {
            const unsigned first = (t0 + i) * (unsigned)s.num_kb, last = first + (unsigned)s.num_kb;
            w.tile = whole + (int)t0 + i;
            w.kb0 = (int)((b0 > first ? b0 : first) - first);
            w.kb1 = (int)((b1 < last ? b1 : last) - first);
            return w;
        }
        i -= parts;
    }
    const int64_t t = pair + (int64_t)i * pairs;
    w.tile = t < whole ? (int)t : -1;
    w.kb0 = 0;
    w.kb1 = s.num_kb;
    return w;
}

__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap* map, uint32_t bar, int32_t x, int32_t y, int32_t z) {
    asm volatile("cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(dst),
                 "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(y), "r"(z)
                 : "memory");
}
__device__ __forceinline__ void tma_store_3d(const CUtensorMap* map, uint32_t src, int32_t x, int32_t y, int32_t z) {
    asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.bulk_group [%0, {%2, %3, %4}], [%1];" ::"l"(reinterpret_cast<uint64_t>(map)),
                 "r"(src), "r"(x), "r"(y), "r"(z)
                 : "memory");
}

// CUT: some tiles are cut along K (else g.cut has none); BOXES: the output has a tensor map.  What a product does not
// need is left out of its code.
template <int NT, int A_IS, int B_IS, bool CUT, bool BOXES>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kGThreads, 1)
    ortho_product_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                         const __grid_constant__ CUtensorMap acrossA, const __grid_constant__ CUtensorMap acrossB,
                         const __grid_constant__ CUtensorMap tmMat, const __grid_constant__ CUtensorMap tmOut, OrthoProduct g,
                         DevStatus* st) {
    constexpr bool kMat = A_IS == kUpper && B_IS == kUpper;  // beta mat + diag I is added
    using Cfg = OrthoCfg<NT>;
    constexpr int S = Cfg::kStages;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    const uint32_t raw = smem_addr(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    uint8_t* gbase = smem_raw + (base - raw);
    const uint32_t staging = base + S * Cfg::kStage;
    uint64_t* bars = reinterpret_cast<uint64_t*>(gbase + S * Cfg::kStage + Cfg::kStaging);
    // stage full [0, S), empty [S, 2S), accumulator full 2S.., empty 2S+2.., drain 2S+4, a warp's boxes
    // of the added matrix 2S+5 + 2 warp ..
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 2 * S + 5 + 2 * kGEpiWarps);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
    auto bar = [&](int i) { return smem_addr(&bars[i]); };
    const int TFULL = 2 * S, TEMPTY = 2 * S + 2, DRAIN = 2 * S + 4, BOX = 2 * S + 5;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = cluster_rank();

    if (g.early) chain_next();
    if (threadIdx.x == 0) {
        *abort_flag = 0;
        for (int i = 0; i < S; ++i) {
            mbar_init(bar(i), 1);
            mbar_init(bar(S + i), 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(bar(TFULL + b), 1);
            mbar_init(bar(TEMPTY + b), 2 * kGEpiWarps);
        }
        mbar_init(bar(DRAIN), 1);
        for (int b = 0; b < 2 * kGEpiWarps; ++b) mbar_init(bar(BOX + b), 1);
        fence_barrier_init();
        if (A_IS != kAcross) prefetch_tensormap(&tmA);
        if (A_IS != kAlong) prefetch_tensormap(&acrossA);
        if (B_IS != kAcross) prefetch_tensormap(&tmB);
        if (B_IS != kAlong) prefetch_tensormap(&acrossB);
        if (kMat) prefetch_tensormap(&tmMat);
        if (BOXES) prefetch_tensormap(&tmOut);
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_addr(tmem_slot))
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    }
    tc_fence_before();
    __syncthreads();
    cluster_sync_all();  // both CTAs' barriers are ready before either signals the other's
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    const int pair = (int)(blockIdx.x >> 1), pairs = (int)(gridDim.x >> 1);

    if (warp == 0) {
        if (lane == 0) {
            const uint64_t pol_a = policy_evict_last(), pol_b = policy_evict_normal();
            int stage = 0;
            uint32_t phase = 0;
            bool ok = true;
            for (int i = 0; ok; ++i) {
                const OrthoWorkItem item = ortho_item<CUT>(g.cut, pair, pairs, i);
                if (item.tile < 0) break;
                const OrthoTile tile = ortho_tile<NT>(g, item.tile);
                if (i == 0) chain_ready();
                const int arow = tile.row + (int)rank * 128, brow = tile.col + (int)rank * (NT / 2);
                for (int kb = item.kb0; kb < item.kb1; ++kb) {
                    if (!mbar_wait_cluster(bar(S + stage), phase ^ 1u, abort_flag)) {
                        report_error(st, -4, kSiteOrthoProducer);
                        ok = false;
                        break;
                    }
                    const uint32_t sa = base + (uint32_t)stage * Cfg::kStage, sb = sa + Cfg::kABytes;
                    const uint32_t full = leader_addr(bar(stage));
                    if (rank == 0) mbar_arrive_expect_tx(bar(stage), 2 * Cfg::kStage);
                    if (A_IS == kAcross || (A_IS == kUpper && mirrored(kb, tile.row))) {
                        tma_load_3d_pair(sa, &acrossA, full, arow, kb * kGK, tile.m, pol_a);
                        tma_load_3d_pair(sa + 8192, &acrossA, full, arow + 64, kb * kGK, tile.m, pol_a);
                    } else {
                        tma_load_3d_pair(sa, &tmA, full, kb * kGK, arow, tile.m, pol_a);
                    }
                    if (B_IS == kAcross || (B_IS == kUpper && mirrored(kb, tile.col))) {
#pragma unroll
                        for (int j = 0; j < NT / 128; ++j)
                            tma_load_3d_pair(sb + j * 8192, &acrossB, full, brow + j * 64, kb * kGK, tile.m, pol_b);
                    } else {
                        tma_load_3d_pair(sb, &tmB, full, kb * kGK, brow, tile.m, pol_b);
                    }
                    if (++stage == S) {
                        stage = 0;
                        phase ^= 1u;
                    }
                }
            }
            // The pair's loads have all landed once every stage that was filled has been freed (its
            // MMAs follow its loads): wait for that before the CTA may end.  After a wait gave up,
            // the leader's full barriers tell it instead.
            volatile int no_abort = 0;
            for (int i = 0; (ok || rank == 0) && i < S; ++i)
                if (!mbar_wait_cluster(bar(ok ? S + i : i), (i < stage) ? phase : (phase ^ 1u), &no_abort))
                    report_error(st, -4, kSiteOrthoDrain);
        }
    } else if (warp == 1) {
        if (rank == 0) {
            const uint32_t lead = elect_lane();
            // D fp32, A and B fp16, N >> 3, M >> 4; bits 15 and 16 say that A, B lie across
            const uint32_t idesc = (1u << 4) | ((uint32_t)(NT >> 3) << 17) | ((uint32_t)(256 >> 4) << 24);
            const uint64_t a_along = along_desc(base), a_across = across_desc(base);
            const uint64_t b_along = along_desc(base + Cfg::kABytes), b_across = across_desc(base + Cfg::kABytes);
            int stage = 0;
            uint32_t phase = 0;
            bool ok = true;
            for (int local = 0; ok; ++local) {
                const OrthoWorkItem item = ortho_item<CUT>(g.cut, pair, pairs, local);
                if (item.tile < 0) break;
                const int buf = local & 1;
                if (!mbar_wait_cluster(bar(TEMPTY + buf), ((uint32_t)(local >> 1) & 1u) ^ 1u, abort_flag)) {
                    report_error(st, -4, kSiteOrthoMma);
                    break;
                }
                tc_fence_after();
                const OrthoTile tile = ortho_tile<NT>(g, item.tile);
                const uint32_t d = tmem + (uint32_t)(buf * NT);
                // It reads shared memory alone, but its waits have a limit, which must not run while the kernels before
                // do: these may take seconds, on few SMs.  (The waits above end at once the first time.)
                if (local == 0) chain_ready();
                for (int kb = item.kb0; kb < item.kb1; ++kb) {
                    if (!mbar_wait_cluster(bar(stage), phase, abort_flag)) {
                        report_error(st, -4, kSiteOrthoMma);
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const bool ta = A_IS == kAcross || (A_IS == kUpper && mirrored(kb, tile.row));
                    const bool tb = B_IS == kAcross || (B_IS == kUpper && mirrored(kb, tile.col));
                    const uint64_t at = (uint64_t)((uint32_t)stage * (Cfg::kStage >> 4));
                    const uint64_t ad = (ta ? a_across : a_along) + at, bd = (tb ? b_across : b_along) + at;
                    // 16 of K: 32 bytes along a line, or two atoms
                    const uint32_t ka = ta ? 2048 >> 4 : 2, kb16 = tb ? 2048 >> 4 : 2;
                    const uint32_t id = idesc | (ta ? 1u << 15 : 0u) | (tb ? 1u << 16 : 0u);
#pragma unroll
                    for (int k = 0; k < kGK / 16; ++k)
                        mma_pair(lead, d, ad + (uint64_t)(k * ka), bd + (uint64_t)(k * kb16), id, k > 0 ? 1u : (uint32_t)(kb > item.kb0));
                    commit_pair(lead, bar(S + stage));
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
            if (!mbar_wait(bar(DRAIN), 0, &no_abort)) report_error(st, -4, kSiteOrthoDrain);
        }
    } else {
        const int q = warp & 3, half = (warp - 2) >> 2;
        const uint32_t box0 = staging + (uint32_t)(warp - 2) * (Cfg::kBoxes * 4096u);
        constexpr int kRounds = NT / 128;  // of 64 columns: half of the tile's
        chain_ready();
        uint32_t mat_phase = 0;
        for (int local = 0;; ++local) {
            const OrthoWorkItem item = ortho_item<CUT>(g.cut, pair, pairs, local);
            if (item.tile < 0) break;
            const OrthoTile tile = ortho_tile<NT>(g, item.tile);
            const int buf = local & 1;
            const int row0 = tile.row + (int)rank * 128 + q * 32, col0 = tile.col + half * (NT / 2);
            const bool cut = CUT && item.kb1 - item.kb0 < g.num_kb;
            const int place = item.tile - (g.cut.tiles - g.cut.split);  // among the cut tiles
            int run0 = 0, run1 = 0;                                     // the runs that have parts of the tile
            // What is added, on its way while the products run: into the boxes that the results go out from.
            auto fetch = [&] {
                if (lane == 0) {
                    bulk_wait_read<0>();
#pragma unroll
                    for (int rd = 0; rd < kRounds; ++rd) {
                        const uint32_t b = bar(BOX + (warp - 2) * 2 + rd);
                        mbar_arrive_expect_tx(b, 4096);
                        tma_load_3d(box0 + (uint32_t)rd * 4096u, &tmMat, b, col0 + rd * 64, row0, tile.m);
                    }
                }
                __syncwarp();
            };
            auto release = [&] {
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive_cluster(leader_addr(bar(TEMPTY + buf)));
            };
            const uint32_t taddr = tmem + ((uint32_t)(q * 32) << 16) + (uint32_t)(buf * NT + half * (NT / 2));
            // The tile's sums are there.
            auto sums_ready = [&] {
                const bool ready = mbar_wait_cluster(bar(TFULL + buf), (uint32_t)(local >> 1) & 1u, abort_flag);
                if (!__all_sync(kAll, ready)) {
                    report_error(st, -4, kSiteOrthoEpilogue);
                    volatile int no_abort = 0;  // what is on its way into the boxes has to land before the CTA ends
                    for (int rd = 0; kMat && !cut && rd < kRounds; ++rd) mbar_wait(bar(BOX + (warp - 2) * 2 + rd), mat_phase, &no_abort);
                    return false;
                }
                tc_fence_after();
                return true;
            };
            // this warp's place in the part that `run` has of the tile
            auto part_of = [&](int run) {
                const int which = run == run0 ? place - (int)(g.cut.begin(run) / (unsigned)g.num_kb) : 0;
                return reinterpret_cast<float4*>(g.parts) + (((run * 2 + which) * 2 + (int)rank) * kGEpiWarps + (warp - 2)) * (kRounds * 512) + lane;
            };
            if (kMat && !cut) fetch();
            if (CUT && cut) {
                if (!sums_ready()) break;
                run0 = g.cut.run_of((unsigned)place * (unsigned)g.num_kb);
                run1 = g.cut.run_of((unsigned)(place + 1) * (unsigned)g.num_kb - 1);
                float4* mine = part_of(pair);
#pragma unroll 1
                for (int p = 0; p < 2 * kRounds; ++p) {
                    uint32_t r[32];
                    tmem_ld32(taddr + (uint32_t)(p * 32), r);
                    tmem_ld_wait();
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        __stcg(mine + (p * 8 + j) * 32, make_float4(__uint_as_float(r[4 * j]), __uint_as_float(r[4 * j + 1]),
                                                                    __uint_as_float(r[4 * j + 2]), __uint_as_float(r[4 * j + 3])));
                }
                release();
                __threadfence();
                __syncwarp();
                int there = 0;
                int* count = g.counts + place * 16 + (int)rank * kGEpiWarps + (warp - 2);
                if (lane == 0) {
                    there = atomicAdd(count, 1);
                    if (there == run1 - run0) *count = 0;  // the last: nobody else comes
                }
                if (__shfl_sync(kAll, there, 0) != run1 - run0) continue;
                __threadfence();
                if (kMat) fetch();
            }
            float alpha = g.alpha;
            for (int i = 0; i < g.times; ++i) alpha *= g.scale[tile.m];
            // 64 columns at a time, and 32 of them, in loops that are left rolled: short code, which a chain of small products
            // fetches again and again (both halves unrolled: 256 x 640 116 us against 103), and no spills, which go all the
            // way to L2, since shared memory leaves L1 next to nothing (1.3 KB: 16 x 1024 x 2048 1198 us against 684).
            //
            // The first tile is preceded by a round on nothing, which stores nothing: the warps would wait for the tile's sums,
            // and so they bring the round's instructions in meanwhile (a product of a small matrix is a chain of first times).
            // Not where the boxes are already being filled.
            bool ok = true;
#pragma unroll 1
            for (int rd = local == 0 && !cut && !kMat ? -1 : 0; rd < kRounds; ++rd) {
                if (rd == 0 && !cut) {
                    ok = sums_ready();
                    if (!ok) break;
                }
                const uint32_t box = box0 + (uint32_t)(rd < 0 ? 0 : rd) * 4096u;
                if (rd < 0) {
                } else if (kMat) {
                    const bool in = mbar_wait(bar(BOX + (warp - 2) * 2 + rd), mat_phase, abort_flag);
                    if (!__all_sync(kAll, in)) report_error(st, -4, kSiteOrthoEpilogue);
                } else {
                    if (lane == 0) bulk_wait_read<Cfg::kBoxes - 1>();  // what the box held has left it
                    __syncwarp();
                }
#pragma unroll 1
                for (int h = 0; h < 2; ++h) {
                    const int p = 2 * rd + h, c0 = col0 + p * 32;
                    uint32_t r[32];
                    if (CUT && cut) {  // the parts in order, whoever adds them up
#pragma unroll
                        for (int j = 0; j < 32; ++j) r[j] = 0;
#pragma unroll 1
                        for (int run = run0; run <= run1; run += 2) {
                            float4 t[2][8];
#pragma unroll
                            for (int k = 0; k < 2; ++k) {
                                const float4* from = part_of(run + k) + p * 256;
#pragma unroll
                                for (int j = 0; j < 8; ++j) t[k][j] = run + k <= run1 ? __ldcg(from + j * 32) : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                            }
#pragma unroll
                            for (int k = 0; k < 2; ++k)
#pragma unroll
                                for (int j = 0; j < 8; ++j) {
                                    r[4 * j] = __float_as_uint(__uint_as_float(r[4 * j]) + t[k][j].x);
                                    r[4 * j + 1] = __float_as_uint(__uint_as_float(r[4 * j + 1]) + t[k][j].y);
                                    r[4 * j + 2] = __float_as_uint(__uint_as_float(r[4 * j + 2]) + t[k][j].z);
                                    r[4 * j + 3] = __float_as_uint(__uint_as_float(r[4 * j + 3]) + t[k][j].w);
                                }
                        }
                    } else if (rd >= 0) {
                        tmem_ld32(taddr + (uint32_t)(p * 32), r);
                        tmem_ld_wait();
                        if (p + 1 == 2 * kRounds) release();
                    } else {
#pragma unroll
                        for (int j = 0; j < 32; ++j) r[j] = 0;
                    }
                    // lane's row of the box: 16-byte chunk j at j ^ (row % 8), as the tensor maps have it
                    const uint32_t line = box + (uint32_t)lane * 128u;
                    if constexpr (kMat) {
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            uint32_t o[4];
                            ld_shared_v4(line + (uint32_t)(((4 * h + j) ^ (lane & 7)) << 4), o);
#pragma unroll
                            for (int k = 0; k < 4; ++k) {
                                const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&o[k]));
                                const int i = 8 * j + 2 * k;
                                r[i] = __float_as_uint(fmaf(g.beta, f.x, alpha * __uint_as_float(r[i])));
                                r[i + 1] = __float_as_uint(fmaf(g.beta, f.y, alpha * __uint_as_float(r[i + 1])));
                            }
                        }
                        if (row0 == c0) {
#pragma unroll
                            for (int j = 0; j < 32; ++j)
                                if (j == lane) r[j] = __float_as_uint(__uint_as_float(r[j]) + g.diag);
                        }
                    } else {
#pragma unroll
                        for (int j = 0; j < 32; ++j) r[j] = __float_as_uint(alpha * __uint_as_float(r[j]));
                    }
                    uint32_t v[16];
                    if (!kMat && g.bf16) {
#pragma unroll
                        for (int j = 0; j < 16; ++j) {
                            const __nv_bfloat162 x = __floats2bfloat162_rn(g.scale_out * __uint_as_float(r[2 * j]), g.scale_out * __uint_as_float(r[2 * j + 1]));
                            v[j] = *reinterpret_cast<const uint32_t*>(&x);
                        }
                    } else {
#pragma unroll
                        for (int j = 0; j < 16; ++j) {
                            const __half2 x = __floats2half2_rn(__uint_as_float(r[2 * j]), __uint_as_float(r[2 * j + 1]));
                            v[j] = *reinterpret_cast<const uint32_t*>(&x);
                        }
                    }
                    if (BOXES) {
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            st_shared_v4(line + (uint32_t)(((4 * h + j) ^ (lane & 7)) << 4), v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
                    } else if (rd >= 0) {
                        store_piece<uint16_t>(v, box, lane, g.width, static_cast<uint16_t*>(g.out) + tile.m * g.stride, row0, g.M - row0, c0,
                                              g.N, g.ld);
                    }
                }
                if (BOXES) {
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0 && rd >= 0) {
                        if (row0 < g.M && col0 + rd * 64 < g.N) tma_store_3d(&tmOut, box, col0 + rd * 64, row0, tile.m);
                        bulk_commit();
                    }
                }
            }
            if (!ok) break;
            if (kMat) mat_phase ^= 1u;
        }
        if (lane == 0) bulk_wait_all();
        __syncwarp();
    }
    tc_fence_before();
    __syncthreads();
    cluster_meet();  // nothing of this CTA's is signalled or read by the other any more
    if (warp == 1) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
    }
}

// ---------------------------------------------------------------- host side

template <int NT, bool CUT, typename F>
static int each_product(F f) {
    constexpr int smem = OrthoCfg<NT>::kSmem;
    int rc = f(ortho_product_kernel<NT, kAlong, kAlong, CUT, true>, smem);
    if (!rc) rc = f(ortho_product_kernel<NT, kAcross, kAcross, CUT, true>, smem);
    if (!rc) rc = f(ortho_product_kernel<NT, kUpper, kUpper, CUT, true>, smem);
    if (!rc) rc = f(ortho_product_kernel<NT, kUpper, kAcross, CUT, true>, smem);
    if (!rc) rc = f(ortho_product_kernel<NT, kAlong, kUpper, CUT, true>, smem);
    if (!rc) rc = f(ortho_product_kernel<NT, kUpper, kAcross, CUT, false>, smem);
    if (!rc) rc = f(ortho_product_kernel<NT, kAlong, kUpper, CUT, false>, smem);
    return rc;
}

int ortho_init_device() {
    auto allow = [](auto kernel, int smem) {
        const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        return e == cudaSuccess ? 0 : set_cuda_error(e, "cudaFuncSetAttribute(orthogonalisation)");
    };
    int rc = each_product<256, false>(allow);
    if (!rc) rc = each_product<256, true>(allow);
    if (!rc) rc = each_product<128, false>(allow);
    if (!rc) rc = each_product<128, true>(allow);
    return rc;
}

// fp16 or bf16 matrices [count][rows][pitch], in boxes of 64 columns x box_rows.  What lies past a matrix reads as zeros.
static int ortho_map(CUtensorMap* map, const void* p, int64_t rows, int64_t cols, int64_t pitch, int count, int box_rows, bool bf16) {
    EncodeTiledFn fn = tensor_map_encode();
    if (!fn) return set_error(-3, "cuTensorMapEncodeTiled entry point unavailable");
    cuuint64_t dims[3] = {(cuuint64_t)cols, (cuuint64_t)rows, (cuuint64_t)count};
    cuuint64_t strides[2] = {(cuuint64_t)pitch * 2, (cuuint64_t)(rows * pitch) * 2};
    cuuint32_t box[3] = {64, (cuuint32_t)box_rows, 1};
    cuuint32_t estr[3] = {1, 1, 1};
    CUresult r = fn(map, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3, const_cast<void*>(p), dims, strides, box, estr,
                    CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                    CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? 0 : set_error(-3, "cuTensorMapEncodeTiled (orthogonalisation) failed");
}

size_t ortho_bytes(int64_t rows, int64_t cols, int count) { return ortho_work(rows, cols, count).bytes; }

template <typename T>
static cudaError_t ortho_in(bool whole, unsigned grid, cudaStream_t s, const OrthoIn& in) {
    auto go = [&](auto norm, auto convert) {
        cudaError_t e = launch_chained(norm, dim3(grid), kOrthoThreads, 0, s, 1, in);
        if (e != cudaSuccess) return e;
        count_launch();
        return launch_chained(convert, dim3(grid), kOrthoThreads, 0, s, 1, in);
    };
    constexpr int kElse = sizeof(T) == 2 ? kShifted : kSingles;
    return whole ? go(ortho_norm_kernel<T, kWhole>, ortho_convert_kernel<T, kWhole>)
                 : go(ortho_norm_kernel<T, kElse>, ortho_convert_kernel<T, kElse>);
}

int ortho_launch(const void* x, int bf16, int64_t rows, int64_t cols, int64_t ld, int count, const float (*coeffs)[3], int steps,
                 double eps, float scale, void* out, int64_t out_ld, void* work, int sm_budget, cudaStream_t s) {
    DeviceState* ds = device_state();
    if (!ds) return -3;
    if (take_fault(kFaultGemmLaunch)) return set_error(-3, "injected failure: GEMM launch");
    OrthoStep step[kOrthoSteps];
    if (!ortho_steps(coeffs, steps, step)) return set_error(-1, "coeffs let the iterates grow without bound");
    const int cap = (sm_budget <= 0 || sm_budget > ds->sm_count) ? ds->sm_count : sm_budget;
    const OrthoWork w = ortho_work(rows, cols, count);
    uint8_t* base = static_cast<uint8_t*>(work);
    const int64_t m = w.short_side;
    const bool tall = rows > cols;

    OrthoIn in;
    in.x = x;
    in.rows = rows;
    in.cols = cols;
    in.ld = ld;
    in.count = count;
    in.eps = eps;
    in.power = step[0].x;
    // Under a budget no kernel starts beside the one before, on SMs that are left to others: one product after the
    // other would wait there with all of an SM's shared memory (20 SMs, 8192 x 8192: a product of 0.1 ms on the
    // other 132 took 3.6 ms).
    in.early = cap == ds->sm_count;
    in.sums = reinterpret_cast<double*>(base + w.sums);
    in.scale = reinterpret_cast<float*>(base + w.scale);
    in.counts = reinterpret_cast<int*>(base + w.counts);
    in.out = reinterpret_cast<__half*>(base + w.x0);
    in.pitch = w.xpitch;
    // parts of a norm: no more than give each warp a span of columns; over all matrices two an SM of the budget, rounded
    // up to whole ones for each matrix
    const int64_t jobs = rows * ((cols + kOrthoSpan - 1) / kOrthoSpan), most = (jobs + kOrthoWarps - 1) / kOrthoWarps;
    const int64_t want = (2 * (int64_t)cap + count - 1) / count;
    in.parts = (int)(most < want ? most : want);
    if (in.parts > ortho_parts(count)) in.parts = ortho_parts(count);
    const int64_t all = (int64_t)in.parts * count, fit = sm_budget > 0 && cap < ds->sm_count ? cap : 2 * (int64_t)cap;
    const bool whole = cols % 8 == 0 && (uintptr_t)x % 16 == 0 && ld % (bf16 ? 8 : 4) == 0;
    const unsigned grid = (unsigned)(all < fit ? all : fit);
    cudaError_t e = bf16 ? ortho_in<__nv_bfloat16>(whole, grid, s, in) : ortho_in<float>(whole, grid, s, in);
    if (e != cudaSuccess) return set_cuda_error(e, "orthogonalisation: norm kernel launch");
    count_launch();

    auto blocks = [](int64_t n, int by) { return (int)((n + by - 1) / by); };
    __half* X[2] = {reinterpret_cast<__half*>(base + w.x0), reinterpret_cast<__half*>(base + w.x1)};
    __half* G = reinterpret_cast<__half*>(base + w.g);
    __half* P = reinterpret_cast<__half*>(base + w.p);
    CUtensorMap xm[2][3], gm[3], pm[3], om;  // boxes of 128, 64 and 32 rows; of the output
    // (A box's last 16-byte unit of a row is written whole.  What so lies behind rows of X, A and P are zeros, of
    // operands' rows that do not exist.)
    // (a map's strides are below 2^40 bytes)
    const bool boxes = (uintptr_t)out % 16 == 0 && out_ld % 8 == 0 && cols % 8 == 0 && out_ld < ((int64_t)1 << 39) / rows;
    int rc = 0;
    for (int j = 0; j < 3 && !rc; ++j) {
        const int box = 128 >> j;
        for (int i = 0; i < 2 && !rc; ++i) rc = ortho_map(&xm[i][j], X[i], rows, cols, w.xpitch, count, box, false);
        if (!rc) rc = ortho_map(&gm[j], G, m, m, w.gpitch, count, box, false);
        if (!rc) rc = ortho_map(&pm[j], P, m, m, w.gpitch, count, box, false);
    }
    if (!rc) rc = boxes ? ortho_map(&om, out, rows, cols, out_ld, count, 32, true) : 0;
    if (!boxes) om = xm[0][2];
    if (rc) return rc;

    // Which product: an operand's two maps are its boxes of 128 and of 64 rows.
    enum { kGramWide, kGramTall, kPoly, kApplyWide, kApplyTall };  // the first three symmetric
    auto product = [&](int which, const CUtensorMap (&a)[3], const CUtensorMap (&b)[3], const CUtensorMap& to, OrthoProduct& g) -> int {
        const int pairs = cap / 2;
        const OrthoPlan plan = ortho_plan(g.M, g.N, which <= kPoly, g.num_kb, count, pairs);
        if (plan.total > 0x7FFFFFFF) return set_error(-5, "orthogonalisation: more than 2^31 tiles");
        g.tiles = plan.tiles;
        g.per_matrix = (int)plan.tiles.total();
        g.cut = plan.cut;
        g.parts = reinterpret_cast<float*>(base + w.parts);
        g.counts = in.counts;
        const int some = g.cut.tiles < g.cut.runs ? g.cut.runs : g.cut.tiles;
        const dim3 ctas((unsigned)(2 * (some < pairs ? some : pairs)));
        auto by_form = [&](auto nt_of, auto cut_of) {
            constexpr int NT = decltype(nt_of)::value;
            constexpr bool CUT = decltype(cut_of)::value;
            auto go = [&](auto kernel) {
                // A along K in boxes of 128 rows, B in boxes of NT / 2; either across K in boxes of 64
                return launch_chained(kernel, ctas, kGThreads, OrthoCfg<NT>::kSmem, s, 1, a[0], b[NT == 128], a[1], b[1], gm[2], to, g, ds->status);
            };
            switch (which) {
                case kGramWide: return go(ortho_product_kernel<NT, kAlong, kAlong, CUT, true>);
                case kGramTall: return go(ortho_product_kernel<NT, kAcross, kAcross, CUT, true>);
                case kPoly: return go(ortho_product_kernel<NT, kUpper, kUpper, CUT, true>);
                case kApplyWide:
                    return g.out ? go(ortho_product_kernel<NT, kUpper, kAcross, CUT, false>) : go(ortho_product_kernel<NT, kUpper, kAcross, CUT, true>);
                default:
                    return g.out ? go(ortho_product_kernel<NT, kAlong, kUpper, CUT, false>) : go(ortho_product_kernel<NT, kAlong, kUpper, CUT, true>);
            }
        };
        auto by_cut = [&](auto nt_of) { return g.cut.runs ? by_form(nt_of, std::true_type()) : by_form(nt_of, std::false_type()); };
        const cudaError_t err = plan.nt == 128 ? by_cut(std::integral_constant<int, 128>()) : by_cut(std::integral_constant<int, 256>());
        if (err != cudaSuccess) return set_cuda_error(err, "orthogonalisation: product kernel launch");
        count_launch();
        return 0;
    };
    for (int i = 0; i < steps; ++i) {
        const OrthoStep& t = step[i];
        const int now = i & 1;
        auto two = [](int p) { return (float)std::ldexp(1.0, p); };
        OrthoProduct g{};
        g.scale = in.scale;
        g.count = count;
        g.early = in.early;
        // A = X X^T (X^T X): the stored 2^x X give 2^2x of it
        g.M = g.N = (int)m;
        g.num_kb = blocks(tall ? rows : cols, kGK);
        g.times = i == 0 ? 2 : 0;
        g.alpha = two(t.g - 2 * t.x);
        if ((rc = product(tall ? kGramTall : kGramWide, xm[now], xm[now], gm[2], g))) return rc;
        // P = a I + b A + c A A
        g.num_kb = blocks(m, kGK);
        g.times = 0;
        g.alpha = t.c * two(t.p - 2 * t.g);
        g.beta = t.b * two(t.p - t.g);
        g.diag = t.a * two(t.p);
        if ((rc = product(kPoly, gm, gm, pm[2], g))) return rc;
        // X <- P X (X P)
        const bool last = i + 1 == steps;
        g.M = (int)rows;
        g.N = (int)cols;
        g.times = i == 0 ? 1 : 0;
        // (one factor of both would be subnormal, and lose digits, for a scale below 2^-103)
        g.alpha = two((last ? 0 : t.next) - t.p - t.x);
        g.scale_out = scale;
        g.bf16 = last;
        if (last && !boxes) {
            g.out = out;
            g.ld = out_ld;
            g.stride = rows * out_ld;
            const uintptr_t bits = (uintptr_t)out | (uintptr_t)(2 * out_ld) | (uintptr_t)(2 * cols);
            g.width = bits % 4 == 0 ? 4 : 2;
        }
        const CUtensorMap& to = last ? om : xm[now ^ 1][2];
        rc = tall ? product(kApplyTall, xm[now], pm, to, g) : product(kApplyWide, pm, xm[now], to, g);
        if (rc) return rc;
    }
    return 0;
}

}  // namespace c3
