// ortho_plan.h -- how an orthogonalisation is laid out and scaled (ortho.cu has the
// kernels).  Host arithmetic alone, so that it can be checked without a GPU.
#pragma once

#include <cmath>
#include <cstddef>
#include <cstdint>

namespace c3 {

constexpr int kOrthoSteps = 32;        // polynomials at most
constexpr int kOrthoTop = 13;          // stored values stay below 2^13 times their bound: 8 times below fp16's largest
constexpr double kOrthoMost = 1 << 20; // the largest singular value that an iterate may reach

// One step: X <- (a + b X X^T + c X X^T X X^T) X.  Matrices are held in fp16 times powers of two,
// 2^x, 2^g and 2^p for X, X X^T and the polynomial, so that the largest entry they can have stays
// well below fp16's range and small ones keep their digits; next: the power for the X that the step makes.
struct OrthoStep {
    float a, b, c;
    int x, g, p, next;
};

// The power of two that takes `bound` below 2^kOrthoTop.
inline int ortho_power(double bound) {
    int e = 0;
    std::frexp(bound > 1.0 / kOrthoMost ? bound : 1.0 / kOrthoMost, &e);
    return kOrthoTop - e;
}

// Entries of a matrix are at most its largest singular value.  Those of X are at most 1 after the
// division by the norm, and a step takes s to s |a + b s^2 + c s^4|: bounds of it, and of the
// polynomial, over 0..s.  False where the iterates may grow past kOrthoMost.
inline bool ortho_steps(const float (*coeffs)[3], int steps, OrthoStep* out) {
    double top = 1.0;
    for (int i = 0; i < steps; ++i) {
        const double a = coeffs[i][0], b = coeffs[i][1], c = coeffs[i][2], q = top * top;
        auto poly = [&](double t) { return std::fabs(a + b * t + c * t * t); };
        auto image = [&](double t) { return std::sqrt(t) * poly(t); };
        double pmax = std::fmax(poly(0), poly(q)), smax = image(q);
        if (c != 0 && -b / (2 * c) > 0 && -b / (2 * c) < q) pmax = std::fmax(pmax, poly(-b / (2 * c)));
        // a + 3 b t + 5 c t^2 = 0, t = s^2, by way of the root that does not cancel: the other would be lost where
        // c is tiny beside b
        const double disc = 9 * b * b - 20 * a * c;
        double roots[2] = {-1, -1};
        if (disc >= 0) {
            const double h = -(3 * b + std::copysign(std::sqrt(disc), b)) / 2;
            if (c != 0) roots[0] = h / (5 * c);
            if (h != 0) roots[1] = a / h;
        }
        for (double t : roots)
            if (t > 0 && t < q) smax = std::fmax(smax, image(t));
        OrthoStep& s = out[i];
        s.a = coeffs[i][0], s.b = coeffs[i][1], s.c = coeffs[i][2];
        s.x = ortho_power(top);
        s.g = ortho_power(q);
        s.p = ortho_power(pmax);
        // values rounded to 11 bits are up to 2^-11 off, four times over, what the bound was found for
        top = 1.002 * smax;
        if (!(top <= kOrthoMost) || !(pmax <= kOrthoMost)) return false;
        s.next = ortho_power(top);
    }
    return true;
}

// Upper triangle of a symmetric product, diagonal included, in tiles of 256 x cols: row block i has
// the columns' blocks from i * 256 / cols on.
struct OrthoTiles {
    int rows, cols;  // blocks
    int skip;        // 256 / width of a column block; 0: every tile
#ifdef __CUDACC__
    __host__ __device__
#endif
    int before(int i) const { return i * cols - skip * (i * (i - 1) / 2); }
    int64_t total() const {
        return skip ? (int64_t)rows * cols - (int64_t)skip * rows * (rows - 1) / 2 : (int64_t)rows * cols;
    }
};

// How a product's tiles are dealt out to pairs of SMs.  Whole turns of all pairs take whole tiles; the
// `split` tiles left over are laid end to end, by K blocks, and cut into as many runs as `runs` says, a pair each.
// A tile that several runs have a part of is put together from their fp32 sums by whoever comes last.
constexpr int kOrthoRuns = 80;  // at most: each has room for two parts of tiles

struct OrthoSplit {
    int tiles;        // of the product
    int split, runs;  // 0: none
    int num_kb;       // at most 2^18, so that 80 x 80 of them have 32-bit numbers
#ifdef __CUDACC__
    __host__ __device__
#endif
    unsigned begin(int run) const { return (unsigned)run * (unsigned)split * (unsigned)num_kb / (unsigned)runs; }
    // The run that has a K block.
#ifdef __CUDACC__
    __host__ __device__
#endif
    int run_of(unsigned block) const { return (int)(((block + 1) * (unsigned)runs - 1) / ((unsigned)split * (unsigned)num_kb)); }
};

constexpr int kOrthoFewest = 8;  // K blocks of a tile that is cut, at least

// Which tiles a product has, 256 x 256 or 256 x 128, and how they are dealt out.
struct OrthoPlan {
    int nt;
    OrthoTiles tiles;  // of one matrix
    int64_t total;     // of all matrices; the cut holds for 2^31 at most
    OrthoSplit cut;
    double us;         // what the turns of the busiest pair are taken to cost
};

// A K block takes 0.3 us in tiles of 256 x 256 and 0.2 in tiles of 256 x 128, which bring in three quarters of the
// bytes for half the products (0.27 to 0.34 and 0.2 measured).  Tiles left over by whole turns of all pairs would take a
// whole one's time; cut, their share of the runs' and what their parts cost to write and read back: of 256 x 256, 1.2 us
// a part, which stops its pair's next tile where it has one, and where no whole tiles hide it 2.4 us for the meeting.
// (16 matrices of 1024 x 2048: 8 of 160 tiles of 32 blocks are left; in 64 parts the product took 50 us, whole 36.)
inline OrthoPlan ortho_plan_of(int64_t M, int64_t N, bool symmetric, int num_kb, int count, int pairs, int nt) {
    OrthoPlan p;
    p.nt = nt;
    p.tiles = OrthoTiles{(int)((M + 255) / 256), (int)((N + nt - 1) / nt), symmetric ? 256 / nt : 0};
    p.total = p.tiles.total() * count;
    p.cut = OrthoSplit{(int)p.total, 0, 0, num_kb};
    const double block = nt == 256 ? 0.3 : 0.2, part = nt == 256 ? 1.2 : 0.6;
    const int64_t left = p.total % pairs, turns = p.total / pairs;
    double last = left ? num_kb * block : 0;
    if (left && num_kb >= kOrthoFewest) {
        const int64_t most = pairs < kOrthoRuns ? pairs : kOrthoRuns, blocks = left * num_kb;
        for (int64_t runs = left + 1; runs <= most && runs <= 8 * left; ++runs) {
            const int64_t each = (blocks + runs - 1) / runs, parts = (runs + left - 1) / left + (runs % left ? 1 : 0);
            const double us = (double)each * block + (double)parts * part + (turns ? 0 : 2.4);
            if (each >= 4 && us < last - 0.5) {
                last = us;
                p.cut.split = (int)left;
                p.cut.runs = (int)runs;
            }
        }
    }
    p.us = (double)turns * num_kb * block + last;
    return p;
}

inline OrthoPlan ortho_plan(int64_t M, int64_t N, bool symmetric, int num_kb, int count, int pairs) {
    const OrthoPlan wide = ortho_plan_of(M, N, symmetric, num_kb, count, pairs, 256);
    const OrthoPlan narrow = ortho_plan_of(M, N, symmetric, num_kb, count, pairs, 128);
    return narrow.us < wide.us ? narrow : wide;
}

// The workspace: where each part begins, in bytes; pitches in elements.
struct OrthoWork {
    int64_t xpitch, gpitch, short_side;
    size_t scale, sums, counts, x0, x1, g, p, parts, bytes;
};

// Partial sums of a matrix's norm, at most: 512 for one matrix, and as many for all of a stack together, rounded up to
// whole ones for each.  (512 a matrix were 268 MB for 65535 of any size.)
constexpr int kOrthoParts = 512;
inline int ortho_parts(int count) { return count ? (kOrthoParts + count - 1) / count : 0; }

inline OrthoWork ortho_work(int64_t rows, int64_t cols, int count) {
    OrthoWork w;
    w.short_side = rows < cols ? rows : cols;
    w.xpitch = (cols + 15) / 16 * 16;  // rows of whole 32-byte sectors
    w.gpitch = (w.short_side + 15) / 16 * 16;
    size_t at = 0;
    auto part = [&](size_t bytes) {
        const size_t from = at;
        at += (bytes + 255) / 256 * 256;
        return from;
    };
    w.scale = part((size_t)count * sizeof(float));
    w.sums = part((size_t)count * (size_t)ortho_parts(count) * sizeof(double));
    w.counts = part((size_t)kOrthoRuns * 16 * sizeof(int));
    const size_t x = (size_t)count * (size_t)rows * (size_t)w.xpitch * 2;
    const size_t g = (size_t)count * (size_t)w.short_side * (size_t)w.gpitch * 2;
    w.x0 = part(x);
    w.x1 = part(x);
    w.g = part(g);
    w.p = part(g);
    // (no product of fewer K blocks is cut)
    w.parts = part(rows > (kOrthoFewest - 1) * 64 || cols > (kOrthoFewest - 1) * 64 ? (size_t)kOrthoRuns * 2 * 256 * 256 * sizeof(float) : 0);
    w.bytes = at;
    return w;
}

}  // namespace c3
