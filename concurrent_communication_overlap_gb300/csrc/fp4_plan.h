// fp4_plan.h -- which form a product of 4-bit matrices takes (fp4_gemm.cu has the
// kernels).  Host arithmetic alone, so that it can be checked without a GPU.
#pragma once

#include <cstdint>

namespace c3 {

constexpr int kTileRows = 128;  // rows of a scale tile; an expert's rows start at a multiple of it
constexpr int kFK = 256;        // columns of a stage: 128 bytes of codes
constexpr int kPN = 192;        // columns of one accumulator of the form for many rows

#ifdef __CUDACC__
#define C3_BOTH __host__ __device__
#else
#define C3_BOTH
#endif

// Row tiles of the experts up to one: `before` and `more`, at most `limit`.  Experts whose rows
// do not overlap have no more than a matrix's tiles and one for each, which the host has found
// to be few enough for 32 bits; counts from the device that say otherwise stop there.
C3_BOTH inline int tiles_up_to(int64_t before, int64_t more, int64_t limit) {
    return (int)(before + more < limit ? before + more : limit);
}

// How a product runs: rows and columns of a tile (512 x 192, 256 x 384 or 256 x 192
// on two SMs; 128, 64 or 32 x 128 with the roles swapped), and over how many CTAs a
// tile's K is split.
struct Fp4Plan {
    int rows, cols, split, ctas;
};

inline Fp4Plan fp4_plan(int64_t M, int64_t N, int64_t K, int experts, bool grouped, int cap, int sms) {
    Fp4Plan p{};
    const int64_t kb = (K + kFK - 1) / kFK;
    auto up = [](int64_t a, int64_t b) { return (a + b - 1) / b; };
    // Rows an expert has on average: the buffer's, less the padding that it has room for
    // (c3_moe_rows).  The counts are on the device: a buffer with far more room than a call's
    // tokens need is planned for as if it were full.
    const int64_t pad = (int64_t)(kTileRows - 1) * experts;
    const int64_t per = !grouped ? M : M > pad ? (M - pad) / experts : 0;
    // Above 128 rows the form for few rows reads the weights once for every 128 of them (us by
    // pairs and by few-row tiles, MX): 160 x 28672 x 8192 30.4 and 44.1, 256 x 28672 x 8192 31.1
    // and 47.0, 256 x 4096 x 4096 10.4 and 13.2.  Up to 64 rows it is the better one, 25.9 against
    // 29.2 and 8.6 against 9.9; of 65 to 128 only where N is large (128 x 28672 x 8192 29.6 against
    // 30.2, but 128 x 4096 x 4096 12.1 against 10.4 and 128 x 8192 x 2048 12.1 against 8.4).
    if (cap >= 2 && per > 128) {
        // Cycles of the busiest pair, from 8192 x 28672 x 8192 in each form (637, 579 and
        // 569 us): a stage of 256 columns of K takes 620 with one accumulator and 1080 with
        // two, whose read-out, 1500, nothing hides, nor the store of the last (256 x 28672 x
        // 8192: 32.8 us in two waves of 192 columns, 34.6 in one of 384).
        const int64_t pairs = cap / 2;
        int64_t best = 0;
        for (int form = 0; form < 3; ++form) {
            const int rows = form == 1 ? 512 : 256, cols = form == 2 ? 2 * kPN : kPN;
            if (grouped && form == 1) continue;  // an expert's last tile would be mostly empty
            // of an expert's rows, half a tile on average is past its count
            const int64_t tiles = grouped ? experts * up(per + rows / 2, rows) : up(M, rows);
            const int64_t cost = up(tiles * up(N, cols), pairs) * (form ? kb * 1080 + 1500 : kb * 620 + 300) + (form ? 6000 : 1200);
            if (best == 0 || cost < best) {
                best = cost;
                p.rows = rows;
                p.cols = cols;
            }
        }
        p.split = 1;
        const int64_t tiles = (up(M, p.rows) + (grouped ? experts : 0)) * up(N, p.cols);
        p.ctas = 2 * (int)(tiles < pairs ? tiles : pairs);
        return p;
    }
    p.rows = grouped ? 64 : per <= 32 ? 32 : per <= 64 ? 64 : 128;
    p.cols = 128;
    const int64_t n = up(N, 128);
    // An expert with any row has whole scale tiles to itself, so busy experts are at
    // most M / 128 and tiles of 64 rows at most M / 64.
    const int64_t tiles = up(M, p.rows) * n;
    const int64_t busy = grouped ? (experts < up(M, kTileRows) ? experts : up(M, kTileRows)) * n : tiles;
    // A budget below the whole machine is kept to the letter: one CTA for each SM of it.
    const int64_t slots = cap < sms ? cap : 2 * (int64_t)cap;
    // The parts' meeting grows with their number and with the rows: up to 8 for 32 rows (32 x
    // 1024 x 8192: 6.6 us with 8, 7.4 with 4, 11.5 with 1), 4 above (100 x 4096 x 4096: 13.3,
    // 11.9 and 11.7; 128 x 8192 x 8192: 15.7 with 4, 20.6 with 1).
    const int most_parts = p.rows == 32 ? 8 : 4;
    p.split = 1;
    while (p.split < most_parts && busy * p.split * 2 <= slots && kb >= 4 * p.split && !(grouped && cap < sms)) p.split *= 2;
    // One wave: of the tiles that the buffer has room for, the counts leave few (26 tokens to
    // 6 of 6 experts of 1440 x 2688, 72 of 168 tiles: a cluster for each takes 3 us more).
    p.ctas = (int)((tiles * p.split < slots ? tiles * p.split : slots) / p.split) * p.split;
    return p;
}

}  // namespace c3
