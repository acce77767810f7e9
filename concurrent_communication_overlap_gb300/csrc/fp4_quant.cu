// fp4_quant.cu -- values to microscaled 4-bit codes and back.
//
// A code has a sign, two exponent bits and one mantissa bit: 0 .5 1 1.5 2 3 4 6.
// MX: 32 consecutive columns share the smallest power of two s with
//     max|x| <= 6 s, kept as its exponent + 127; no element saturates.
// NV: 16 consecutive columns share an e4m3 number s = max|y| / 6, rounded to
//     nearest even and at most 448, where y = x * (1 / g) and g is one fp32
//     number of the whole matrix.
// The code is x / s (y / s) to the nearest value, ties to the even code.  A
// block that holds a NaN or an infinity gets a NaN scale.
//
// Scales lie in tiles of 128 rows x 4 blocks, 512 bytes, in the order in which
// the tensor cores take them: byte (r % 32) * 16 + (r / 32) * 4 + block.
#include "ops_device.cuh"
#include "c3_internal.h"

#include <cuda_bf16.h>

#include <type_traits>

namespace c3 {

constexpr int kQRows = 32;                 // rows of a CTA's tile: one row group of a scale tile
constexpr int kQCols = 256;                // columns of a CTA's tile
constexpr int kQThreads = 256;             // eight threads a row, 16 columns each

// Eight signed values to eight codes, the first in the lowest four bits.
__device__ __forceinline__ uint32_t to_codes(const float* v) {
    uint32_t r;
    asm("{\n\t.reg .b8 a, b, c, d;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
        "mov.b32 %0, {a, b, c, d};\n\t}"
        : "=r"(r)
        : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
    return r;
}

__device__ __forceinline__ uint32_t to_e4m3(float v) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(0.0f), "f"(v));
    return r & 0xffu;
}
__device__ __forceinline__ float from_e4m3(uint32_t b) {
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)b));
    float f;
    asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tcvt.f32.f16 %0, lo;\n\t}" : "=f"(f) : "r"(h));
    return f;
}

// Two fp32 operations an instruction.
__device__ __forceinline__ uint64_t pack2(float a, float b) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ void unpack2(uint64_t v, float& a, float& b) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
// The larger of |a| and |b|; NaN if either is.
__device__ __forceinline__ float max_abs_nan(float a, float b) {
    float r;
    asm("{\n\t.reg .f32 x, y;\n\tabs.f32 x, %1;\n\tabs.f32 y, %2;\n\tmax.NaN.f32 %0, x, y;\n\t}" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

__device__ __forceinline__ uint32_t mx_byte(uint32_t u, bool bad) {
    // amax = m 2^E, m in [1, 2): 6 2^e holds it with e = E - 2 up to m = 1.5, with E - 1 above.
    // The biased exponent of a subnormal is 0: what follows clamps at 0 anyway.
    const int e = (int)(u >> 23) - 2 + ((u & 0x7fffffu) > 0x400000u ? 1 : 0);
    return bad ? 0xffu : (uint32_t)min(max(e, 0), 253);
}

// Codes of 16 values whose block has the largest magnitude amax (NaN if one of them is).
template <bool NV>
__device__ __forceinline__ void encode16(float (&v)[16], float amax, uint32_t& byte, uint2& codes) {
    const bool bad = !(amax <= 3.402823466e38f);
    if (!NV) {
        byte = mx_byte(__float_as_uint(amax), bad);
        const float inv = __uint_as_float((254u - min(byte, 253u)) << 23);  // 2^-e
        const uint64_t i2 = pack2(inv, inv);
#pragma unroll
        for (int i = 0; i < 16; i += 2) unpack2(mul2(pack2(v[i], v[i + 1]), i2), v[i], v[i + 1]);
    } else {
        // amax / 6 and 1 / s, correctly rounded, by one correction each (Markstein, IBM J. Res.
        // Dev. 34, 1990): of a product with the rounded 1 / 6 (a quotient so small that the
        // remainder underflows is scale 0 either way), and of the reciprocal instruction's result,
        // which is off by an ulp at most (s has four bits, so its significand is not all ones).
        const float sixth = 1.0f / 6.0f, quot = amax * sixth;
        byte = to_e4m3(fmaf(fmaf(-6.0f, quot, amax), sixth, quot));
        const float s = from_e4m3(byte);
        float inv;
        asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(inv) : "f"(s));
        inv = byte ? fmaf(inv, fmaf(-s, inv, 1.0f), inv) : 0.0f;
        const uint64_t i2 = pack2(inv, inv), s2 = pack2(-s, -s);
        // v / s, correctly rounded, from the rounded reciprocal and one correction by the
        // remainder (Markstein, IBM J. Res. Dev. 34, 1990); what is so small that the
        // remainder underflows rounds to code 0 either way.  A scale of 0 makes every code 0.
#pragma unroll
        for (int i = 0; i < 16; i += 2) {
            const uint64_t x = pack2(v[i], v[i + 1]), q = mul2(x, i2);
            unpack2(fma2(fma2(q, s2, x), i2, q), v[i], v[i + 1]);
        }
        if (bad) byte = 0x7fu;
    }
    codes.x = to_codes(v);
    codes.y = to_codes(v + 8);
    if (NV && byte == 0u) codes.x = codes.y = 0u;
}
// The largest magnitude of the block of 16 (NV) or 32 (MX: the other half is with lane ^ 1) values.
template <bool NV>
__device__ __forceinline__ float block_max(const float (&v)[16]) {
    float amax = max_abs_nan(v[0], v[1]);
#pragma unroll
    for (int i = 2; i < 16; ++i) amax = max_abs_nan(amax, v[i]);
    return NV ? amax : max_abs_nan(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
}

// ---- bf16 rows to MX codes, two values an instruction
//
// The conversion instruction to 4-bit codes is slow: alone it bounds the
// quantisation of 8192 x 8192 at about 29 us.  Half the columns take it, the other
// half the same rounding in packed bf16 arithmetic, so that neither pipe waits for
// the other.  With a = |x / scale| <= 6, exact in bf16, and p the power of two below
// max(a, 1): codes step by p / 2 around a, and so do bf16 numbers around 96 p, so
// r = a + 96 p is rounded to nearest even at the right place, and
//   code = (r's low three bits) + 2 log2(p), the latter in r's exponent.
__device__ __forceinline__ uint32_t bmul2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
__device__ __forceinline__ uint32_t bfma2(uint32_t a, uint32_t b, uint32_t c) {
    uint32_t r;
    asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(c));
    return r;
}
__device__ __forceinline__ uint32_t bmax2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("max.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
__device__ __forceinline__ uint32_t bmax2_nan(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
// Two codes, in the low four bits of either half.
__device__ __forceinline__ uint32_t two_codes(uint32_t y) {
    const uint32_t a = y & 0x7fff7fffu;
    const uint32_t p = bmax2(a, 0x3f803f80u) & 0x7f807f80u;
    const uint32_t r = bfma2(p, 0x42c042c0u, a);  // 96; the exponent's low bits are 1 + log2(p)
    return ((r & 0x00070007u) + ((r >> 6) & 0x00060006u) - 0x00020002u) | ((y >> 12) & 0x00080008u);
}
// Eight values in memory order, as four words of two, times `inv`, to eight codes.
__device__ __forceinline__ uint32_t eight_codes(const uint32_t* w, uint32_t inv) {
    // (0, 4) (1, 5) (2, 6) (3, 7): the halves of the result then hold 0..3 and 4..7
    uint32_t r = two_codes(bmul2(__byte_perm(w[0], w[2], 0x5410), inv));
    r |= two_codes(bmul2(__byte_perm(w[0], w[2], 0x7632), inv)) << 4;
    r |= two_codes(bmul2(__byte_perm(w[1], w[3], 0x5410), inv)) << 8;
    r |= two_codes(bmul2(__byte_perm(w[1], w[3], 0x7632), inv)) << 12;
    return r;
}
// The largest magnitude of 16 bf16 values, in the low half, and (MX) of the 16 with lane ^ 1; as fp32 bits.
template <bool NV>
__device__ __forceinline__ uint32_t block_max_bf16(const uint32_t (&w)[8]) {
    uint32_t m = w[0] & 0x7fff7fffu;
#pragma unroll
    for (int i = 1; i < 8; ++i) m = bmax2_nan(m, w[i] & 0x7fff7fffu);
    if (!NV) m = bmax2_nan(m, __shfl_xor_sync(0xffffffffu, m, 1));
    return bmax2_nan(m, m >> 16) << 16;
}
__device__ __forceinline__ void encode16_mx_bf16(const uint32_t (&w)[8], uint32_t& byte, uint2& codes) {
    const uint32_t u = block_max_bf16<false>(w);
    byte = mx_byte(u, u >= 0x7f800000u);
    const uint32_t inv = ((254u - min(byte, 253u)) << 7) * 0x00010001u;  // 2^-e in both halves
    codes.x = eight_codes(w, inv);
    float v[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t y = bmul2(w[4 + i], inv);
        v[2 * i] = __uint_as_float(y << 16);
        v[2 * i + 1] = __uint_as_float(y & 0xffff0000u);
    }
    codes.y = to_codes(v);
}

// The codes and the scale byte of columns c .. c + 15 of row r to their places; every lane of the warp takes part.
template <bool NV>
__device__ __forceinline__ void put16(uint32_t byte, uint2 codes, bool have, const Fp4& q, int64_t mat_row, uint8_t* tile_row,
                                      int64_t c, int64_t pitch, int64_t k_tiles) {
    // The four scales of a tile's row as one word: from lanes 2 apart (MX) or neighbours (NV).
    constexpr int kStep = NV ? 1 : 2;
    const int lane = threadIdx.x & 31;
    const int lead = NV ? (lane & ~3) : (lane & ~7);
    uint32_t word = byte << (8 * ((lane / kStep) & 3));
    word |= __shfl_xor_sync(0xffffffffu, word, kStep);
    word |= __shfl_xor_sync(0xffffffffu, word, 2 * kStep);
    if (!have) return;
    if (c < pitch * 2) *reinterpret_cast<uint2*>(q.codes + mat_row * pitch + c / 2) = codes;
    const int64_t kt = c / (NV ? 64 : 128);
    if (lane == lead && kt < k_tiles) *reinterpret_cast<uint32_t*>(tile_row + kt * 512) = word;
}

// 16 columns of a row as they lie in memory: 8 words of bf16 pairs or 16 of fp32; zeros past `most`.
template <typename T>
struct Raw16 {
    static constexpr int kWords = 4 * sizeof(T);
    uint32_t w[kWords];
    // VEC: every row starts on 16 bytes.  Else the aligned 16-byte pieces around the
    // columns are loaded and shifted into place, if they lie in [lo, hi): 1518 x 16361
    // bf16 takes 16 us that way, 19 a value at a time.
    template <bool VEC>
    __device__ __forceinline__ void load(const T* p, int64_t most, const T* lo, const T* hi) {
        if (VEC && most >= 16) {
#pragma unroll
            for (int i = 0; i < kWords / 4; ++i) {
                const uint4 a = reinterpret_cast<const uint4*>(p)[i];
                w[4 * i] = a.x, w[4 * i + 1] = a.y, w[4 * i + 2] = a.z, w[4 * i + 3] = a.w;
            }
            return;
        }
        if constexpr (!VEC) {
            const uintptr_t from = (uintptr_t)p & ~(uintptr_t)15;
            const unsigned off = (unsigned)(uintptr_t)p & 15u;
            if (most >= 16 && from >= (uintptr_t)lo && from + 4 * (kWords + 4) <= (uintptr_t)hi) {
                uint32_t u[kWords + 4];
#pragma unroll
                for (int i = 0; i <= kWords / 4; ++i) {
                    const uint4 a = reinterpret_cast<const uint4*>(from)[i];
                    u[4 * i] = a.x, u[4 * i + 1] = a.y, u[4 * i + 2] = a.z, u[4 * i + 3] = a.w;
                }
#pragma unroll
                for (int i = 0; i < kWords + 2; ++i) u[i] = off & 8u ? u[i + 2] : u[i];
#pragma unroll
                for (int i = 0; i < kWords + 1; ++i) u[i] = off & 4u ? u[i + 1] : u[i];
#pragma unroll
                for (int i = 0; i < kWords; ++i) w[i] = off & 2u ? __byte_perm(u[i], u[i + 1], 0x5432) : u[i];
                return;
            }
        }
        if constexpr (sizeof(T) == 2) {
            const uint16_t* s = reinterpret_cast<const uint16_t*>(p);
#pragma unroll
            for (int i = 0; i < 8; ++i)
                w[i] = (2 * i < most ? s[2 * i] : 0u) | (2 * i + 1 < most ? (uint32_t)s[2 * i + 1] << 16 : 0u);
        } else {
#pragma unroll
            for (int i = 0; i < 16; ++i) w[i] = i < most ? reinterpret_cast<const uint32_t*>(p)[i] : 0u;
        }
    }
    __device__ __forceinline__ void values(float (&v)[16]) const {
#pragma unroll
        for (int i = 0; i < 16; ++i)
            v[i] = __uint_as_float(sizeof(T) == 4 ? w[i & (kWords - 1)]
                                                  : (i & 1) ? w[i / 2] & 0xffff0000u : w[i / 2] << 16);
    }
};

__device__ __forceinline__ void scale16(float (&v)[16], float t) {
#pragma unroll
    for (int j = 0; j < 16; j += 2) unpack2(mul2(pack2(v[j], v[j + 1]), pack2(t, t)), v[j], v[j + 1]);
}

template <typename T, bool NV>
__device__ __forceinline__ void encode_raw(const Raw16<T>& x, float inv_t, uint32_t& byte, uint2& codes) {
    if constexpr (!NV && sizeof(T) == 2) {
        encode16_mx_bf16(x.w, byte, codes);
    } else {
        float v[16];
        x.values(v);
        // multiplying by a number and rounding keep the order: the maximum may come first.  A block
        // of zeros has scale 0 whatever the matrix's, 1 / 0 for a matrix of zeros by its own maximum.
        float amax;
        if constexpr (sizeof(T) == 2) amax = __uint_as_float(block_max_bf16<NV>(x.w));
        else amax = block_max<NV>(v);
        if (NV) {
            scale16(v, inv_t);
            amax = amax == 0.0f ? 0.0f : amax * fabsf(inv_t);
        }
        encode16<NV>(v, amax, byte, codes);
    }
}

// One CTA: 32 rows of one matrix, 128 columns at a time, `across` CTAs a row tile;
// a thread's next 16 columns are on their way while these are encoded.  Eight
// threads a row: a row's scales of a tile are one word, and codes leave 64 bytes at
// a time.  8192 x 8192 bf16 to MX takes 32 us, 5.3 TB/s; 32768 gathered rows of 4096
// bf16 to NV 54 us, bound by the conversion instruction.
template <typename T, bool NV, bool VEC>
__global__ void __launch_bounds__(kQThreads)
    fp4_quantize_kernel(const T* __restrict__ x, int64_t x_rows, int64_t ld, const int32_t* __restrict__ row_of,
                        Fp4 q, int64_t pitch, int64_t k_tiles, int64_t scale_bytes, int64_t x_stride, unsigned spans,
                        unsigned across) {
    const int i = threadIdx.x >> 3, g = threadIdx.x & 7;
    const unsigned rt = blockIdx.x / across;
    const int64_t r = (int64_t)rt * kQRows + i;
    const int mat = blockIdx.y;
    bool have = r < q.rows;
    int64_t src = r;
    chain_wait();
    if (row_of) {
        if (have) {
            src = row_of[r];
            have = src >= 0 && src < x_rows;
        }
        if (!__any_sync(0xffffffffu, have)) return;  // none of the warp's four rows
    }
    const float inv_t = NV && q.tensor_scale ? __fdiv_rn(1.0f, q.tensor_scale[mat]) : 1.0f;
    uint8_t* tile_row = q.scales + (int64_t)mat * scale_bytes + (r / kTileRows) * k_tiles * 512 + (r % 32) * 16 +
                        (r % kTileRows) / 32 * 4;
    const T* lo = x + (int64_t)mat * x_stride;
    const T* hi = lo + (x_rows - 1) * ld + q.cols;
    const T* xr = lo + src * ld;
    unsigned u = blockIdx.x - rt * across;
    int64_t c = (int64_t)u * 128 + g * 16;
    Raw16<T> now;
    now.template load<VEC>(xr + c, have ? q.cols - c : 0, lo, hi);
    for (; u < spans; u += across) {
        const int64_t next = c + (int64_t)across * 128;
        Raw16<T> ahead;
        ahead.template load<VEC>(xr + next, have && u + across < spans ? q.cols - next : 0, lo, hi);
        uint32_t byte;
        uint2 codes;
        encode_raw<T, NV>(now, inv_t, byte, codes);
        put16<NV>(byte, codes, have, q, (int64_t)mat * q.rows + r, tile_row, c, pitch, k_tiles);
        now = ahead;
        c = next;
    }
}

// The transpose of what lies in memory: 64 rows x 128 columns, turned in shared
// memory, which holds the values of two neighbouring rows as one word, column after
// column.  A lane loads two values of a column at once where PAIRS (else one after
// the other) and encodes 16 columns of two rows.  The columns' skew of 4 (bf16) or 2
// (fp32) words for each 16 lets the lanes of a warp, 4 pairs of rows x 8 lots of 16
// columns, meet in no bank.  All of a thread's loads are on their way before the first
// is stored: 8192 x 8192 bf16 to NV takes 43 us, where a load waited for the store before
// it 133, and with a value at a time, each in a word of its own, 83; fp32 to MX 49 us
// (bytes 45); 2050 x 4100 fp32 to NV 7.4 us.  Four CTAs an SM: three take 48 and 53 us for
// the large ones, five, whose registers spill, 43 and 60.
constexpr int kTRows = 64;
constexpr int kTCols = 128;

template <typename T, bool NV, bool PAIRS>
__global__ void __launch_bounds__(kQThreads, 4)
    fp4_quantize_turned_kernel(const T* __restrict__ x, int64_t ld, Fp4 q, int64_t pitch, int64_t k_tiles,
                               int64_t scale_bytes, int64_t x_stride, unsigned row_tiles) {
    using Two = typename std::conditional<sizeof(T) == 2, uint32_t, uint2>::type;
    constexpr int kSkew = sizeof(T) == 2 ? 4 : 2, kPairs = kTRows / 2, kWarps = kQThreads / 32;
    __shared__ Two tile[kTCols * kPairs + kTCols / 16 * kSkew];
    const int i = threadIdx.x >> 3, g = threadIdx.x & 7, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    // neighbouring CTAs read neighbours in memory
    const unsigned ct = blockIdx.x / row_tiles, rt = blockIdx.x - ct * row_tiles;
    const int64_t c0 = (int64_t)ct * kTCols;
    const int mat = blockIdx.y;
    const int64_t row = (int64_t)rt * kTRows + 2 * lane;  // the lane loads it and the next
    const int most = (int)min((int64_t)kTCols, q.cols - c0);
    const int rows = (int)max((int64_t)0, min((int64_t)2, q.rows - row));
    const T* from = x + (int64_t)mat * x_stride + (c0 + warp) * ld + row;
    chain_wait();
    const float inv_t = NV && q.tensor_scale ? __fdiv_rn(1.0f, q.tensor_scale[mat]) : 1.0f;
    using Bits = typename std::conditional<sizeof(T) == 2, uint16_t, uint32_t>::type;
    Two v[kTCols / kWarps];  // all on their way before the first is stored
#pragma unroll
    for (int n = 0; n < kTCols / kWarps; ++n, from += kWarps * ld) {
        const int have = warp + n * kWarps < most ? rows : 0;
        const Bits* p = reinterpret_cast<const Bits*>(from);
        if constexpr (PAIRS) {
            v[n] = Two{};
            if (have == 2) v[n] = *reinterpret_cast<const Two*>(p);
        } else {
            Bits lo = 0, hi = 0;
            if (have > 0) lo = p[0];
            if (have > 1) hi = p[1];
            if constexpr (sizeof(T) == 2)
                v[n] = lo | (uint32_t)hi << 16;
            else
                v[n] = make_uint2(lo, hi);
        }
    }
    if (PAIRS && rows == 1) {  // an odd number of rows
        from -= kTCols * ld;
#pragma unroll 1
        for (int n = 0; n < kTCols / kWarps; ++n, from += kWarps * ld) {
            if (warp + n * kWarps >= most) break;
            const Bits last = *reinterpret_cast<const Bits*>(from);
            tile[(warp + n * kWarps) * kPairs + n / 2 * kSkew + lane] = Two{last};
        }
    }
#pragma unroll
    for (int n = 0; n < kTCols / kWarps; ++n)
        if (!(PAIRS && rows == 1 && warp + n * kWarps < most))
            tile[(warp + n * kWarps) * kPairs + n / 2 * kSkew + lane] = v[n];
    __syncthreads();
    Two u[16];
#pragma unroll
    for (int j = 0; j < 16; ++j) u[j] = tile[(g * 16 + j) * kPairs + g * kSkew + i];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        Raw16<T> raw;
#pragma unroll
        for (int j = 0; j < Raw16<T>::kWords; ++j) {
            if constexpr (sizeof(T) == 2)
                raw.w[j] = __byte_perm(u[2 * j], u[2 * j + 1], h ? 0x7632 : 0x5410);
            else
                raw.w[j] = h ? u[j].y : u[j].x;
        }
        uint32_t byte;
        uint2 codes;
        encode_raw<T, NV>(raw, inv_t, byte, codes);
        const int64_t r = (int64_t)rt * kTRows + 2 * i + h;
        uint8_t* tile_row = q.scales + (int64_t)mat * scale_bytes + (r / kTileRows) * k_tiles * 512 + (r % 32) * 16 +
                            (r % kTileRows) / 32 * 4;
        put16<NV>(byte, codes, r < q.rows, q, (int64_t)mat * q.rows + r, tile_row, c0 + g * 16, pitch, k_tiles);
    }
}

// Eight codes, the first in the lowest four bits, as bf16 pairs in order.  A
// code's three magnitude bits pick the two bytes of its bf16 number out of tables
// in registers (0 .5 1 1.5 2 3 4 6 are 0000 3f00 3f80 3fc0 4000 4040 4080 40c0); the
// sign, the selector's top bit, spreads the sign bit of a table of 80s to ff.
__device__ __forceinline__ void from_codes(uint32_t w, uint32_t (&v)[4]) {
    const uint32_t m = w & 0x77777777u;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const uint32_t sel = h ? m >> 16 : m & 0xffffu, all = h ? w >> 16 : w & 0xffffu;
        const uint32_t hi = __byte_perm(0x3f3f3f00u, 0x40404040u, sel);
        const uint32_t lo = __byte_perm(0xc0800000u, 0xc0804000u, sel);
        uint32_t sign;  // the intrinsic masks the replicating bit of its selector, the instruction does not
        asm("prmt.b32 %0, %1, %1, %2;" : "=r"(sign) : "r"(0x80808080u), "r"(all));
        const uint32_t top = hi | ((sign << 1) & 0x80808080u);
        v[2 * h] = __byte_perm(lo, top, 0x5140);
        v[2 * h + 1] = __byte_perm(lo, top, 0x7362);
    }
}

__device__ __forceinline__ void store_v(float* p, float v) { *p = v; }
__device__ __forceinline__ void store_v(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }

__device__ __forceinline__ void store8(float* dst, const float (&v)[8]) {
    reinterpret_cast<float4*>(dst)[0] = make_float4(v[0], v[1], v[2], v[3]);
    reinterpret_cast<float4*>(dst)[1] = make_float4(v[4], v[5], v[6], v[7]);
}
__device__ __forceinline__ void store8(__nv_bfloat16* dst, const float (&v)[8]) {
    uint32_t u[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * j], v[2 * j + 1]);
        u[j] = *reinterpret_cast<const uint32_t*>(&h);
    }
    *reinterpret_cast<uint4*>(dst) = make_uint4(u[0], u[1], u[2], u[3]);
}

// One CTA: 32 rows x 256 columns.  A warp takes four rows, a lane 8 columns of
// each, so that a warp reads and writes whole runs (8192 x 8192 to bf16: 29 us, 5.8 TB/s).  VEC: rows of x are whole
// 16-byte units; else a row goes through shared memory and out a value a lane.
template <typename T, bool NV, bool VEC>
__global__ void __launch_bounds__(kQThreads)
    fp4_dequantize_kernel(Fp4 q, int64_t pitch, int64_t k_tiles, int64_t scale_bytes, T* __restrict__ x, int64_t ld,
                          unsigned col_tiles) {
    constexpr int kWarps = kQThreads / 32, kRows = kQRows / kWarps;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const unsigned rt = blockIdx.x / col_tiles;
    const int64_t c0 = (int64_t)(blockIdx.x - rt * col_tiles) * kQCols, c = c0 + lane * 8;
    const int64_t row0 = (int64_t)rt * kQRows;
    const int mat = blockIdx.y;
    const bool in = c < q.cols;
    const uint8_t* codes = q.codes + ((int64_t)mat * q.rows + row0) * pitch + c / 2;
    const int64_t blk = c / (NV ? 16 : 32);
    const uint8_t* scales = q.scales + (int64_t)mat * scale_bytes + ((row0 / kTileRows) * k_tiles + blk / 4) * 512 +
                            (row0 % kTileRows) / 32 * 4 + blk % 4;
    uint32_t w[kRows], byte[kRows];
    chain_wait();
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
        const int r = warp + i * kWarps;
        const bool have = in && row0 + r < q.rows;
        w[i] = have ? __ldcs(reinterpret_cast<const uint32_t*>(codes + r * pitch)) : 0u;
        byte[i] = have ? scales[r * 16] : 0u;
    }
    const float t = q.tensor_scale ? q.tensor_scale[mat] : 1.0f;
    __shared__ __align__(16) T turn[VEC ? 1 : kWarps][VEC ? 8 : kQCols];
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
        const int64_t r = row0 + warp + i * kWarps;
        if (r >= q.rows) break;
        uint32_t p[4];
        from_codes(w[i], p);
        T* row = x + ((int64_t)mat * q.rows + r) * ld;
        if constexpr (!NV && sizeof(T) == 2) {
            // a code times a power of two is a bf16 number: no rounding, no detour by fp32
            const uint32_t s = byte[i] == 255u ? 0x7fc0u : byte[i] ? byte[i] << 7 : 0x40u;
#pragma unroll
            for (int j = 0; j < 4; ++j) p[j] = bmul2(p[j], s * 0x00010001u);
            if (VEC && c + 8 <= q.cols) {
                *reinterpret_cast<uint4*>(row + c) = make_uint4(p[0], p[1], p[2], p[3]);
                continue;
            }
        }
        float v[8];
        const float s = NV ? from_e4m3(byte[i])
                           : sizeof(T) == 2 ? 1.0f
                           : byte[i] == 255u ? NAN : __uint_as_float(byte[i] ? byte[i] << 23 : 1u << 22);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            v[2 * j] = __uint_as_float(p[j] << 16) * s * t;
            v[2 * j + 1] = __uint_as_float(p[j] & 0xffff0000u) * s * t;
        }
        if constexpr (VEC) {
            if (c + 8 <= q.cols) {
                store8(row + c, v);
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    if (c + j < q.cols) store_v(row + c + j, v[j]);
            }
        } else {
            store8(&turn[warp][lane * 8], v);
            __syncwarp();
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (c0 + j * 32 + lane < q.cols) row[c0 + j * 32 + lane] = turn[warp][j * 32 + lane];
            __syncwarp();
        }
    }
}

// ---------------------------------------------------------------- host side

// `per_tile` CTAs for each `rows` rows of each matrix.
static int fp4_grid(const Fp4& q, int rows, int64_t per_tile, dim3* grid) {
    const int64_t n = (q.rows + rows - 1) / rows * per_tile;
    if (n > 0x7fffffff || q.count > 65535) return set_error(-5, "4-bit matrix has too many tiles for one launch");
    *grid = dim3((unsigned)n, (unsigned)q.count);
    return 0;
}

static bool vec_ok(const void* p, int64_t ld, int bf16) {
    return ((uintptr_t)p & 15u) == 0 && (ld * (bf16 ? 2 : 4)) % 16 == 0;
}

int fp4_quantize_launch(const void* x, int bf16, int64_t x_rows, int64_t ld, int transpose, const int32_t* row_of,
                        const Fp4& q, cudaStream_t s) {
    dim3 grid;
    // a k tile's padding is written too: MX tiles are 128 columns wide, NV tiles 64
    const int64_t cols = q.k_tiles() * (q.nv ? 64 : 128);
    const int64_t stride = (transpose ? q.cols : x_rows) * ld;
    int rc;
    cudaError_t e;
    if (transpose) {
        const unsigned col_tiles = (unsigned)((cols + kTCols - 1) / kTCols);
        if ((rc = fp4_grid(q, kTRows, col_tiles, &grid))) return rc;
        const unsigned row_tiles = (unsigned)((q.rows + kTRows - 1) / kTRows);
        const bool pairs = (uintptr_t)x % (bf16 ? 4 : 8) == 0 && ld % 2 == 0;
#define C3_GO(T_, NV_, PAIRS_)                                                                                  \
    e = launch_chained(fp4_quantize_turned_kernel<T_, NV_, PAIRS_>, grid, kQThreads, 0, s, 1,                     \
                       static_cast<const T_*>(x), ld, q, q.pitch(), q.k_tiles(), q.scale_bytes(), stride, row_tiles)
#define C3_PICK(T_)                                    \
    do {                                               \
        if (q.nv && pairs) C3_GO(T_, true, true);      \
        else if (q.nv) C3_GO(T_, true, false);         \
        else if (pairs) C3_GO(T_, false, true);        \
        else C3_GO(T_, false, false);                  \
    } while (0)
        if (bf16) C3_PICK(__nv_bfloat16);
        else C3_PICK(float);
#undef C3_PICK
#undef C3_GO
    } else {
        // Up to eight spans of 128 columns a CTA, so that loads run ahead, but six CTAs an
        // SM first, which is one wave: 4096 x 4096 bf16 to MX takes 8.8 us, with one span a
        // CTA 12.3, with sixteen an SM's share 12.3 and with two 13.1.  Gathered rows are
        // mostly absent when each expert has a handful, and a CTA that finds none of its 32
        // leaves: eight (192 of 8320 rows of 4096: 6.9 us, with six 7.8, with sixteen 6.2; 4096 of
        // 12224: 10.9 with six and eight, 11.8 with sixteen).
        const unsigned spans = (unsigned)((cols + 127) / 128);
        const int64_t tiles = (q.rows + kQRows - 1) / kQRows * q.count;
        DeviceState* ds = device_state();
        if (!ds) return -3;
        const int64_t share = tiles * spans / ((int64_t)ds->sm_count * (row_of ? 8 : 6));
        const unsigned each = (unsigned)(share < 1 ? 1 : share < 8 ? share : 8), across = (spans + each - 1) / each;
        if ((rc = fp4_grid(q, kQRows, across, &grid))) return rc;
        const bool vec = vec_ok(x, ld, bf16) && (q.count == 1 || (stride * (bf16 ? 2 : 4)) % 16 == 0);
#define C3_GO(T_, NV_, VEC_)                                                                                   \
    e = launch_chained(fp4_quantize_kernel<T_, NV_, VEC_>, grid, kQThreads, 0, s, 1, static_cast<const T_*>(x),  \
                       x_rows, ld, row_of, q, q.pitch(), q.k_tiles(), q.scale_bytes(), stride, spans, across)
#define C3_PICK(T_)                                  \
    do {                                             \
        if (q.nv && vec) C3_GO(T_, true, true);      \
        else if (q.nv) C3_GO(T_, true, false);       \
        else if (vec) C3_GO(T_, false, true);        \
        else C3_GO(T_, false, false);                \
    } while (0)
        if (bf16) C3_PICK(__nv_bfloat16);
        else C3_PICK(float);
#undef C3_PICK
#undef C3_GO
    }
    if (e != cudaSuccess) return set_cuda_error(e, "4-bit quantise kernel launch");
    count_launch();
    return 0;
}

int fp4_dequantize_launch(const Fp4& q, void* x, int bf16, int64_t ld, cudaStream_t s) {
    dim3 grid;
    const unsigned col_tiles = (unsigned)((q.cols + kQCols - 1) / kQCols);
    int rc = fp4_grid(q, kQRows, col_tiles, &grid);
    if (rc) return rc;
    const bool vec = vec_ok(x, ld, bf16);
    cudaError_t e;
#define C3_GO(T_, NV_, VEC_)                                                                                 \
    e = launch_chained(fp4_dequantize_kernel<T_, NV_, VEC_>, grid, kQThreads, 0, s, 1, q, q.pitch(), q.k_tiles(), \
                       q.scale_bytes(), static_cast<T_*>(x), ld, col_tiles)
#define C3_PICK(T_)                                  \
    do {                                             \
        if (q.nv && vec) C3_GO(T_, true, true);      \
        else if (q.nv) C3_GO(T_, true, false);       \
        else if (vec) C3_GO(T_, false, true);        \
        else C3_GO(T_, false, false);                \
    } while (0)
    if (bf16) C3_PICK(__nv_bfloat16);
    else C3_PICK(float);
#undef C3_PICK
#undef C3_GO
    if (e != cudaSuccess) return set_cuda_error(e, "4-bit dequantise kernel launch");
    count_launch();
    return 0;
}

}  // namespace c3
