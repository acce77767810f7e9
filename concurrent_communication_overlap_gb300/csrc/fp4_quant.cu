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
#include "c3_device.cuh"
#include "c3_internal.h"

#include <cuda_bf16.h>
#include <cuda_fp16.h>

namespace c3 {

constexpr int kQRows = 32;                 // rows of a CTA's tile: one row group of a scale tile
constexpr int kQCols = 256;                // columns of a CTA's tile
constexpr int kQThreads = kQRows * kQCols / 32;  // a thread takes twice 16 columns of a row

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

// Scale byte and codes of 16 columns a thread.  MX: the thread's neighbour (lane ^ 1) holds the block's other half.
template <bool NV>
__device__ __forceinline__ void encode16(float (&v)[16], uint32_t& byte, uint2& codes) {
    float amax = max_abs_nan(v[0], v[1]);
#pragma unroll
    for (int i = 2; i < 16; ++i) amax = max_abs_nan(amax, v[i]);
    if (!NV) amax = max_abs_nan(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
    const bool bad = !(amax <= 3.402823466e38f);
    if (!NV) {
        // amax = m 2^E, m in [1, 2): 6 2^e holds it with e = E - 2 up to m = 1.5, with E - 1 above.
        // The biased exponent of a subnormal is 0: what follows clamps at 0 anyway.
        const uint32_t u = __float_as_uint(amax);
        const int e = (int)(u >> 23) - 2 + ((u & 0x7fffffu) > 0x400000u ? 1 : 0);
        byte = (uint32_t)min(max(e, 0), 253);
        const float inv = __uint_as_float((254u - byte) << 23);  // 2^-e
        const uint64_t i2 = pack2(inv, inv);
#pragma unroll
        for (int i = 0; i < 16; i += 2) unpack2(mul2(pack2(v[i], v[i + 1]), i2), v[i], v[i + 1]);
        if (bad) byte = 0xffu;
    } else {
        byte = to_e4m3(__fdiv_rn(amax, 6.0f));
        const float s = from_e4m3(byte);
        const float inv = byte ? __frcp_rn(s) : 0.0f;
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

__device__ __forceinline__ void load16(const float* p, float (&v)[16]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float4 a = reinterpret_cast<const float4*>(p)[i];
        v[4 * i] = a.x, v[4 * i + 1] = a.y, v[4 * i + 2] = a.z, v[4 * i + 3] = a.w;
    }
}
__device__ __forceinline__ void load16(const __nv_bfloat16* p, float (&v)[16]) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const uint4 a = reinterpret_cast<const uint4*>(p)[h];
        const uint32_t u[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[8 * h + 2 * i] = __uint_as_float(u[i] << 16);
            v[8 * h + 2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
        }
    }
}
__device__ __forceinline__ float load1(const float* p) { return *p; }
__device__ __forceinline__ float load1(const __nv_bfloat16* p) { return __bfloat162float(*p); }

// Columns c .. c + 15 of row r, encoded, to their places; every lane of the warp takes part.
template <bool NV>
__device__ __forceinline__ void put16(float (&v)[16], bool have, float inv_t, const Fp4& q, int64_t mat_row, uint8_t* tile_row,
                                      int64_t c, int64_t pitch, int64_t k_tiles) {
    if (NV) {
#pragma unroll
        for (int j = 0; j < 16; j += 2) unpack2(mul2(pack2(v[j], v[j + 1]), pack2(inv_t, inv_t)), v[j], v[j + 1]);
    }
    uint32_t byte;
    uint2 codes;
    encode16<NV>(v, byte, codes);
    // The four scales of a tile's row as one word: from lanes 2 apart (MX) or neighbours (NV).
    constexpr int kStep = NV ? 1 : 2;
    const int lane = threadIdx.x & 31;
    const int lead = NV ? (lane & ~3) : (lane & ~7);
    uint32_t word = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) word |= __shfl_sync(0xffffffffu, byte, lead + j * kStep) << (8 * j);
    if (!have) return;
    if (c < pitch * 2) *reinterpret_cast<uint2*>(q.codes + mat_row * pitch + c / 2) = codes;
    const int64_t kt = c / (NV ? 64 : 128);
    if (lane == lead && kt < k_tiles) *reinterpret_cast<uint32_t*>(tile_row + kt * 512) = word;
}

// One CTA: 32 rows of one matrix, 256 columns at a time, two spans of 16 columns
// a thread, both loaded before either is encoded.  `across` CTAs share a row
// tile's columns.  TRANS: the matrix is the transpose of what lies in memory,
// and a tile goes through shared memory.
template <typename T, bool NV, bool TRANS>
__global__ void __launch_bounds__(kQThreads)
    fp4_quantize_kernel(const T* __restrict__ x, int64_t x_rows, int64_t ld, int vec, const int32_t* __restrict__ row_of,
                        Fp4 q, int64_t pitch, int64_t k_tiles, int64_t scale_bytes, int64_t x_stride, unsigned col_tiles,
                        unsigned across) {
    const int i = threadIdx.x >> 3, g = threadIdx.x & 7;
    const unsigned rt = blockIdx.x / across;
    const int64_t r = (int64_t)rt * kQRows + i;
    const int mat = blockIdx.y;
    x += (int64_t)mat * x_stride;
    bool have = r < q.rows;
    int64_t src = r;
    if (!TRANS && row_of) {
        if (have) {
            src = row_of[r];
            have = src >= 0 && src < x_rows;
        }
        if (!__any_sync(0xffffffffu, have)) return;  // none of the warp's four rows
    }
    const float inv_t = NV && q.tensor_scale ? __fdiv_rn(1.0f, q.tensor_scale[mat]) : 1.0f;
    uint8_t* tile_row = q.scales + (int64_t)mat * scale_bytes + (r / kTileRows) * k_tiles * 512 + (r % 32) * 16 +
                        (r % kTileRows) / 32 * 4;
    for (unsigned ct = blockIdx.x - rt * across; ct < col_tiles; ct += across) {
        const int64_t c0 = (int64_t)ct * kQCols, c = c0 + g * 16;
        float v[2][16];
        if constexpr (TRANS) {
            // rows of shared memory are columns of the matrix; 32 values and one of padding each
            __shared__ float tile[kQCols][kQRows + 1];
            const int rr = threadIdx.x & 31;
            const int64_t row = (int64_t)rt * kQRows + rr;
            const T* from = x + c0 * ld + row;
            const int most = (int)min((int64_t)kQCols, q.cols - c0);
#pragma unroll 16
            for (int cc = threadIdx.x >> 5; cc < kQCols; cc += kQThreads / 32)
                tile[cc][rr] = (cc < most && row < q.rows) ? load1(from + cc * ld) : 0.0f;
            __syncthreads();
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int j = 0; j < 16; ++j) v[h][j] = tile[h * 128 + g * 16 + j][i];
            __syncthreads();
        } else {
            const T* xr = x + src * ld + c;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                if (have && vec && c + h * 128 + 16 <= q.cols) {
                    load16(xr + h * 128, v[h]);
                } else {
#pragma unroll
                    for (int j = 0; j < 16; ++j)
                        v[h][j] = (have && c + h * 128 + j < q.cols) ? load1(xr + h * 128 + j) : 0.0f;
                }
            }
        }
#pragma unroll
        for (int h = 0; h < 2; ++h)
            put16<NV>(v[h], have, inv_t, q, (int64_t)mat * q.rows + r, tile_row, c + h * 128, pitch, k_tiles);
    }
}

// Eight codes, the first in the lowest four bits, as fp32.
__device__ __forceinline__ void from_codes(uint32_t w, float* v) {
    uint32_t h[4];
    asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, a;\n\tcvt.rn.f16x2.e2m1x2 %1, b;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, c;\n\tcvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
        : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
        : "r"(w));
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h[i]));
        v[2 * i] = f.x, v[2 * i + 1] = f.y;
    }
}

__device__ __forceinline__ void store_v(float* p, float v) { *p = v; }
__device__ __forceinline__ void store_v(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }

__device__ __forceinline__ void store16(float* dst, const float (&v)[16]) {
#pragma unroll
    for (int j = 0; j < 4; ++j)
        reinterpret_cast<float4*>(dst)[j] = make_float4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
}
__device__ __forceinline__ void store16(__nv_bfloat16* dst, const float (&v)[16]) {
    uint32_t u[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * j], v[2 * j + 1]);
        u[j] = *reinterpret_cast<const uint32_t*>(&h);
    }
    reinterpret_cast<uint4*>(dst)[0] = make_uint4(u[0], u[1], u[2], u[3]);
    reinterpret_cast<uint4*>(dst)[1] = make_uint4(u[4], u[5], u[6], u[7]);
}

// The same tiles and the same places of a thread as the quantisation.  VEC:
// rows of x are whole 16-byte units and a thread stores its own columns; else the
// tile goes through shared memory and a warp stores 32 neighbours at a time.
template <typename T, bool NV, bool VEC>
__global__ void __launch_bounds__(kQThreads)
    fp4_dequantize_kernel(Fp4 q, int64_t pitch, int64_t k_tiles, int64_t scale_bytes, T* __restrict__ x, int64_t ld,
                          unsigned col_tiles) {
    const int i = threadIdx.x >> 3, g = threadIdx.x & 7;
    const unsigned rt = blockIdx.x / col_tiles;
    const int64_t c0 = (int64_t)(blockIdx.x - rt * col_tiles) * kQCols, c = c0 + g * 16;
    const int64_t r = (int64_t)rt * kQRows + i;
    const int mat = blockIdx.y;
    const uint8_t* codes = q.codes + ((int64_t)mat * q.rows + r) * pitch + c / 2;
    const uint8_t* tile_row = q.scales + (int64_t)mat * scale_bytes + (r / kTileRows) * k_tiles * 512 + (r % 32) * 16 +
                              (r % kTileRows) / 32 * 4;
    constexpr int kBlock = NV ? 16 : 32;
    uint2 w[2] = {};
    uint32_t byte[2] = {};
#pragma unroll
    for (int h = 0; h < 2; ++h)
        if (r < q.rows && c + h * 128 < q.cols) {
            w[h] = __ldcs(reinterpret_cast<const uint2*>(codes + h * 64));
            const int64_t blk = (c + h * 128) / kBlock;
            byte[h] = tile_row[blk / 4 * 512 + blk % 4];
        }
    const float t = q.tensor_scale ? q.tensor_scale[mat] : 1.0f;
    T* dst = x + ((int64_t)mat * q.rows + r) * ld + c;
    __shared__ T tile[VEC ? 1 : kQRows][VEC ? 1 : kQCols + 2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const float s = NV ? from_e4m3(byte[h])
                           : byte[h] == 255u ? NAN : __uint_as_float(byte[h] ? byte[h] << 23 : 1u << 22);
        float v[16];
        from_codes(w[h].x, v);
        from_codes(w[h].y, v + 8);
#pragma unroll
        for (int j = 0; j < 16; ++j) v[j] = v[j] * s * t;
        if constexpr (VEC) {
            if (r < q.rows && c + h * 128 + 16 <= q.cols) {
                store16(dst + h * 128, v);
            } else if (r < q.rows) {
#pragma unroll
                for (int j = 0; j < 16; ++j)
                    if (c + h * 128 + j < q.cols) store_v(dst + h * 128 + j, v[j]);
            }
        } else {
#pragma unroll
            for (int j = 0; j < 16; ++j) store_v(&tile[i][h * 128 + g * 16 + j], v[j]);
        }
    }
    if constexpr (!VEC) {
        __syncthreads();
        const int lane = threadIdx.x & 31;
        for (int rr = threadIdx.x >> 5; rr < kQRows && (int64_t)rt * kQRows + rr < q.rows; rr += kQThreads / 32) {
            T* row = x + ((int64_t)mat * q.rows + (int64_t)rt * kQRows + rr) * ld + c0;
#pragma unroll
            for (int cc = lane; cc < kQCols; cc += 32)
                if (c0 + cc < q.cols) row[cc] = tile[rr][cc];
        }
    }
}

// ---------------------------------------------------------------- host side

// CTAs along the columns of a row tile: all column tiles, or `most` of them.
static int fp4_grid(const Fp4& q, int64_t cols_padded, int64_t most, dim3* grid, unsigned* col_tiles, unsigned* across) {
    *col_tiles = (unsigned)((cols_padded + kQCols - 1) / kQCols);
    *across = *col_tiles > most ? (unsigned)most : *col_tiles;
    const int64_t n = (q.rows + kQRows - 1) / kQRows * *across;
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
    unsigned col_tiles, across;
    // A k tile's padding is written too: MX tiles are 128 columns wide, NV tiles 64.
    // Gathered rows are mostly absent when each expert has a handful, and a CTA that
    // finds none of its 32 leaves: four CTAs a row tile instead of one each 256 columns
    // (8256 x 4096 with 192 rows present: 11 us against 18; all 32768 present: 69 against 91).
    int rc = fp4_grid(q, q.k_tiles() * (q.nv ? 64 : 128), row_of ? 4 : 1 << 30, &grid, &col_tiles, &across);
    if (rc) return rc;
    const int64_t stride = (transpose ? q.cols : x_rows) * ld;
    const int vec = vec_ok(x, ld, bf16) && (q.count == 1 || (stride * (bf16 ? 2 : 4)) % 16 == 0);
#define C3_GO(T_, NV_, TR_)                                                                                       \
    fp4_quantize_kernel<T_, NV_, TR_><<<grid, kQThreads, 0, s>>>(static_cast<const T_*>(x), x_rows, ld, vec, row_of, q, \
                                                                 q.pitch(), q.k_tiles(), q.scale_bytes(), stride, col_tiles, across)
#define C3_PICK(T_)                                       \
    do {                                                  \
        if (q.nv && transpose) C3_GO(T_, true, true);     \
        else if (q.nv) C3_GO(T_, true, false);            \
        else if (transpose) C3_GO(T_, false, true);       \
        else C3_GO(T_, false, false);                     \
    } while (0)
    if (bf16) C3_PICK(__nv_bfloat16);
    else C3_PICK(float);
#undef C3_PICK
#undef C3_GO
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return set_cuda_error(e, "4-bit quantise kernel launch");
    count_launch();
    return 0;
}

int fp4_dequantize_launch(const Fp4& q, void* x, int bf16, int64_t ld, cudaStream_t s) {
    dim3 grid;
    unsigned col_tiles, across;
    int rc = fp4_grid(q, q.cols, 1 << 30, &grid, &col_tiles, &across);
    if (rc) return rc;
    const bool vec = vec_ok(x, ld, bf16);
#define C3_GO(T_, NV_, VEC_)                                                                                     \
    fp4_dequantize_kernel<T_, NV_, VEC_><<<grid, kQThreads, 0, s>>>(q, q.pitch(), q.k_tiles(), q.scale_bytes(),   \
                                                                    static_cast<T_*>(x), ld, col_tiles)
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
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return set_cuda_error(e, "4-bit dequantise kernel launch");
    count_launch();
    return 0;
}

}  // namespace c3
