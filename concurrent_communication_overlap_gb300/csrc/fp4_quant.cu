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

namespace c3 {

constexpr int kQRows = 32;                 // rows of a CTA's tile: one row group of a scale tile
constexpr int kQCols = 128;                // columns of a CTA's tile
constexpr int kQThreads = kQRows * kQCols / 16;  // a thread takes 16 columns of a row

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

// Scale byte and codes of 16 columns a thread.  MX: the thread's neighbour (lane ^ 1) holds the block's other half.
template <bool NV>
__device__ __forceinline__ void encode16(float (&v)[16], uint32_t& byte, uint2& codes) {
    float amax = 0.0f;
    bool bad = false;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        const float a = fabsf(v[i]);
        bad |= !(a <= 3.402823466e38f);
        amax = fmaxf(amax, a);
    }
    if (!NV) {
        amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
        bad |= __shfl_xor_sync(0xffffffffu, (int)bad, 1) != 0;
        // amax = m 2^E, m in [1, 2): 6 2^e holds it with e = E - 2 up to m = 1.5, with E - 1 above.
        // The biased exponent of a subnormal is 0: what follows clamps at 0 anyway.
        const uint32_t u = __float_as_uint(amax);
        int e = (int)(u >> 23) - 2 + ((u & 0x7fffffu) > 0x400000u ? 1 : 0);
        byte = (uint32_t)max(e, 0);
        const float inv = __uint_as_float((254u - byte) << 23);  // 2^-e; byte is at most 253
#pragma unroll
        for (int i = 0; i < 16; ++i) v[i] *= inv;
        if (bad) byte = 0xffu;
    } else {
        byte = to_e4m3(__fdiv_rn(amax, 6.0f));
        const float s = from_e4m3(byte);
#pragma unroll
        for (int i = 0; i < 16; ++i) v[i] = byte ? __fdiv_rn(v[i], s) : 0.0f;
        if (bad) byte = 0x7fu;
    }
    codes.x = to_codes(v);
    codes.y = to_codes(v + 8);
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

// One CTA: 32 rows x 128 columns of one matrix.  TRANS: the matrix is the
// transpose of what lies in memory, and the tile goes through shared memory.
template <typename T, bool NV, bool TRANS>
__global__ void __launch_bounds__(kQThreads)
    fp4_quantize_kernel(const T* __restrict__ x, int64_t x_rows, int64_t ld, int vec, const int32_t* __restrict__ row_of,
                        Fp4 q, int64_t pitch, int64_t k_tiles, int64_t scale_bytes, int64_t x_stride,
                        int64_t col_tiles) {
    const int i = threadIdx.x >> 3, g = threadIdx.x & 7;
    const int64_t rt = (int64_t)blockIdx.x / col_tiles;
    const int64_t c0 = ((int64_t)blockIdx.x - rt * col_tiles) * kQCols;
    const int64_t r = rt * kQRows + i, c = c0 + g * 16;
    const int mat = blockIdx.y;
    x += (int64_t)mat * x_stride;
    float v[16];
    bool have = r < q.rows;
    if constexpr (TRANS) {
        __shared__ float tile[kQCols][kQRows + 1];
        for (int j = threadIdx.x; j < kQRows * kQCols; j += kQThreads) {
            const int cc = j >> 5, rr = j & 31;
            const int64_t col = c0 + cc, row = rt * kQRows + rr;
            tile[cc][rr] = (col < q.cols && row < q.rows) ? load1(x + col * ld + row) : 0.0f;
        }
        __syncthreads();
#pragma unroll
        for (int j = 0; j < 16; ++j) v[j] = tile[g * 16 + j][i];
    } else {
        int64_t src = r;
        if (have && row_of) {
            src = row_of[r];
            have = src >= 0 && src < x_rows;
        }
        if (have && vec && c + 16 <= q.cols) {
            load16(x + src * ld + c, v);
        } else {
#pragma unroll
            for (int j = 0; j < 16; ++j) v[j] = (have && c + j < q.cols) ? load1(x + src * ld + c + j) : 0.0f;
        }
    }
    if (NV && q.tensor_scale) {
        const float inv = __fdiv_rn(1.0f, q.tensor_scale[mat]);
#pragma unroll
        for (int j = 0; j < 16; ++j) v[j] *= inv;
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
    if (c < pitch * 2) *reinterpret_cast<uint2*>(q.codes + ((int64_t)mat * q.rows + r) * pitch + c / 2) = codes;
    const int64_t kt = c / (NV ? 64 : 128);
    if (lane == lead && kt < k_tiles)
        *reinterpret_cast<uint32_t*>(q.scales + (int64_t)mat * scale_bytes + ((r / kTileRows) * k_tiles + kt) * 512 +
                                     (r % 32) * 16 + (r % kTileRows) / 32 * 4) = word;
}

__device__ __forceinline__ float code_value(uint32_t c) {
    // halves of 0 1 2 3 4 6 8 12, from the exponent and mantissa bits
    const uint32_t e = (c >> 1) & 3u, m = c & 1u;
    const float a = e ? (float)((2u + m) << (e - 1)) * 0.5f : (float)m * 0.5f;
    return (c & 8u) ? -a : a;
}

__device__ __forceinline__ void store_v(float* p, float v) { *p = v; }
__device__ __forceinline__ void store_v(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }

template <typename T, bool NV>
__global__ void __launch_bounds__(kQThreads)
    fp4_dequantize_kernel(Fp4 q, int64_t pitch, int64_t k_tiles, int64_t scale_bytes, T* __restrict__ x, int64_t ld,
                          int vec, int64_t col_tiles) {
    const int i = threadIdx.x >> 3, g = threadIdx.x & 7;
    const int64_t rt = (int64_t)blockIdx.x / col_tiles;
    const int64_t c = ((int64_t)blockIdx.x - rt * col_tiles) * kQCols + g * 16;
    const int64_t r = rt * kQRows + i;
    const int mat = blockIdx.y;
    if (r >= q.rows || c >= q.cols) return;
    const uint2 w = *reinterpret_cast<const uint2*>(q.codes + ((int64_t)mat * q.rows + r) * pitch + c / 2);
    const int64_t blk = c / (NV ? 16 : 32);
    const uint32_t byte = q.scales[(int64_t)mat * scale_bytes + ((r / kTileRows) * k_tiles + blk / 4) * 512 +
                                   (r % 32) * 16 + (r % kTileRows) / 32 * 4 + blk % 4];
    float s;
    if (NV)
        s = from_e4m3(byte);
    else
        s = byte == 255u ? NAN : byte ? __uint_as_float(byte << 23) : __uint_as_float(1u << 22);
    const float t = q.tensor_scale ? q.tensor_scale[mat] : 1.0f;
    float v[16];
#pragma unroll
    for (int j = 0; j < 16; ++j) v[j] = code_value((j < 8 ? w.x >> (4 * j) : w.y >> (4 * (j - 8))) & 15u) * s * t;
    T* dst = x + ((int64_t)mat * q.rows + r) * ld + c;
    if (vec && c + 16 <= q.cols) {
        if constexpr (sizeof(T) == 4) {
#pragma unroll
            for (int j = 0; j < 4; ++j)
                reinterpret_cast<float4*>(dst)[j] = make_float4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
        } else {
            uint32_t u[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * j], v[2 * j + 1]);
                u[j] = *reinterpret_cast<const uint32_t*>(&h);
            }
            reinterpret_cast<uint4*>(dst)[0] = make_uint4(u[0], u[1], u[2], u[3]);
            reinterpret_cast<uint4*>(dst)[1] = make_uint4(u[4], u[5], u[6], u[7]);
        }
    } else {
#pragma unroll
        for (int j = 0; j < 16; ++j)
            if (c + j < q.cols) store_v(dst + j, v[j]);
    }
}

// ---------------------------------------------------------------- host side

static int fp4_grid(const Fp4& q, int64_t cols_padded, dim3* grid, int64_t* col_tiles) {
    *col_tiles = (cols_padded + kQCols - 1) / kQCols;
    const int64_t n = (q.rows + kQRows - 1) / kQRows * *col_tiles;
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
    int64_t col_tiles;
    // a k tile's padding is written too: MX tiles are 128 columns wide, NV tiles 64
    int rc = fp4_grid(q, q.k_tiles() * (q.nv ? 64 : 128), &grid, &col_tiles);
    if (rc) return rc;
    const int64_t stride = (transpose ? q.cols : x_rows) * ld;
    const int vec = vec_ok(x, ld, bf16) && (q.count == 1 || (stride * (bf16 ? 2 : 4)) % 16 == 0);
#define C3_GO(T_, NV_, TR_)                                                                                       \
    fp4_quantize_kernel<T_, NV_, TR_><<<grid, kQThreads, 0, s>>>(static_cast<const T_*>(x), x_rows, ld, vec, row_of, q, \
                                                                 q.pitch(), q.k_tiles(), q.scale_bytes(), stride, col_tiles)
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
    int64_t col_tiles;
    int rc = fp4_grid(q, q.cols, &grid, &col_tiles);
    if (rc) return rc;
    const int vec = vec_ok(x, ld, bf16);
#define C3_GO(T_, NV_)                                                                                           \
    fp4_dequantize_kernel<T_, NV_><<<grid, kQThreads, 0, s>>>(q, q.pitch(), q.k_tiles(), q.scale_bytes(),         \
                                                              static_cast<T_*>(x), ld, vec, col_tiles)
    if (bf16 && q.nv) C3_GO(__nv_bfloat16, true);
    else if (bf16) C3_GO(__nv_bfloat16, false);
    else if (q.nv) C3_GO(float, true);
    else C3_GO(float, false);
#undef C3_GO
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return set_cuda_error(e, "4-bit dequantise kernel launch");
    count_launch();
    return 0;
}

}  // namespace c3
