// route.cu -- routing of tokens to experts: scores, the choice of the best,
// their weights, and the gradient of the weights with respect to the logits.
//
// One warp a token.  Lane l holds the logits of NI consecutive experts, l NI
// and up, in registers.  The choice compares 32-bit integers that order as the
// float keys do: a maximum over the warp is one redux instruction, and of equal
// keys the lowest lane, and in it the lowest register, is the lowest expert.
#include "c3_device.cuh"
#include "c3_internal.h"

#include <cuda_bf16.h>

namespace c3 {

constexpr int kRouteWarps = 8;  // tokens per CTA and pass
constexpr unsigned kFull = 0xffffffffu;

__device__ __forceinline__ float load_f(const float* p) { return __ldg(p); }
__device__ __forceinline__ float load_f(const __nv_bfloat16* p) { return __bfloat162float(*p); }
__device__ __forceinline__ void store_f(float* p, float v) { *p = v; }
__device__ __forceinline__ void store_f(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }

// Whole numbers that order as floats do; -0 and +0 get the same one, and 0 is
// below every float above -inf: it stands for "not eligible".
__device__ __forceinline__ uint32_t order_key(float v) {
    const uint32_t u = __float_as_uint(v + 0.0f);
    return u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
}
__device__ __forceinline__ float order_value(uint32_t k) {
    return __uint_as_float((k & 0x80000000u) ? (k & 0x7fffffffu) : ~k);
}
__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
    for (int o = 16; o; o >>= 1) v = fmaxf(v, __shfl_xor_sync(kFull, v, o));
    return v;
}
__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(kFull, v, o);
    return v;
}
__device__ __forceinline__ float sigmoid_f(float x) { return __frcp_rn(1.0f + expf(-x)); }

// N consecutive logits of a row from expert e0 on; -inf past the last.
template <int N>
__device__ __forceinline__ void load_row(const float* xr, int e0, int E, bool vec, float (&x)[N]) {
    if (vec) {
        if constexpr (N % 4 == 0) {
#pragma unroll
            for (int i = 0; i < N; i += 4) {
                const float4 v = *reinterpret_cast<const float4*>(xr + e0 + i);
                x[i] = v.x, x[i + 1] = v.y, x[i + 2] = v.z, x[i + 3] = v.w;
            }
            return;
        }
    }
#pragma unroll
    for (int i = 0; i < N; ++i) x[i] = e0 + i < E ? load_f(xr + e0 + i) : -INFINITY;
}
template <int N>
__device__ __forceinline__ void load_row(const __nv_bfloat16* xr, int e0, int E, bool vec, float (&x)[N]) {
    if (vec) {
        if constexpr (N % 8 == 0) {
#pragma unroll
            for (int i = 0; i < N; i += 8) {
                const uint4 v = *reinterpret_cast<const uint4*>(xr + e0 + i);
                const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    x[i + 2 * j] = __uint_as_float(u[j] << 16);
                    x[i + 2 * j + 1] = __uint_as_float(u[j] & 0xffff0000u);
                }
            }
            return;
        }
    }
#pragma unroll
    for (int i = 0; i < N; ++i) x[i] = e0 + i < E ? load_f(xr + e0 + i) : -INFINITY;
}

// Groups that are whole runs of 2^j lanes: score and rank them with shuffles.
// Sets the keys of groups outside the best `keep` to 0.
template <int NI>
__device__ __forceinline__ void groups_by_lanes(uint32_t (&key)[NI], int gs, int best_of, int keep, int lane) {
    uint32_t b1 = 0u, b2 = 0u;
#pragma unroll
    for (int i = 0; i < NI; ++i) {
        b2 = max(b2, min(b1, key[i]));
        b1 = max(b1, key[i]);
    }
    const int lanes = gs / NI;
    for (int o = 1; o < lanes; o <<= 1) {
        const uint32_t c1 = __shfl_xor_sync(kFull, b1, o), c2 = __shfl_xor_sync(kFull, b2, o);
        b2 = max(max(b2, c2), min(b1, c1));
        b1 = max(b1, c1);
    }
    const uint32_t score = (best_of == 2 && b2) ? order_key(order_value(b1) + order_value(b2)) : b1;
    const int mine = lane / lanes, groups = 32 / lanes;
    int rank = 0;
    for (int g = 0; g < groups; ++g) {
        const uint32_t other = __shfl_sync(kFull, score, g * lanes);
        rank += other > score || (other == score && g < mine);
    }
    if (rank >= keep) {
#pragma unroll
        for (int i = 0; i < NI; ++i) key[i] = 0u;
    }
}

// Groups of any size, by way of shared memory (1024 words a warp): lane g + 32 j
// takes group g + 32 j, each lane reading from a place of its own on.
template <int NI>
__device__ __forceinline__ void groups_by_memory(uint32_t (&key)[NI], uint32_t* gk, int E, int G, int best_of, int keep,
                                                 int lane) {
    const int gs = E / G;
#pragma unroll
    for (int i = 0; i < NI; ++i)
        if (lane * NI + i < E) gk[lane * NI + i] = key[i];
    __syncwarp();
    uint32_t score[NI];
#pragma unroll
    for (int i = 0; i < NI; ++i) {
        const int g = lane + 32 * i;
        score[i] = 0u;
        if (g < G) {
            uint32_t b1 = 0u, b2 = 0u;
            for (int j = 0, at = g % gs; j < gs; ++j, at = at + 1 == gs ? 0 : at + 1) {
                const uint32_t v = gk[g * gs + at];
                b2 = max(b2, min(b1, v));
                b1 = max(b1, v);
            }
            score[i] = (best_of == 2 && b2) ? order_key(order_value(b1) + order_value(b2)) : b1;
        }
    }
    __syncwarp();
#pragma unroll
    for (int i = 0; i < NI; ++i)
        if (lane + 32 * i < G) gk[lane + 32 * i] = 0u;
    __syncwarp();
    for (int j = 0; j < keep; ++j) {
        uint32_t best = 0u;
#pragma unroll
        for (int i = 0; i < NI; ++i) best = max(best, score[i]);
        best = __reduce_max_sync(kFull, best);
        if (best == 0u) break;
        unsigned at = 0xffffu;
#pragma unroll
        for (int i = NI - 1; i >= 0; --i)
            if (score[i] == best) at = lane + 32 * i;
        at = __reduce_min_sync(kFull, at);
#pragma unroll
        for (int i = 0; i < NI; ++i)
            if ((unsigned)(lane + 32 * i) == at) {
                score[i] = 0u;
                gk[at] = 1u;
            }
    }
    __syncwarp();
#pragma unroll
    for (int i = 0; i < NI; ++i) {
        const int e = lane * NI + i;
        if (e < E && gk[e / gs] == 0u) key[i] = 0u;
    }
    __syncwarp();
}

// Descending order of N keys, by a bitonic network.
template <int N>
__device__ __forceinline__ void sort_down(uint32_t (&k)[N]) {
#pragma unroll
    for (int size = 2; size <= N; size <<= 1)
#pragma unroll
        for (int d = size >> 1; d; d >>= 1)
#pragma unroll
            for (int i = 0; i < N; ++i)
                if ((i & d) == 0) {
                    const uint32_t a = k[i], b = k[i | d];
                    const bool down = (i & size) == 0 || size == N;
                    k[i] = down ? max(a, b) : min(a, b);
                    k[i | d] = down ? min(a, b) : max(a, b);
                }
}

// The weight of this lane's choice (expert `mine`, or -1), unscaled.
template <typename T>
__device__ __forceinline__ float choice_weight(const T* xr, int mine, const RouteArgs& a, float top, float total) {
    const float x = mine >= 0 ? load_f(xr + mine) : -INFINITY;
    if (a.score == 0 && a.renorm) {
        const float m = warp_max(x);
        const float p = mine >= 0 ? expf(x - m) : 0.0f;
        const float s = warp_sum(p);
        return mine >= 0 ? p / s : 0.0f;
    }
    if (a.score == 0) return mine >= 0 ? expf(x - top) / total : 0.0f;
    const float w = mine >= 0 ? sigmoid_f(x) : 0.0f;
    if (!a.renorm) return w;
    const float s = warp_sum(w);
    return s > 0.0f ? w / s : 0.0f;
}

// NI: experts a lane holds, ceil(E / 32) rounded up to a power of two.  GROUPS:
// 0 none, 1 whole runs of lanes, 2 any.  vec: rows are whole and 16-byte aligned.
template <typename T, int NI, int GROUPS>
__global__ void __launch_bounds__(kRouteWarps * 32)
    route_kernel(const T* __restrict__ logits, int64_t ld, int64_t tokens, int vec, RouteArgs a,
                 int32_t* __restrict__ idx, float* __restrict__ weights) {
    __shared__ uint32_t group_keys[GROUPS == 2 ? kRouteWarps : 1][GROUPS == 2 ? 1024 : 1];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int E = a.experts, k = a.topk, e0 = lane * NI;
    const bool soft = a.score == 0;
    float bias[NI];
#pragma unroll
    for (int i = 0; i < NI; ++i) bias[i] = a.bias && e0 + i < E ? a.bias[e0 + i] : 0.0f;
    for (int64_t row = (int64_t)blockIdx.x * kRouteWarps + warp; row < tokens;
         row += (int64_t)gridDim.x * kRouteWarps) {
        const T* xr = logits + row * ld;
        float x[NI];
        load_row<NI>(xr, e0, E, vec, x);
        bool bad = false;
#pragma unroll
        for (int i = 0; i < NI; ++i) bad |= isnan(x[i]);
        bad = __any_sync(kFull, bad);
        float top = 0.0f, total = 1.0f;
        if (soft && (a.by_score || !a.renorm)) {
            top = x[0];
#pragma unroll
            for (int i = 1; i < NI; ++i) top = fmaxf(top, x[i]);
            top = warp_max(top);
            total = 0.0f;
#pragma unroll
            for (int i = 0; i < NI; ++i) total += x[i] > -INFINITY ? expf(x[i] - top) : 0.0f;
            total = warp_sum(total);
        }
        uint32_t key[NI];
#pragma unroll
        for (int i = 0; i < NI; ++i) {
            float v = x[i];
            if (!soft)
                v = sigmoid_f(v) + bias[i];
            else if (a.by_score)
                v = expf(v - top) / total + bias[i];
            key[i] = x[i] > -INFINITY && v > -INFINITY ? order_key(v) : 0u;
        }
        if constexpr (GROUPS == 1) groups_by_lanes<NI>(key, E / a.groups, a.group_best, a.topk_groups, lane);
        if constexpr (GROUPS == 2) groups_by_memory<NI>(key, group_keys[warp], E, a.groups, a.group_best, a.topk_groups, lane);
        // The choice: every lane sorts its keys, and the best of the lanes' heads is
        // taken k times.  Lane j keeps the j-th: its key and the lane it came from.
        uint32_t line[NI];
#pragma unroll
        for (int i = 0; i < NI; ++i) line[i] = key[i];
        sort_down<NI>(line);
        uint32_t my_key = 0u;
        int my_lane = 0;
        for (int j = 0; j < k; ++j) {
            const uint32_t most = __reduce_max_sync(kFull, line[0]);
            if (most == 0u) break;
            const int from = __ffs(__ballot_sync(kFull, line[0] == most)) - 1;
            if (lane == j) {
                my_key = most;
                my_lane = from;
            }
            if (lane == from) {
#pragma unroll
                for (int i = 0; i + 1 < NI; ++i) line[i] = line[i + 1];
                line[NI - 1] = 0u;
            }
        }
        // Which of that lane's experts it was: the first with the key, or the one after as
        // many as earlier choices took of the same key there.
        const unsigned alike = __match_any_sync(kFull, my_key) & __match_any_sync(kFull, my_lane) & ((1u << lane) - 1);
        int skip = __popc(alike), mine = -1;
#pragma unroll
        for (int i = 0; i < NI; ++i) {
            const uint32_t there = __shfl_sync(kFull, key[i], my_lane);
            if (there == my_key && mine < 0 && skip-- == 0) mine = my_lane * NI + i;
        }
        if (my_key == 0u) mine = -1;
        float w = choice_weight(xr, mine, a, top, total) * a.scale;
        if (bad && mine >= 0) w = NAN;
        if (lane < k) {
            idx[row * k + lane] = mine;
            weights[row * k + lane] = w;
        }
    }
}

// dlogits of one token a warp, from the logits, the choice and the weights'
// gradient: nothing of the forward pass is kept.
template <typename T, int NI>
__global__ void __launch_bounds__(kRouteWarps * 32)
    route_backward_kernel(const T* __restrict__ logits, int64_t ld, int64_t tokens, RouteArgs a,
                          const int32_t* __restrict__ idx, const float* __restrict__ dweights,
                          T* __restrict__ dlogits, int64_t dld) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int E = a.experts, k = a.topk;
    const bool soft = a.score == 0;
    for (int64_t row = (int64_t)blockIdx.x * kRouteWarps + warp; row < tokens;
         row += (int64_t)gridDim.x * kRouteWarps) {
        const T* xr = logits + row * ld;
        T* dr = dlogits + row * dld;
        int mine = lane < k ? idx[row * k + lane] : -1;
        if (mine < 0 || mine >= E) mine = -1;
        const float g = mine >= 0 ? a.scale * dweights[row * k + lane] : 0.0f;
        const float xm = mine >= 0 ? load_f(xr + mine) : -INFINITY;
        float d;
        if (soft && !a.renorm) {
            float x[NI];
            float top = -INFINITY, total = 0.0f;
#pragma unroll
            for (int i = 0; i < NI; ++i) {
                const int e = lane + 32 * i;
                x[i] = e < E ? load_f(xr + e) : -INFINITY;
                top = fmaxf(top, x[i]);
            }
            top = warp_max(top);
#pragma unroll
            for (int i = 0; i < NI; ++i) {
                x[i] = (x[i] == -INFINITY) ? 0.0f : expf(x[i] - top);
                total += x[i];
            }
            total = warp_sum(total);
            const float inv = total == 0.0f ? 0.0f : 1.0f / total;
            const float p = mine >= 0 ? expf(xm - top) * inv : 0.0f;
            const float dot = warp_sum(p * g);
#pragma unroll
            for (int i = 0; i < NI; ++i) {
                const int e = lane + 32 * i;
                if (e < E) store_f(dr + e, x[i] * inv * (0.0f - dot));
            }
            d = p * (g - dot);
        } else {
            if (soft) {
                const float m = warp_max(xm);
                const float p = mine >= 0 ? expf(xm - m) : 0.0f;
                const float s = warp_sum(p);
                const float q = mine >= 0 ? p / s : 0.0f;
                const float dot = warp_sum(q * g);
                d = q * (g - dot);
            } else {
                const float s = mine >= 0 ? sigmoid_f(xm) : 0.0f;
                if (a.renorm) {
                    const float S = warp_sum(s);
                    const float dot = S > 0.0f ? warp_sum(s * g) / S : 0.0f;
                    d = S > 0.0f ? (g - dot) / S * s * (1.0f - s) : 0.0f;
                } else {
                    d = g * s * (1.0f - s);
                }
            }
#pragma unroll
            for (int i = 0; i < NI; ++i)
                if (lane + 32 * i < E) store_f(dr + lane + 32 * i, 0.0f);
        }
        // the chosen experts' values over the row's: the warp's stores above come first
        __syncwarp();
        if (mine >= 0) store_f(dr + mine, d);
    }
}

// ---------------------------------------------------------------- host side

static int route_grid(int64_t tokens) {
    DeviceState* ds = device_state();
    if (!ds) return 0;
    const int64_t need = (tokens + kRouteWarps - 1) / kRouteWarps;
    const int64_t most = (int64_t)ds->sm_count * 8;
    return (int)(need < most ? need : most);
}

// GROUPS 1 needs lanes that are all used: groups of NI 2^j experts over 32 NI.
static int group_form(const RouteArgs& a, int NI) {
    if (a.groups == 1) return 0;
    const int gs = a.experts / a.groups, lanes = gs / NI;
    return a.experts == 32 * NI && gs % NI == 0 && (lanes & (lanes - 1)) == 0 ? 1 : 2;
}

template <typename T, int NI>
static void route_ni(int grid, cudaStream_t s, const T* x, int64_t ld, int64_t tokens, const RouteArgs& a, int32_t* idx,
                     float* w) {
    const int vec = a.experts == 32 * NI && ((uintptr_t)x & 15u) == 0 && (ld * (int64_t)sizeof(T)) % 16 == 0;
    const int form = group_form(a, NI);
    const dim3 b(kRouteWarps * 32);
    if (form == 0) route_kernel<T, NI, 0><<<grid, b, 0, s>>>(x, ld, tokens, vec, a, idx, w);
    else if (form == 1) route_kernel<T, NI, 1><<<grid, b, 0, s>>>(x, ld, tokens, vec, a, idx, w);
    else route_kernel<T, NI, 2><<<grid, b, 0, s>>>(x, ld, tokens, vec, a, idx, w);
}

template <typename T>
static void route_go(int grid, cudaStream_t s, const T* x, int64_t ld, int64_t tokens, const RouteArgs& a, int32_t* idx,
                     float* w) {
    const int ni = (a.experts + 31) / 32;
    if (ni <= 1) route_ni<T, 1>(grid, s, x, ld, tokens, a, idx, w);
    else if (ni <= 2) route_ni<T, 2>(grid, s, x, ld, tokens, a, idx, w);
    else if (ni <= 4) route_ni<T, 4>(grid, s, x, ld, tokens, a, idx, w);
    else if (ni <= 8) route_ni<T, 8>(grid, s, x, ld, tokens, a, idx, w);
    else if (ni <= 16) route_ni<T, 16>(grid, s, x, ld, tokens, a, idx, w);
    else route_ni<T, 32>(grid, s, x, ld, tokens, a, idx, w);
}

template <typename T>
static void route_back_go(int grid, cudaStream_t s, const T* x, int64_t ld, int64_t tokens, const RouteArgs& a,
                          const int32_t* idx, const float* dw, T* dx, int64_t dld) {
    const int ni = (a.experts + 31) / 32;
#define C3_GO(N_) route_backward_kernel<T, N_><<<grid, kRouteWarps * 32, 0, s>>>(x, ld, tokens, a, idx, dw, dx, dld)
    if (ni <= 1) C3_GO(1);
    else if (ni <= 2) C3_GO(2);
    else if (ni <= 4) C3_GO(4);
    else if (ni <= 8) C3_GO(8);
    else if (ni <= 16) C3_GO(16);
    else C3_GO(32);
#undef C3_GO
}

static int route_done(const char* what) {
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return set_cuda_error(e, what);
    count_launch();
    return 0;
}

int route_launch(const void* logits, int bf16, int64_t ld, int64_t tokens, const RouteArgs& a, int32_t* idx,
                 float* weights, cudaStream_t s) {
    const int grid = route_grid(tokens);
    if (grid == 0) return -3;
    if (bf16)
        route_go(grid, s, static_cast<const __nv_bfloat16*>(logits), ld, tokens, a, idx, weights);
    else
        route_go(grid, s, static_cast<const float*>(logits), ld, tokens, a, idx, weights);
    return route_done("route kernel launch");
}

int route_backward_launch(const void* logits, int bf16, int64_t ld, int64_t tokens, const RouteArgs& a,
                          const int32_t* idx, const float* dweights, void* dlogits, int64_t dld, cudaStream_t s) {
    const int grid = route_grid(tokens);
    if (grid == 0) return -3;
    if (bf16)
        route_back_go(grid, s, static_cast<const __nv_bfloat16*>(logits), ld, tokens, a, idx, dweights,
                      static_cast<__nv_bfloat16*>(dlogits), dld);
    else
        route_back_go(grid, s, static_cast<const float*>(logits), ld, tokens, a, idx, dweights,
                      static_cast<float*>(dlogits), dld);
    return route_done("route backward kernel launch");
}

}  // namespace c3
