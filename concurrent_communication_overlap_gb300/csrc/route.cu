// route.cu -- routing of tokens to experts: scores, the choice of the best,
// their weights, and the gradient of the weights with respect to the logits.
//
// One warp a token.  Lane l holds the logits of experts l, l + 32, ... in
// registers.  The choice compares 32-bit integers that order as the float keys
// do, so a maximum over the warp is one redux instruction and equal keys are
// settled by a second redux over the expert numbers (lowest wins).
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
    return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
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
__device__ __forceinline__ float sigmoid_f(float x) { return __fdiv_rn(1.0f, 1.0f + expf(-x)); }

// NI: experts a lane holds, ceil(E / 32) rounded up to a power of two.
template <typename T, int NI>
__global__ void __launch_bounds__(kRouteWarps * 32)
    route_kernel(const T* __restrict__ logits, int64_t ld, int64_t tokens, RouteArgs a, int32_t* __restrict__ idx,
                 float* __restrict__ weights) {
    __shared__ uint32_t group_keys[kRouteWarps][1024];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int E = a.experts, k = a.topk, G = a.groups, gs = E / G;
    const bool soft = a.score == 0;
    for (int64_t row = (int64_t)blockIdx.x * kRouteWarps + warp; row < tokens;
         row += (int64_t)gridDim.x * kRouteWarps) {
        const T* xr = logits + row * ld;
        float x[NI];
        uint32_t key[NI];
        float top = -INFINITY;
        bool bad = false;
#pragma unroll
        for (int i = 0; i < NI; ++i) {
            const int e = lane + 32 * i;
            x[i] = e < E ? load_f(xr + e) : -INFINITY;
            bad |= isnan(x[i]);
            top = fmaxf(top, x[i]);
        }
        bad = __any_sync(kFull, bad);
        float total = 1.0f;
        if (soft) {
            top = warp_max(top);
            total = 0.0f;
#pragma unroll
            for (int i = 0; i < NI; ++i) total += x[i] > -INFINITY ? expf(x[i] - top) : 0.0f;
            total = warp_sum(total);
        }
#pragma unroll
        for (int i = 0; i < NI; ++i) {
            const int e = lane + 32 * i;
            float v = x[i];
            if (v > -INFINITY) {
                if (!soft)
                    v = sigmoid_f(v);
                else if (a.by_score)
                    v = expf(v - top) / total;
                if (a.bias) v += __ldg(a.bias + e);
            }
            key[i] = v > -INFINITY ? order_key(v) : 0u;
        }
        if (G > 1) {
            // The groups' scores: lane g + 32 j takes group g + 32 j, reading its
            // members from shared memory, each lane from a place of its own on.
            uint32_t* gk = group_keys[warp];
#pragma unroll
            for (int i = 0; i < NI; ++i)
                if (lane + 32 * i < E) gk[lane + 32 * i] = key[i];
            __syncwarp();
            uint32_t gscore[NI];
#pragma unroll
            for (int i = 0; i < NI; ++i) {
                const int g = lane + 32 * i;
                gscore[i] = 0u;
                if (g < G) {
                    uint32_t b1 = 0u, b2 = 0u;
                    for (int j = 0, at = g % gs; j < gs; ++j, at = at + 1 == gs ? 0 : at + 1) {
                        const uint32_t v = gk[g * gs + at];
                        if (v > b1) {
                            b2 = b1;
                            b1 = v;
                        } else if (v > b2) {
                            b2 = v;
                        }
                    }
                    gscore[i] = (a.group_best == 2 && b2) ? order_key(order_value(b1) + order_value(b2)) : b1;
                }
            }
            __syncwarp();
            // Keep the best topk_groups groups: mark them in shared memory.
#pragma unroll
            for (int i = 0; i < NI; ++i)
                if (lane + 32 * i < G) gk[lane + 32 * i] = 0u;
            __syncwarp();
            for (int j = 0; j < a.topk_groups; ++j) {
                uint32_t best = 0u;
#pragma unroll
                for (int i = 0; i < NI; ++i) best = max(best, gscore[i]);
                best = __reduce_max_sync(kFull, best);
                if (best == 0u) break;
                unsigned at = 0xffffu;
#pragma unroll
                for (int i = NI - 1; i >= 0; --i)
                    if (gscore[i] == best) at = lane + 32 * i;
                at = __reduce_min_sync(kFull, at);
#pragma unroll
                for (int i = 0; i < NI; ++i)
                    if ((unsigned)(lane + 32 * i) == at) {
                        gscore[i] = 0u;
                        gk[at] = 1u;
                    }
            }
            __syncwarp();
#pragma unroll
            for (int i = 0; i < NI; ++i) {
                const int e = lane + 32 * i;
                if (e < E && gk[e / gs] == 0u) key[i] = 0u;
            }
            __syncwarp();
        }
        // The choice; lane j keeps the j-th.
        int mine = -1;
        for (int j = 0; j < k; ++j) {
            uint32_t best = 0u;
#pragma unroll
            for (int i = 0; i < NI; ++i) best = max(best, key[i]);
            best = __reduce_max_sync(kFull, best);
            if (best == 0u) break;
            unsigned at = 0xffffu;
#pragma unroll
            for (int i = NI - 1; i >= 0; --i)
                if (key[i] == best) at = lane + 32 * i;
            at = __reduce_min_sync(kFull, at);
#pragma unroll
            for (int i = 0; i < NI; ++i)
                if ((unsigned)(lane + 32 * i) == at) key[i] = 0u;
            if (lane == j) mine = (int)at;
        }
        // The weights.
        float w = 0.0f;
        const float xm = mine >= 0 ? load_f(xr + mine) : -INFINITY;
        if (soft && a.renorm) {
            const float m = warp_max(xm);
            const float p = mine >= 0 ? expf(xm - m) : 0.0f;
            const float s = warp_sum(p);
            w = mine >= 0 ? p / s : 0.0f;
        } else if (soft) {
            w = mine >= 0 ? expf(xm - top) / total : 0.0f;
        } else {
            w = mine >= 0 ? sigmoid_f(xm) : 0.0f;
            if (a.renorm) {
                const float s = warp_sum(w);
                w = s > 0.0f ? w / s : 0.0f;
            }
        }
        w *= a.scale;
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

template <typename T>
static void route_go(int grid, cudaStream_t s, const T* x, int64_t ld, int64_t tokens, const RouteArgs& a, int32_t* idx,
                     float* w) {
    const int ni = (a.experts + 31) / 32;
#define C3_GO(N_) route_kernel<T, N_><<<grid, kRouteWarps * 32, 0, s>>>(x, ld, tokens, a, idx, w)
    if (ni <= 1) C3_GO(1);
    else if (ni <= 2) C3_GO(2);
    else if (ni <= 4) C3_GO(4);
    else if (ni <= 8) C3_GO(8);
    else if (ni <= 16) C3_GO(16);
    else C3_GO(32);
#undef C3_GO
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
