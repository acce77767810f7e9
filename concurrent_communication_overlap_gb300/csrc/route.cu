// route.cu -- routing of tokens to experts: scores, the choice of the best,
// their weights, and the gradient of the weights with respect to the logits.
//
// L lanes a token (8, 16 or 32, so a warp takes 4, 2 or 1).  Lane l of them
// holds the logits of NI consecutive experts, l NI and up (in groups, those of a run
// of lanes being a group), in registers.  The choice compares 32-bit integers that
// order as the float keys do; of equal keys the lowest lane, and in it the lowest
// register, is the lowest expert.  Without a bias the keys are the logits: the scores
// order as they do, but fp32 scores of different logits can be equal (every sigmoid
// above 17 is 1).
//
// Few lanes a token, because the exchange between lanes, which is the same for
// one token as for four, is most of the work: 32768 x 60, 6 chosen, took 354
// instructions a token with 32 lanes and 192 with 8 (16384 x 60: 6.7 us and 4.9).
//
// Not bytes bound it.  65536 x 256, sigmoids, bias and groups, takes 55 us, its bytes
// need 10.5: 742 instructions a token fill 71% of the issue slots (without a bias or
// groups 432, 64%, 37 us); for the rest a CTA's 8 warps, 4 CTAs an SM, wait for one
// another's shuffles and shared memory, for fixed latencies and for the ALU, 61% busy.
// 32768 x 60, softmax: 7.6 us for 182 instructions a token, 65%; its gradient 5.0, most
// of it waiting for loads (an index, the logit that it names, then the row): 50%.
#include "ops_device.cuh"
#include "c3_internal.h"

#include <cuda_bf16.h>

namespace c3 {

constexpr int kRouteWarps = 8;  // of a CTA, each with 32 / L tokens a pass
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
// Over the L lanes of a token.
template <int L>
__device__ __forceinline__ float lanes_max(float v) {
#pragma unroll
    for (int o = L / 2; o; o >>= 1) v = fmaxf(v, __shfl_xor_sync(kFull, v, o));
    return v;
}
template <int L>
__device__ __forceinline__ uint32_t lanes_max(uint32_t v) {
    if constexpr (L == 32) {
        return __reduce_max_sync(kFull, v);
    } else {
#pragma unroll
        for (int o = L / 2; o; o >>= 1) v = max(v, __shfl_xor_sync(kFull, v, o));
        return v;
    }
}
template <int L>
__device__ __forceinline__ float lanes_sum(float v) {
#pragma unroll
    for (int o = L / 2; o; o >>= 1) v += __shfl_xor_sync(kFull, v, o);
    return v;
}
// The vote of a token's lanes, its lane 0 in bit 0.
template <int L>
__device__ __forceinline__ unsigned lanes_ballot(bool v, int lane) {
    const unsigned b = __ballot_sync(kFull, v);
    return L == 32 ? b : (b >> (lane & ~(L - 1))) & ((1u << (L & 31)) - 1);
}
__device__ __forceinline__ float sigmoid_f(float x) { return __frcp_rn(1.0f + expf(-x)); }

// Values of a vector load of N consecutive ones.
template <typename T, int N>
__host__ __device__ constexpr int vector_of() {
    return N % 4 ? 1 : sizeof(T) == 2 && N % 8 == 0 ? 8 : 4;
}

// N consecutive logits of a row from expert e0 on; -inf from expert `end` on.  vec:
// rows start on 16 bytes and lanes end at whole vectors.
template <int N, typename T>
__device__ __forceinline__ void load_row(const T* xr, int e0, int end, bool vec, float (&x)[N]) {
    constexpr int V = vector_of<T, N>();
    if (V == 1 || !vec) {
#pragma unroll
        for (int i = 0; i < N; ++i) x[i] = e0 + i < end ? load_f(xr + e0 + i) : -INFINITY;
        return;
    }
    const auto vector = [&](int i) {
        if constexpr (sizeof(T) == 4) {
            const float4 v = *reinterpret_cast<const float4*>(xr + e0 + i);
            x[i] = v.x, x[i + 1] = v.y, x[i + 2] = v.z, x[i + 3] = v.w;
        } else {
            uint32_t u[V / 2 + 1];
            if constexpr (V == 8) {
                const uint4 v = *reinterpret_cast<const uint4*>(xr + e0 + i);
                u[0] = v.x, u[1] = v.y, u[2] = v.z, u[3] = v.w;
            } else {
                const uint2 v = *reinterpret_cast<const uint2*>(xr + e0 + i);
                u[0] = v.x, u[1] = v.y;
            }
#pragma unroll
            for (int j = 0; j < V / 2; ++j) {
                x[i + 2 * j] = __uint_as_float(u[j] << 16);
                x[i + 2 * j + 1] = __uint_as_float(u[j] & 0xffff0000u);
            }
        }
    };
    if constexpr (V > 1) {
        if (e0 + N <= end) {
#pragma unroll
            for (int i = 0; i < N; i += V) vector(i);
        } else {
#pragma unroll
            for (int i = 0; i < N; ++i) x[i] = -INFINITY;
#pragma unroll
            for (int i = 0; i < N; i += V)
                if (e0 + i < end) vector(i);
        }
    }
}

// The same by way of shared memory, for rows that no vector load fits: neighbouring
// lanes read neighbouring values.  `stage` is the warp's, 32 N words; a line of it
// (8 chunks of 16 bytes) has its chunks in an order of its own, so that lanes that
// read N words each meet in no bank (12 words do not meet as they are).  16000 tokens of 371 experts,
// 16 a lane: 30.6 us, with loads N apart 34.4.
template <int N, int L, typename T>
__device__ __forceinline__ void load_staged(const T* xr, int E, float none, uint32_t* stage, int lane, float (&x)[N]) {
    const int at_lane = lane & (L - 1), base = (lane / L) * L * N;
    const auto place = [](int w) { return N & (N - 1) ? w : w ^ ((w >> 3) & 28); };
    __syncwarp();
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const int e = at_lane + L * i;
        stage[place(base + e)] = __float_as_uint(e < E ? load_f(xr + e) : none);
    }
    __syncwarp();
#pragma unroll
    for (int i = 0; i < N; i += 4) {
        const float4 v = *reinterpret_cast<const float4*>(stage + place(base + at_lane * N + i));
        x[i] = v.x, x[i + 1] = v.y, x[i + 2] = v.z, x[i + 3] = v.w;
    }
    __syncwarp();
}

// The same for lanes whose first experts e0 are not N apart: value by value, each 32
// skewed by one word, which keeps lanes 12 or 16 experts apart in banks of their own.
template <int N, int L, typename T>
__device__ __forceinline__ void load_staged(const T* xr, int E, int e0, int end, float none, uint32_t* stage, int lane,
                                            float (&x)[N]) {
    const int at_lane = lane & (L - 1), base = (lane / L) * (L * N / 32 * 33);
    __syncwarp();
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const int e = at_lane + L * i;
        if (e < E) stage[base + e + (e >> 5)] = __float_as_uint(load_f(xr + e));
    }
    __syncwarp();
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const int e = e0 + i;
        x[i] = e < end ? __uint_as_float(stage[base + e + (e >> 5)]) : none;
    }
    __syncwarp();
}

// Groups that are whole runs of `lanes`, a power of two, of the token's lanes: score and
// rank them with shuffles, by their best key or the sum of the scores of the best two.
// Sets the keys of groups outside the best `keep` to 0.
template <int NI, int L, typename Score>
__device__ __forceinline__ void groups_by_lanes(uint32_t (&key)[NI], int lanes, int best_of, int keep, int lane,
                                                const Score& score_of) {
    uint32_t b1 = 0u, b2 = 0u;
#pragma unroll
    for (int i = 0; i < NI; ++i) {
        b2 = max(b2, min(b1, key[i]));
        b1 = max(b1, key[i]);
    }
    for (int o = 1; o < lanes; o <<= 1) {
        const uint32_t c1 = __shfl_xor_sync(kFull, b1, o), c2 = __shfl_xor_sync(kFull, b2, o);
        b2 = max(max(b2, c2), min(b1, c1));
        b1 = max(b1, c1);
    }
    uint32_t score = b1;
    if (best_of == 2 && b1) score = order_key(score_of(b1) + (b2 ? score_of(b2) : 0.0f));
    const int mine = (lane & (L - 1)) / lanes, groups = L / lanes;
    int rank = 0;
    for (int g = 0; g < groups; ++g) {
        const uint32_t other = __shfl_sync(kFull, score, g * lanes, L);
        rank += other > score || (other == score && g < mine);
    }
    if (rank >= keep) {
#pragma unroll
        for (int i = 0; i < NI; ++i) key[i] = 0u;
    }
}

// Groups of any size, by way of shared memory (1024 words a warp: the keys, or where keys
// are logits and two scores are summed (sum_scores) the scores): lane g + 32 j takes group
// g + 32 j, each lane reading from a place of its own on.
template <int NI, typename Score>
__device__ __forceinline__ void groups_by_memory(uint32_t (&key)[NI], uint32_t* gk, int E, int G, int best_of, int keep,
                                                 int lane, bool sum_scores, const Score& score_of) {
    const int gs = E / G;
#pragma unroll
    for (int i = 0; i < NI; ++i)
        if (lane * NI + i < E) gk[lane * NI + i] = key[i];
    if (sum_scores) {
#pragma unroll
        for (int i = 0; i < NI; ++i)
            if (lane * NI + i < E && key[i]) gk[lane * NI + i] = order_key(score_of(key[i]));
    }
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

// Descending order of N keys, by a bitonic network of a power of two: what it has
// above N is 0, which the compiler sees through.
template <int N>
__device__ __forceinline__ void sort_down(uint32_t (&keys)[N]) {
    constexpr int P = N <= 1 ? 1 : N <= 2 ? 2 : N <= 4 ? 4 : N <= 8 ? 8 : N <= 16 ? 16 : 32;
    uint32_t k[P];
#pragma unroll
    for (int i = 0; i < P; ++i) k[i] = i < N ? keys[i < N ? i : 0] : 0u;
#pragma unroll
    for (int size = 2; size <= P; size <<= 1)
#pragma unroll
        for (int d = size >> 1; d; d >>= 1)
#pragma unroll
            for (int i = 0; i < P; ++i)
                if ((i & d) == 0) {
                    const uint32_t a = k[i], b = k[i | d];
                    const bool down = (i & size) == 0 || size == P;
                    k[i] = down ? max(a, b) : min(a, b);
                    k[i | d] = down ? min(a, b) : max(a, b);
                }
#pragma unroll
    for (int i = 0; i < N; ++i) keys[i] = k[i];
}

// The weight of this lane's choice (expert `mine`, or -1), unscaled.
template <typename T, int L>
__device__ __forceinline__ float choice_weight(const T* xr, int mine, const RouteArgs& a, float top, float total) {
    const float x = mine >= 0 ? load_f(xr + mine) : -INFINITY;
    if (a.score == 0 && a.renorm) {
        const float m = lanes_max<L>(x);
        const float p = mine >= 0 ? expf(x - m) : 0.0f;
        const float s = lanes_sum<L>(p);
        return mine >= 0 ? p / s : 0.0f;
    }
    if (a.score == 0) return mine >= 0 ? expf(x - top) / total : 0.0f;
    const float w = mine >= 0 ? sigmoid_f(x) : 0.0f;
    if (!a.renorm) return w;
    const float s = lanes_sum<L>(w);
    return s > 0.0f ? w / s : 0.0f;
}

// NI experts a lane, L NI >= E.  GROUPS: 0 none, 1 a run of L / groups lanes each (groups
// a power of two), 2 any (L = 32).  vec: as load_row's.  topk <= L.
// Registers: 65536 x 256 takes 55 us with 64 and 60 with 80; 16000 x 1000 takes 72 with
// 128, 77 with 80 and 119 with 218.  Groups by way of memory spill 56 bytes with NI = 16
// and 16 with NI = 32, the others none.
template <typename T, int NI, int L, int GROUPS>
__global__ void __launch_bounds__(kRouteWarps * 32, NI == 12 || NI == 16 ? 4 : NI == 32 ? 2 : 1)
    route_kernel(const T* __restrict__ logits, int64_t ld, int64_t tokens, int vec, RouteArgs a,
                 int32_t* __restrict__ idx, float* __restrict__ weights) {
    constexpr int kRows = 32 / L;  // tokens of a warp
    constexpr bool kInMemory = NI >= 8;
    // 8 lanes of 8 share the lines that they load: staged, 32768 x 60 took 2 us more
    constexpr bool kStaged = NI >= 12 || (NI == 8 && L == 32);
    // a warp's scratch: the groups' keys first, then the sorted lines
    constexpr int kScratch = GROUPS == 2 ? 1024 : kInMemory ? NI * (GROUPS == 1 ? 33 : 32) : 1;
    __shared__ __align__(16) uint32_t scratch[kRouteWarps][kScratch];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int at_lane = lane & (L - 1);
    const int E = a.experts, k = a.topk;
    // This lane's experts, [e0, end): a run of L / groups lanes has a group's, else each lane the next NI.
    const int run = GROUPS == 1 ? L / a.groups : 1, shift = GROUPS == 1 ? __ffs(run) - 1 : 0;
    const int size = GROUPS == 1 ? E / a.groups : 0;
    const auto first_of = [&](int l) { return GROUPS == 1 ? (l >> shift) * size + (l & (run - 1)) * NI : l * NI; };
    const int e0 = first_of(at_lane), end = GROUPS == 1 ? (at_lane >> shift) * size + size : E;
    const bool soft = a.score == 0;
    chain_wait();
    float bias[NI] = {};
    if constexpr (kStaged) {
        if (a.bias) {
            if constexpr (GROUPS == 1)
                load_staged<NI, L>(a.bias, E, e0, end, 0.0f, scratch[warp], lane, bias);
            else
                load_staged<NI, L>(a.bias, E, 0.0f, scratch[warp], lane, bias);
        }
    } else if (a.bias) {
#pragma unroll
        for (int i = 0; i < NI; ++i) bias[i] = e0 + i < end ? a.bias[e0 + i] : 0.0f;
    }
    const int64_t step = (int64_t)gridDim.x * kRouteWarps * kRows;
    for (int64_t row0 = ((int64_t)blockIdx.x * kRouteWarps + warp) * kRows; row0 < tokens; row0 += step) {
        const int64_t row = row0 + lane / L;
        const bool live = row < tokens;
        const T* xr = logits + (live ? row : row0) * ld;  // a lane without a token repeats another's
        float x[NI];
        if (kStaged && !vec) {
            if constexpr (kStaged && GROUPS == 1)
                load_staged<NI, L>(xr, E, e0, end, -INFINITY, scratch[warp], lane, x);
            else if constexpr (kStaged)
                load_staged<NI, L>(xr, E, -INFINITY, scratch[warp], lane, x);
        } else {
            load_row<NI>(xr, e0, end, vec, x);
        }
        // weights are NaN where a logit is NaN, or +inf with the softmax
        bool bad = false;
#pragma unroll
        for (int i = 0; i < NI; ++i) bad |= soft ? !(x[i] < INFINITY) : isnan(x[i]);
        bad = lanes_ballot<L>(bad, lane) != 0u;
        float top = 0.0f, total = 1.0f;
        if (soft && (a.by_score || a.pairs || !a.renorm)) {
            top = x[0];
#pragma unroll
            for (int i = 1; i < NI; ++i) top = fmaxf(top, x[i]);
            top = lanes_max<L>(top);
            total = 0.0f;
#pragma unroll
            for (int i = 0; i < NI; ++i) total += x[i] > -INFINITY ? expf(x[i] - top) : 0.0f;
            total = lanes_sum<L>(total);
        }
        uint32_t key[NI];
        const auto set_key = [&](int i, float v) { key[i] = x[i] > -INFINITY && v > -INFINITY ? order_key(v) : 0u; };
        const bool no_score = soft && !(top < INFINITY);  // +inf in the row: the scores are NaN
        if (!a.by_score || no_score) {
#pragma unroll
            for (int i = 0; i < NI; ++i) set_key(i, x[i] + bias[i]);
        } else if (soft) {
#pragma unroll
            for (int i = 0; i < NI; ++i) set_key(i, expf(x[i] - top) / total + bias[i]);
        } else {
#pragma unroll
            for (int i = 0; i < NI; ++i) set_key(i, sigmoid_f(x[i]) + bias[i]);
        }
        const auto score_of = [&](uint32_t key) {
            const float v = order_value(key);
            if (a.by_score || no_score) return v;
            return soft ? expf(v - top) / total : sigmoid_f(v);
        };
        if constexpr (GROUPS == 1) groups_by_lanes<NI, L>(key, run, a.group_best, a.topk_groups, lane, score_of);
        if constexpr (GROUPS == 2)
            groups_by_memory<NI>(key, scratch[warp], E, a.groups, a.group_best, a.topk_groups, lane,
                                 a.pairs && !a.by_score, score_of);
        // The choice: every lane sorts its keys, and the best of the lanes' heads is
        // taken k times.  Lane j keeps the j-th: its key and the lane it came from.
        uint32_t line[NI];
#pragma unroll
        for (int i = 0; i < NI; ++i) line[i] = key[i];
        sort_down<NI>(line);
        // A line of eight or more waits in shared memory, which costs a load a choice instead
        // of shifting it through registers.
        uint32_t my_key = 0u;
        int my_lane = 0;
        uint32_t head = line[0];
        const uint32_t* behind = nullptr;
        if constexpr (kInMemory) {
#pragma unroll
            for (int i = 1; i < NI; ++i) scratch[warp][(i - 1) * 32 + lane] = line[i];
            scratch[warp][(NI - 1) * 32 + lane] = 0u;
            behind = &scratch[warp][lane];
        }
        for (int j = 0; j < k; ++j) {
            const uint32_t most = lanes_max<L>(head);
            const int from = __ffs(lanes_ballot<L>(head == most, lane)) - 1;
            if (at_lane == j) {
                my_key = most;
                my_lane = from;
            }
            const bool take = at_lane == from && most != 0u;
            if constexpr (kInMemory) {
                if (take) {
                    head = *behind;
                    behind += 32;
                }
            } else {
#pragma unroll
                for (int i = 0; i + 1 < NI; ++i) line[i] = take ? line[i + 1] : line[i];
                line[NI - 1] = take ? 0u : line[NI - 1];
                head = line[0];
            }
        }
        if constexpr (GROUPS == 2) __syncwarp();  // the scratch is another's again
        // Which of that lane's experts it was: the first with the key, or the one after as
        // many as earlier choices took of the same key there.  Those are the choices just
        // before: equal keys go by lane, then by register.
        const uint32_t key_up = __shfl_up_sync(kFull, my_key, 1, L);
        const int lane_up = __shfl_up_sync(kFull, my_lane, 1, L);
        const unsigned starts = lanes_ballot<L>(at_lane == 0 || key_up != my_key || lane_up != my_lane, lane);
        const int from0 = first_of(my_lane);
        int skip = __clz(starts << (31 - at_lane)), mine = -1;
#pragma unroll
        for (int i = 0; i < NI; ++i) {
            const uint32_t there = __shfl_sync(kFull, key[i], my_lane, L);
            if (there == my_key && mine < 0 && skip-- == 0) mine = from0 + i;
        }
        if (my_key == 0u) mine = -1;
        float w = choice_weight<T, L>(xr, mine, a, top, total) * a.scale;
        if (bad && mine >= 0) w = NAN;
        if (live && at_lane < k) {
            idx[row * k + at_lane] = mine;
            weights[row * k + at_lane] = w;
        }
    }
}

// dlogits of L lanes' token, from the logits, the choice and the weights'
// gradient: nothing of the forward pass is kept.
template <typename T, int NI, int L>
__global__ void __launch_bounds__(kRouteWarps * 32)
    route_backward_kernel(const T* __restrict__ logits, int64_t ld, int64_t tokens, RouteArgs a,
                          const int32_t* __restrict__ idx, const float* __restrict__ dweights,
                          T* __restrict__ dlogits, int64_t dld) {
    constexpr int kRows = 32 / L;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int at_lane = lane & (L - 1);
    const int E = a.experts, k = a.topk;
    const bool soft = a.score == 0;
    chain_wait();
    const int64_t step = (int64_t)gridDim.x * kRouteWarps * kRows;
    for (int64_t row0 = ((int64_t)blockIdx.x * kRouteWarps + warp) * kRows; row0 < tokens; row0 += step) {
        const int64_t row = row0 + lane / L;
        const bool live = row < tokens;
        const T* xr = logits + (live ? row : row0) * ld;
        T* dr = dlogits + (live ? row : row0) * dld;
        int mine = live && at_lane < k ? idx[row * k + at_lane] : -1;
        if (mine < 0 || mine >= E) mine = -1;
        const float g = mine >= 0 ? a.scale * dweights[row * k + at_lane] : 0.0f;
        const float xm = mine >= 0 ? load_f(xr + mine) : -INFINITY;
        float d;
        if (soft && !a.renorm) {
            // lane l holds experts l, l + L, ...: neighbours load and store neighbours
            float x[NI];
            float top = -INFINITY, total = 0.0f;
#pragma unroll
            for (int i = 0; i < NI; ++i) {
                const int e = at_lane + L * i;
                x[i] = e < E ? load_f(xr + e) : -INFINITY;
                top = fmaxf(top, x[i]);
            }
            top = lanes_max<L>(top);
#pragma unroll
            for (int i = 0; i < NI; ++i) {
                x[i] = (x[i] == -INFINITY) ? 0.0f : expf(x[i] - top);
                total += x[i];
            }
            total = lanes_sum<L>(total);
            const float inv = total == 0.0f ? 0.0f : 1.0f / total;
            const float p = mine >= 0 ? expf(xm - top) * inv : 0.0f;
            const float dot = lanes_sum<L>(p * g);
#pragma unroll
            for (int i = 0; i < NI; ++i) {
                const int e = at_lane + L * i;
                if (live && e < E) store_f(dr + e, x[i] * inv * (0.0f - dot));
            }
            d = p * (g - dot);
        } else {
            if (soft) {
                const float m = lanes_max<L>(xm);
                const float p = mine >= 0 ? expf(xm - m) : 0.0f;
                const float s = lanes_sum<L>(p);
                const float q = mine >= 0 ? p / s : 0.0f;
                const float dot = lanes_sum<L>(q * g);
                d = q * (g - dot);
            } else {
                // 1 - s cancels where s is near 1: there it is exp(-x) s.  And s / S comes first:
                // (g - sg / S) / S may overflow.
                const float e = expf(-xm), s = mine >= 0 ? __frcp_rn(1.0f + e) : 0.0f;
                const float c = e < 1.0f ? e * s : 1.0f - s;
                if (a.renorm) {
                    const float S = lanes_sum<L>(s);
                    const float sg = lanes_sum<L>(s * g);
                    d = S > 0.0f ? s / S * (g - sg / S) * c : 0.0f;
                } else {
                    d = g * s * c;
                }
            }
#pragma unroll
            for (int i = 0; i < NI; ++i)
                if (live && at_lane + L * i < E) store_f(dr + at_lane + L * i, 0.0f);
        }
        // the chosen experts' values over the row's: the warp's stores above come first
        __syncwarp();
        if (mine >= 0) store_f(dr + mine, d);
    }
}

// ---------------------------------------------------------------- host side

static int route_grid(int64_t tokens, int lanes) {
    DeviceState* ds = device_state();
    if (!ds) return 0;
    const int64_t per = kRouteWarps * (32 / lanes);
    const int64_t need = (tokens + per - 1) / per;
    const int64_t most = (int64_t)ds->sm_count * 8;
    return (int)(need < most ? need : most);
}

static int route_done(cudaError_t e, const char* what) {
    if (e != cudaSuccess) return set_cuda_error(e, what);
    count_launch();
    return 0;
}

constexpr int64_t kFewTokens = 4096;

// Lanes a token and experts a lane.  8 lanes hold 128 experts in 16 registers, 16
// lanes 256; more registers a lane would cost more in sorting and shifting them
// than the exchange saves.  Few tokens do not fill the machine: a whole warp is
// then the shortest way (softmax, fp32, us with a whole warp and with fewer lanes: 2048 x 256
// 3.6 and 6.6, 4096 x 256 5.3 and 7.5, 8192 x 256 7.9 and 8.0, 16384 x 256 12.9 and 11.8;
// 8192 x 128 5.1 and 7.1, 16384 x 128 8.3 and 7.8; 8192 x 60 4.4 and 4.5, 16384 x 60 6.7 and
// 4.9: kFewTokens could be two to three times what it is).  Groups that are a power of two
// in number have a run of lanes each, whatever their size (16000 x 160 in 8 groups: 14 us; by
// way of memory, as other numbers of groups, which take a whole warp, 41).
struct RouteForm {
    int lanes, per_lane, groups;
};

// Powers of two, and 12: 16 would sort and score a quarter more (16000 x 371 with a bias: 23.4 us against 30.6).
static int registers_for(int n) {
    if (n > 8 && n <= 12) return 12;
    int p = 1;
    while (p < n) p *= 2;
    return p;
}

static RouteForm route_form(const RouteArgs& a, int64_t tokens) {
    RouteForm f;
    for (int lanes = tokens < kFewTokens ? 32 : 8; lanes <= 32; lanes *= 2) {
        f.lanes = lanes;
        const int run = (a.groups & (a.groups - 1)) == 0 ? lanes / a.groups : 0;  // lanes a group
        f.groups = a.groups == 1 ? 0 : run ? 1 : 2;
        const int share = f.groups == 1 ? run : lanes, held = f.groups == 1 ? a.experts / a.groups : a.experts;
        f.per_lane = registers_for((held + share - 1) / share);
        if (a.topk <= lanes && f.per_lane <= 16 && f.groups != 2) return f;
    }
    return f;  // 32 lanes
}

template <typename T, int NI, int L>
static int route_go(const RouteForm& f, cudaStream_t s, const T* x, int64_t ld, int64_t tokens, const RouteArgs& a,
                    int32_t* idx, float* w) {
    const int grid = route_grid(tokens, L);
    if (grid == 0) return -3;
    const int whole = f.groups == 1 ? a.experts / a.groups : a.experts;
    const int vec = whole % vector_of<T, NI>() == 0 && ((uintptr_t)x & 15u) == 0 && (ld * (int64_t)sizeof(T)) % 16 == 0;
    const auto go = [&](auto kernel) {
        return route_done(launch_chained(kernel, dim3(grid), kRouteWarps * 32, 0, s, 1, x, ld, tokens, vec, a, idx, w),
                          "route kernel launch");
    };
    if constexpr (L == 32)
        if (f.groups == 2) return go(route_kernel<T, NI, L, 2>);
    return f.groups == 0 ? go(route_kernel<T, NI, L, 0>) : go(route_kernel<T, NI, L, 1>);
}

template <typename T, int NI, int L>
static int route_back_go(cudaStream_t s, const T* x, int64_t ld, int64_t tokens, const RouteArgs& a, const int32_t* idx,
                         const float* dw, T* dx, int64_t dld) {
    const int grid = route_grid(tokens, L);
    if (grid == 0) return -3;
    return route_done(launch_chained(route_backward_kernel<T, NI, L>, dim3(grid), kRouteWarps * 32, 0, s, 1, x, ld, tokens, a,
                                     idx, dw, dx, dld),
                      "route backward kernel launch");
}

// f.lanes and f.per_lane as template arguments NI_ and L_ of CALL.
#define C3_ROUTE_FORMS(CALL)                                             \
    do {                                                                 \
        if (f.lanes == 8) switch (f.per_lane) {                          \
            case 1: return CALL(1, 8);                                   \
            case 2: return CALL(2, 8);                                   \
            case 4: return CALL(4, 8);                                   \
            case 8: return CALL(8, 8);                                   \
            case 12: return CALL(12, 8);                                 \
            default: return CALL(16, 8);                                 \
        }                                                                \
        if (f.lanes == 16) switch (f.per_lane) {                         \
            case 1: return CALL(1, 16);                                  \
            case 2: return CALL(2, 16);                                  \
            case 4: return CALL(4, 16);                                  \
            case 8: return CALL(8, 16);                                  \
            case 12: return CALL(12, 16);                                \
            default: return CALL(16, 16);                                \
        }                                                                \
        switch (f.per_lane) {                                            \
            case 1: return CALL(1, 32);                                  \
            case 2: return CALL(2, 32);                                  \
            case 4: return CALL(4, 32);                                  \
            case 8: return CALL(8, 32);                                  \
            case 12: return CALL(12, 32);                                \
            case 16: return CALL(16, 32);                                \
            default: return CALL(32, 32);                                \
        }                                                                \
    } while (0)

template <typename T>
static int route_any(const RouteForm& f, cudaStream_t s, const T* x, int64_t ld, int64_t tokens, const RouteArgs& a,
                     int32_t* idx, float* w) {
#define C3_CALL(NI_, L_) route_go<T, NI_, L_>(f, s, x, ld, tokens, a, idx, w)
    C3_ROUTE_FORMS(C3_CALL);
#undef C3_CALL
}

template <typename T>
static int route_back_any(const RouteForm& f, cudaStream_t s, const T* x, int64_t ld, int64_t tokens, const RouteArgs& a,
                          const int32_t* idx, const float* dw, T* dx, int64_t dld) {
#define C3_CALL(NI_, L_) route_back_go<T, NI_, L_>(s, x, ld, tokens, a, idx, dw, dx, dld)
    C3_ROUTE_FORMS(C3_CALL);
#undef C3_CALL
}

int route_launch(const void* logits, int bf16, int64_t ld, int64_t tokens, const RouteArgs& a, int32_t* idx,
                 float* weights, cudaStream_t s) {
    const RouteForm f = route_form(a, tokens);
    return bf16 ? route_any(f, s, static_cast<const __nv_bfloat16*>(logits), ld, tokens, a, idx, weights)
                : route_any(f, s, static_cast<const float*>(logits), ld, tokens, a, idx, weights);
}

int route_backward_launch(const void* logits, int bf16, int64_t ld, int64_t tokens, const RouteArgs& a,
                          const int32_t* idx, const float* dweights, void* dlogits, int64_t dld, cudaStream_t s) {
    RouteArgs plain = a;
    plain.groups = 1;  // the gradient does not see groups
    const RouteForm f = route_form(plain, tokens);
    return bf16 ? route_back_any(f, s, static_cast<const __nv_bfloat16*>(logits), ld, tokens, a, idx, dweights,
                                 static_cast<__nv_bfloat16*>(dlogits), dld)
                : route_back_any(f, s, static_cast<const float*>(logits), ld, tokens, a, idx, dweights,
                                 static_cast<float*>(dlogits), dld);
}

}  // namespace c3
