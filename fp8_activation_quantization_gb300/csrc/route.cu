// route.cu -- routing of tokens to experts and its gradient.
//
// Forward, for each token: scores of its E logits x (softmax over the experts
// or the sigmoid of each), keys = scores + bias, optionally the best
// topk_groups of `groups` groups of E / groups consecutive experts, and of what
// is left the k largest keys in falling order, ties to the lowest index.  The
// weights are scale * score, renormalised or not: the bias moves the choice
// and no weight.
//   score_e = 1 / (1 + exp(-x_e))           or  exp(x_e - m) / sum_j exp(x_j - m)
//   w_i     = scale * score_(e_i) [/ sum_j score_(e_j)]
// Backward, with a_i = scale * dw_i, p_i the chosen scores and S their sum:
//   ds_i = a_i,  or renormalised  (a_i - sum_j a_j (p_j / S)) / S
//   dx_e = ds_e s_e (1 - s_e)               or  s_e (ds_e - sum_j ds_j s_j)
//
// An expert is absent from a token's row when its logit is -inf or NaN: it has
// no share in the softmax, is never chosen and gets no gradient.  When fewer
// than k experts are left the remaining ids are -1 with weight 0, so a row
// without any expert is all -1.  A logit of +inf counts as the largest finite
// number, which keeps exp(x - m) defined.
//
// One warp per token, the logits in registers (lane l holds experts l, l + 32,
// ...).  All maxima are taken on order-preserving integer images of the floats
// by the warp's integer reduction, so the choice is exact and does not depend
// on any order of evaluation.
#include <type_traits>

#include <cuda_runtime.h>

#include "tkq_device.cuh"
#include "tkq_internal.h"

namespace tkq {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr unsigned kAll = 0xffffffffu;
constexpr float kLargest = 3.402823466e+38f;
constexpr float kMinusInf = -__builtin_huge_valf();

// Order-preserving image of a key, 0 for a key that cannot be chosen (-inf, NaN).
__device__ __forceinline__ uint32_t image(float key) {
    const uint32_t b = __float_as_uint(key);
    const uint32_t u = b ^ (static_cast<uint32_t>(static_cast<int32_t>(b) >> 31) | 0x80000000u);
    return key > kMinusInf ? u : 0u;
}
__device__ __forceinline__ float from_image(uint32_t u) {
    return __uint_as_float(u ^ ((u >> 31) ? 0x80000000u : 0xffffffffu));
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kAll, v, o);
    return v;
}

// One logit; -inf stands for an absent expert, +inf becomes the largest number.
template <bool BF16>
__device__ __forceinline__ float load_logit(const void* row, int e) {
    float x;
    if constexpr (BF16)
        x = __uint_as_float(static_cast<uint32_t>(ld_ro(static_cast<const uint16_t*>(row) + e))
                            << 16);
    else
        x = ld_ro(static_cast<const float*>(row) + e);
    return x > kMinusInf ? fminf(x, kLargest) : kMinusInf;
}

template <bool BF16>
__device__ __forceinline__ const void* row_of(const void* logits, int64_t t, int64_t ld) {
    return static_cast<const char*>(logits) + t * ld * (BF16 ? 2 : 4);
}

// Scores of the lane's logits in place (x becomes the score, 0 where absent).
template <int SLOTS>
__device__ __forceinline__ void to_scores(float (&x)[SLOTS], bool sigmoid) {
    if (sigmoid) {
#pragma unroll
        for (int s = 0; s < SLOTS; ++s)
            x[s] = x[s] > kMinusInf ? __fdiv_rn(1.0f, 1.0f + expf(-x[s])) : 0.0f;
        return;
    }
    uint32_t m = 0;
#pragma unroll
    for (int s = 0; s < SLOTS; ++s) m = max(m, image(x[s]));
    m = __reduce_max_sync(kAll, m);
    const float top = m ? from_image(m) : 0.0f;
    float sum = 0.0f;
#pragma unroll
    for (int s = 0; s < SLOTS; ++s) {
        x[s] = x[s] > kMinusInf ? expf(x[s] - top) : 0.0f;
        sum += x[s];
    }
    sum = fmaxf(warp_sum(sum), 1.0f);  // at least exp(0) unless no expert is there
#pragma unroll
    for (int s = 0; s < SLOTS; ++s) x[s] = __fdiv_rn(x[s], sum);
}

template <int SLOTS, bool BF16>
__global__ void __launch_bounds__(kThreads)
    route_topk_kernel(const void* __restrict__ logits, const float* __restrict__ bias,
                      int32_t* __restrict__ ids, float* __restrict__ weights,
                      int32_t* __restrict__ counts, int64_t T, int64_t ld, RouteShape sh) {
    extern __shared__ uint32_t shared[];
    grid_dependency_launch();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int32_t* tally = reinterpret_cast<int32_t*>(shared);  // [E], when counts are wanted
    uint32_t* keys = shared + (counts ? sh.E : 0) + warp * sh.E;  // [E] a warp, with groups
    if (counts) {
        for (int e = threadIdx.x; e < sh.E; e += kThreads) tally[e] = 0;
        __syncthreads();
    }
    grid_dependency_wait();
    float b[SLOTS];
#pragma unroll
    for (int s = 0; s < SLOTS; ++s) {
        const int e = lane + 32 * s;
        b[s] = bias && e < sh.E ? ld_ro(bias + e) : 0.0f;
    }
    const int per = sh.E / sh.groups;
    for (int64_t t = static_cast<int64_t>(blockIdx.x) * kWarps + warp; t < T;
         t += static_cast<int64_t>(gridDim.x) * kWarps) {
        const void* row = row_of<BF16>(logits, t, ld);
        float x[SLOTS];
        uint32_t u[SLOTS];
#pragma unroll
        for (int s = 0; s < SLOTS; ++s) {
            const int e = lane + 32 * s;
            x[s] = e < sh.E ? load_logit<BF16>(row, e) : kMinusInf;
            u[s] = x[s] > kMinusInf;
        }
        to_scores<SLOTS>(x, sh.sigmoid);
#pragma unroll
        for (int s = 0; s < SLOTS; ++s) u[s] = u[s] ? image(x[s] + b[s]) : 0u;

        if (sh.groups > 1) {
            // lane g scores group g from the warp's copy of the keys
            __syncwarp();
#pragma unroll
            for (int s = 0; s < SLOTS; ++s)
                if (lane + 32 * s < sh.E) keys[lane + 32 * s] = u[s];
            __syncwarp();
            uint32_t best = 0, second = 0;
            if (lane < sh.groups)
                for (int i = 0; i < per; ++i) {
                    const uint32_t v = keys[lane * per + i];
                    second = max(second, min(best, v));
                    best = max(best, v);
                }
            uint32_t score = best;
            if (sh.group_top == 2 && second) score = image(from_image(best) + from_image(second));
            unsigned kept = 0;
            for (int i = 0; i < sh.topk_groups; ++i) {
                const uint32_t m = __reduce_max_sync(kAll, score);
                const int g = __ffs(__ballot_sync(kAll, score == m)) - 1;
                kept |= 1u << g;
                if (lane == g) score = 0;
                if (m == 0) break;
            }
#pragma unroll
            for (int s = 0; s < SLOTS; ++s)
                if (!(kept >> ((lane + 32 * s) / per) & 1u)) u[s] = 0;
        }

        // k rounds of: the largest key, its lowest index, taken out
        int my_id = -1;
        float my_w = 0.0f;
        for (int i = 0; i < sh.k; ++i) {
            uint32_t lmax = 0;
#pragma unroll
            for (int s = 0; s < SLOTS; ++s) lmax = max(lmax, u[s]);
            const uint32_t m = __reduce_max_sync(kAll, lmax);
            if (m == 0) break;
            unsigned e = ~0u;
            float sc = 0.0f;
#pragma unroll
            for (int s = SLOTS - 1; s >= 0; --s)
                if (u[s] == m) {
                    e = lane + 32 * s;
                    sc = x[s];
                }
            const unsigned first = __reduce_min_sync(kAll, e);
            const float w = __shfl_sync(kAll, sc, first & 31);
#pragma unroll
            for (int s = 0; s < SLOTS; ++s)
                if (first == lane + 32u * s) u[s] = 0;
            if (lane == i) {
                my_id = static_cast<int>(first);
                my_w = w;
            }
        }
        if (sh.renorm) {
            const float total = warp_sum(my_w);
            my_w = total > 0.0f ? __fdiv_rn(my_w, total) : 0.0f;
        }
        if (lane < sh.k) {
            st_plain(ids + t * sh.k + lane, my_id);
            st_plain(weights + t * sh.k + lane, my_w * sh.scale);
            if (counts && my_id >= 0) atomicAdd(tally + my_id, 1);
        }
    }
    if (counts) {
        __syncthreads();
        for (int e = threadIdx.x; e < sh.E; e += kThreads)
            if (tally[e]) atomic_add_count(counts + e, tally[e]);
    }
}

template <int SLOTS, bool BF16>
__global__ void __launch_bounds__(kThreads)
    route_backward_kernel(const void* __restrict__ logits, const int32_t* __restrict__ ids,
                          const float* __restrict__ dweights, void* __restrict__ dlogits,
                          int64_t T, int64_t ld, RouteShape sh) {
    extern __shared__ uint32_t shared[];
    grid_dependency_launch();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    float* ds = reinterpret_cast<float*>(shared) + warp * sh.E;  // [E] a warp
    grid_dependency_wait();
    for (int64_t t = static_cast<int64_t>(blockIdx.x) * kWarps + warp; t < T;
         t += static_cast<int64_t>(gridDim.x) * kWarps) {
        const void* row = row_of<BF16>(logits, t, ld);
        float x[SLOTS], p[SLOTS];
#pragma unroll
        for (int s = 0; s < SLOTS; ++s) {
            const int e = lane + 32 * s;
            x[s] = e < sh.E ? load_logit<BF16>(row, e) : kMinusInf;
            p[s] = x[s];
        }
        to_scores<SLOTS>(p, sh.sigmoid);
        // ids outside [0, E) are empty slots
        int id = lane < sh.k ? ld_ro(ids + t * sh.k + lane) : -1;
        if (id < 0 || id >= sh.E) id = -1;
        float a = id >= 0 ? sh.scale * ld_ro(dweights + t * sh.k + lane) : 0.0f;
        __syncwarp();
        if (sh.renorm) {
#pragma unroll
            for (int s = 0; s < SLOTS; ++s)
                if (lane + 32 * s < sh.E) ds[lane + 32 * s] = p[s];
            __syncwarp();
            const float score = id >= 0 ? ds[id] : 0.0f;
            const float total = warp_sum(score);
            // by the weights p / S, which are exactly 1 for a single expert: its gradient is 0
            const float dot = warp_sum(total > 0.0f ? a * __fdiv_rn(score, total) : 0.0f);
            a = total > 0.0f && id >= 0 ? __fdiv_rn(a - dot, total) : 0.0f;
            __syncwarp();
        }
#pragma unroll
        for (int s = 0; s < SLOTS; ++s)
            if (lane + 32 * s < sh.E) ds[lane + 32 * s] = 0.0f;
        __syncwarp();
        for (int i = 0; i < sh.k; ++i) {  // in order: an id given twice adds up the same each time
            if (lane == i && id >= 0) ds[id] += a;
            __syncwarp();
        }
        float dot = 0.0f;
        float g[SLOTS];
#pragma unroll
        for (int s = 0; s < SLOTS; ++s) {
            g[s] = lane + 32 * s < sh.E ? ds[lane + 32 * s] : 0.0f;
            dot += g[s] * p[s];
        }
        if (!sh.sigmoid) dot = warp_sum(dot);
        char* out = static_cast<char*>(dlogits) + t * sh.E * (BF16 ? 2 : 4);
#pragma unroll
        for (int s = 0; s < SLOTS; ++s) {
            const int e = lane + 32 * s;
            if (e >= sh.E) continue;
            float d;
            if (sh.sigmoid) {
                // s (1 - s) = exp(-|x|) / (1 + exp(-|x|))^2, without cancellation
                const float q = expf(-fabsf(x[s]));
                d = __fdiv_rn(g[s] * q, (1.0f + q) * (1.0f + q));
            } else {
                d = p[s] * (g[s] - dot);
            }
            if (!(x[s] > kMinusInf)) d = 0.0f;
            if constexpr (BF16)
                st_plain(reinterpret_cast<uint16_t*>(out) + e,
                         static_cast<uint16_t>(pack_bf16x2(d, 0.0f)));
            else
                st_plain(reinterpret_cast<float*>(out) + e, d);
        }
        __syncwarp();
    }
}

// Registers for E logits a lane: the next power of two of E / 32.
template <typename F>
cudaError_t with_slots(int E, F&& f) {
    if (E <= 32) return f(std::integral_constant<int, 1>());
    if (E <= 64) return f(std::integral_constant<int, 2>());
    if (E <= 128) return f(std::integral_constant<int, 4>());
    if (E <= 256) return f(std::integral_constant<int, 8>());
    if (E <= 512) return f(std::integral_constant<int, 16>());
    return f(std::integral_constant<int, 32>());
}

}  // namespace

cudaError_t launch_route_topk(const void* logits, const float* bias, int32_t* ids, float* weights,
                              int32_t* counts, int64_t T, int64_t ld, const RouteShape& sh,
                              cudaStream_t stream) {
    return with_slots(sh.E, [&](auto slots) {
        constexpr int S = decltype(slots)::value;
        auto* k = sh.bf16 ? &route_topk_kernel<S, true> : &route_topk_kernel<S, false>;
        const size_t smem = 4u * sh.E * ((counts ? 1 : 0) + (sh.groups > 1 ? kWarps : 0));
        const int grid = persistent_grid(reinterpret_cast<const void*>(k), kThreads, smem,
                                         (T + kWarps - 1) / kWarps);
        if (const cudaError_t e = upload_checks(stream)) return e;
        return launch_pdl(k, grid, kThreads, smem, stream, true, logits, bias, ids, weights,
                          counts, T, ld, sh);
    });
}

cudaError_t launch_route_topk_backward(const void* logits, const int32_t* ids,
                                       const float* dweights, void* dlogits, int64_t T, int64_t ld,
                                       const RouteShape& sh, cudaStream_t stream) {
    return with_slots(sh.E, [&](auto slots) {
        constexpr int S = decltype(slots)::value;
        auto* k = sh.bf16 ? &route_backward_kernel<S, true> : &route_backward_kernel<S, false>;
        const size_t smem = 4u * sh.E * kWarps;
        const int grid = persistent_grid(reinterpret_cast<const void*>(k), kThreads, smem,
                                         (T + kWarps - 1) / kWarps);
        if (const cudaError_t e = upload_checks(stream)) return e;
        return launch_pdl(k, grid, kThreads, smem, stream, true, logits, ids, dweights, dlogits, T,
                          ld, sh);
    });
}

}  // namespace tkq
