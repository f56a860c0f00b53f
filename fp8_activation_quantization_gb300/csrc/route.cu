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
// Backward, with a_i = scale * dw_i, p_i the chosen scores, S their sum, r_i = p_i / S:
//   dx_e = a_e s_e (1 - s_e)                or  s_e (a_e - sum_j a_j p_j), renormalised
//   dx_e = (a_e - sum_j a_j r_j) r_e [(1 - s_e)]  of the chosen, 0 elsewhere: the
// sum over the experts that the softmax's gradient takes off is then 0.  The r_i
// come from the chosen logits alone, by the distance from the largest of them, so
// that they hold where the scores themselves underflow.
//
// An expert is absent from a token's row when its logit is -inf or NaN: it has
// no share in the softmax, is never chosen and gets no gradient.  When fewer
// than k experts are left the remaining ids are -1 with weight 0, so a row
// without any expert is all -1.  A logit of +inf counts as the largest finite
// number, which keeps exp(x - m) defined.
//
// Logits in registers: lane l of a token's lanes holds the SLOTS experts from
// l * SLOTS on, so a lower lane holds lower indices and a group of experts is a
// run of lanes.  The forward is bound by instructions, not memory (16384 x 256
// fp32 is 2.7 us of reads).  So a token has 8 or 16 lanes where its experts fit
// (LANES, `with_lanes`), and 4 or 2 tokens share a warp's instructions; and the
// choice is made in two steps: the k-th largest of the lanes' maxima bounds the
// k-th largest key from below; the few keys that reach it are gathered and ranked
// by counting.  8 of 256 experts at 16384 tokens, sigmoid: 12.8 us, in 8 groups of
// which 4 are searched, with a bias, 17.9 us (35.0 us with k rounds over all keys);
// from memory 13.8 and 18.8 us.
// The backward has one warp per token and writes each row through shared memory,
// so that it leaves as 16-byte vectors.  16384 x 256 fp32, softmax: 6.5 us with
// renormalised weights, for which the chosen logits are read alone, 7.5 us without;
// sigmoid: 7.0 and 5.0 us.  These are with 70 MB of inputs and outputs, which stay
// in L2; with 1 GB of them in turn 8.7, 9.2, 9.0 and 7.5 us.
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
// Below this sum of the chosen scores the smallest of them may have lost bits that
// count, or the sigmoid's (below 2^-126, about exp(-87)) be 0.
constexpr float kTinyTotal = 0x1p-64f;

// Sum and maximum (no NaN) over LANES consecutive lanes.
template <int LANES>
__device__ __forceinline__ float team_sum(float v) {
#pragma unroll
    for (int o = LANES / 2; o > 0; o >>= 1) v += __shfl_xor_sync(kAll, v, o);
    return v;
}
__device__ __forceinline__ float warp_sum(float v) { return team_sum<32>(v); }
template <int LANES>
__device__ __forceinline__ float team_max(float v) {
    if constexpr (LANES == 32) {
        float r;
        asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
        return r;
    } else {
#pragma unroll
        for (int o = LANES / 2; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(kAll, v, o));
        return v;
    }
}

// A lane's logits as loaded.  `wide`: rows and E allow loads of a lane's logits
// as vectors (wide_rows below), else they are read one by one.
template <int SLOTS, bool BF16>
struct Raw {
    static constexpr int kItem = BF16 ? 2 : 4;
    static constexpr int kBytes = SLOTS * kItem < 16 ? SLOTS * kItem : 16;  // of one load
    static constexpr int kVec = kBytes / kItem;                            // its logits
    uint32_t w[(SLOTS * kItem + 3) / 4];

    // -inf everywhere: what no load overwrites, beyond the last expert, is absent.
    __device__ __forceinline__ void clear() {
#pragma unroll
        for (int i = 0; i < static_cast<int>(sizeof w / 4); ++i) w[i] = BF16 ? 0xff80ff80u : 0xff800000u;
    }
    __device__ __forceinline__ void load(const void* row, int lane, int E, bool wide) {
        const char* p = static_cast<const char*>(row) + lane * SLOTS * kItem;
        if (kBytes >= 8 && wide) {
#pragma unroll
            for (int s = 0; s < SLOTS; s += kVec) {
                if (lane * SLOTS + s >= E) continue;
                uint32_t* to = w + s * kItem / 4;
                if constexpr (kBytes == 16) {
                    const uint4 v = ld_ro(reinterpret_cast<const uint4*>(p + s * kItem));
                    to[0] = v.x; to[1] = v.y; to[2] = v.z; to[3] = v.w;
                } else if constexpr (kBytes == 8) {
                    const uint2 v = ld_ro(reinterpret_cast<const uint2*>(p + s * kItem));
                    to[0] = v.x; to[1] = v.y;
                }
            }
            return;
        }
#pragma unroll
        for (int s = 0; s < SLOTS; ++s) {
            if (lane * SLOTS + s >= E) continue;
            if constexpr (BF16) {
                const uint32_t v = ld_ro(reinterpret_cast<const uint16_t*>(p) + s);
                w[s / 2] = s % 2 ? (w[s / 2] & 0xffffu) | v << 16 : (w[s / 2] & 0xffff0000u) | v;
            } else {
                w[s] = __float_as_uint(ld_ro(reinterpret_cast<const float*>(p) + s));
            }
        }
    }
    // -inf stands for an absent expert, +inf becomes the largest number.
    __device__ __forceinline__ void values(float (&x)[SLOTS]) const {
#pragma unroll
        for (int s = 0; s < SLOTS; ++s) {
            float v;
            if constexpr (BF16)
                v = s % 2 ? bf16_hi(w[s / 2]) : bf16_lo(w[s / 2]);
            else
                v = __uint_as_float(w[s]);
            x[s] = v > kMinusInf ? fminf(v, kLargest) : kMinusInf;
        }
    }
};

template <int SLOTS, bool BF16>
bool wide_rows(const void* base, int64_t ld, int E) {
    using R = Raw<SLOTS, BF16>;
    return reinterpret_cast<uintptr_t>(base) % R::kBytes == 0 && ld * R::kItem % R::kBytes == 0 &&
           E % R::kVec == 0;
}

template <bool BF16>
__device__ __forceinline__ const void* row_of(const void* logits, int64_t t, int64_t ld) {
    return static_cast<const char*>(logits) + t * ld * (BF16 ? 2 : 4);
}

__device__ __forceinline__ float logistic(float x) { return rcp_approx(1.0f + expf(-x)); }

// Scores of the lane's logits (0 where absent).
template <int SLOTS, int LANES>
__device__ __forceinline__ void scores_of(const float (&x)[SLOTS], bool sigmoid,
                                          float (&p)[SLOTS]) {
    if (sigmoid) {
#pragma unroll
        for (int s = 0; s < SLOTS; ++s) p[s] = logistic(x[s]);  // exp(inf) = inf gives 0
        return;
    }
    float m = x[0];
#pragma unroll
    for (int s = 1; s < SLOTS; ++s) m = fmaxf(m, x[s]);
    m = team_max<LANES>(m);
    const float top = m > kMinusInf ? m : 0.0f;
    float sum = 0.0f;
#pragma unroll
    for (int s = 0; s < SLOTS; ++s) {
        p[s] = expf(x[s] - top);
        sum += p[s];
    }
    // at least exp(0) unless no expert is there
    const float r = __fdiv_rn(1.0f, fmaxf(team_sum<LANES>(sum), 1.0f));
#pragma unroll
    for (int s = 0; s < SLOTS; ++s) p[s] *= r;
}

// What a token keeps in shared memory: the gathered keys (-inf where there is
// none) with their experts and scores, and the choice in order.
constexpr int kBench = 64;  // keys gathered at most
struct alignas(16) Bench {
    float key[kBench], score[kBench], chosen_score[32];
    int id[kBench], chosen[32];

    template <int LANES>
    __device__ __forceinline__ void clear(int l) {
        for (int i = 4 * l; i < kBench; i += 4 * LANES)
            *reinterpret_cast<float4*>(key + i) =
                make_float4(kMinusInf, kMinusInf, kMinusInf, kMinusInf);
        for (int i = l; i < 32; i += LANES) {
            chosen[i] = -1;
            chosen_score[i] = 0.0f;
        }
    }
};

// Takes the keys of the experts outside the best topk_groups groups out.  A
// group's score comes from its lanes where groups are runs of 1, 2, 4 .. lanes
// (group_lanes > 0), else one lane reads a group's keys from shared memory.
template <int SLOTS, int LANES>
__device__ __forceinline__ void keep_groups(float (&key)[SLOTS], const RouteShape& sh, int l,
                                            int group_lanes, float* shared_keys) {
    const int per = sh.E / sh.groups;
    float best = kMinusInf, second = kMinusInf;
    const auto take = [&](float v) {
        second = fmaxf(second, fminf(best, v));
        best = fmaxf(best, v);
    };
    const auto score_of = [&] {
        return sh.group_top == 2 && second > kMinusInf ? best + second : best;
    };
    // rank of a group: how many are better, or equal and before it
    if (group_lanes > 0) {
#pragma unroll
        for (int s = 0; s < SLOTS; ++s) take(key[s]);
        for (int o = 1; o < group_lanes; o <<= 1) {
            const float b = __shfl_xor_sync(kAll, best, o), c = __shfl_xor_sync(kAll, second, o);
            second = fmaxf(fmaxf(second, c), fminf(best, b));
            best = fmaxf(best, b);
        }
        const float score = score_of();
        const int mine = l / group_lanes;
        int rank = 0;
#pragma unroll 4
        for (int g = 0; g < sh.groups; ++g) {
            const float v = __shfl_sync(kAll, score, g * group_lanes, LANES);
            rank += v > score || (v == score && g < mine);
        }
        if (rank >= sh.topk_groups) {
#pragma unroll
            for (int s = 0; s < SLOTS; ++s) key[s] = kMinusInf;
        }
        return;
    }
    // [E] keys, then [32] scores; as many lanes a group as there are, a part of
    // its keys each
    float* scores = shared_keys + sh.E;
    __syncwarp();
#pragma unroll
    for (int s = 0; s < SLOTS; ++s)
        if (l * SLOTS + s < sh.E) shared_keys[l * SLOTS + s] = key[s];
    __syncwarp();
    int parts = 1;
    while (parts * 2 * sh.groups <= LANES) parts *= 2;
    for (int g0 = 0; g0 < sh.groups; g0 += LANES / parts) {
        const int g = g0 + l / parts;
        best = second = kMinusInf;
        if (g < sh.groups)
            for (int i = l % parts; i < per; i += parts) take(shared_keys[g * per + i]);
        for (int o = 1; o < parts; o <<= 1) {
            const float b = __shfl_xor_sync(kAll, best, o), c = __shfl_xor_sync(kAll, second, o);
            second = fmaxf(fmaxf(second, c), fminf(best, b));
            best = fmaxf(best, b);
        }
        if (g < sh.groups && l % parts == 0) scores[g] = score_of();
    }
    __syncwarp();
    unsigned kept = 0;
    for (int g = l; g < sh.groups; g += LANES) {
        const float mine = scores[g];
        int rank = 0;
        for (int i = 0; i < sh.groups; ++i) {
            const float v = scores[i];
            rank += v > mine || (v == mine && i < g);
        }
        kept |= (rank < sh.topk_groups ? 1u : 0u) << g;
    }
    __syncwarp();
#pragma unroll
    for (int o = LANES / 2; o > 0; o >>= 1) kept |= __shfl_xor_sync(kAll, kept, o);
    int g = l * SLOTS / per, left = per - (l * SLOTS - g * per);  // of the group's experts
#pragma unroll
    for (int s = 0; s < SLOTS; ++s) {
        if (g > 31 || !(kept >> g & 1u)) key[s] = kMinusInf;
        if (--left == 0) {
            ++g;
            left = per;
        }
    }
}

// The k largest keys in falling order, ties to the lowest index, into
// bench.chosen / chosen_score (untouched beyond what there is).  All tokens of the
// warp go through the same steps.
template <int SLOTS, int LANES>
__device__ __forceinline__ void choose(float (&key)[SLOTS], const float (&score)[SLOTS], int k,
                                       int l, Bench& bench) {
    float top = key[0];
#pragma unroll
    for (int s = 1; s < SLOTS; ++s) top = fmaxf(top, key[s]);
    // the k-th largest of the lanes' maxima: the least of those that fewer than k
    // others exceed; any key there is, if there are fewer lanes than k with one
    int larger = 0;
#pragma unroll
    for (int o = 1; o < LANES; ++o) larger += __shfl_xor_sync(kAll, top, o) > top;
    const float least = -team_max<LANES>(larger < k ? -top : kMinusInf);
    const float bound = k <= LANES ? fmaxf(least, -kLargest) : -kLargest;
    // gathered in the order of the lanes and their slots, which is that of the experts
    unsigned in = 0;
#pragma unroll
    for (int s = 0; s < SLOTS; ++s) in |= (key[s] >= bound ? 1u : 0u) << s;
    const int own = __popc(in);
    int upto = own;
#pragma unroll
    for (int o = 1; o < LANES; o <<= 1) {
        const int v = __shfl_up_sync(kAll, upto, o, LANES);
        if (l >= o) upto += v;
    }
    const int count = __shfl_sync(kAll, upto, LANES - 1, LANES);
    const int most = __reduce_max_sync(kAll, count);
    if (most <= kBench) {
        int at = upto - own;
#pragma unroll
        for (int s = 0; s < SLOTS; ++s)
            if (in >> s & 1u) {
                bench.key[at] = key[s];
                bench.score[at] = score[s];
                bench.id[at] = l * SLOTS + s;
                ++at;
            }
        __syncwarp();
        for (int c = l; c - l < most; c += LANES) {
            // rank: how many are larger, or equal and before it
            const float mine = c < kBench ? bench.key[c] : kMinusInf;
            int rank = 0;
            for (int i = 0; i < most; i += 4) {
                const float4 v = *reinterpret_cast<const float4*>(bench.key + i);
                rank += v.x > mine || (v.x == mine && i < c);
                rank += v.y > mine || (v.y == mine && i + 1 < c);
                rank += v.z > mine || (v.z == mine && i + 2 < c);
                rank += v.w > mine || (v.w == mine && i + 3 < c);
            }
            if (c < count && rank < k) {
                bench.chosen[rank] = bench.id[c];
                bench.chosen_score[rank] = bench.score[c];
            }
        }
    } else {
        // many ties, or k near the number of lanes: one key a round
        const int base = threadIdx.x & 31 & ~(LANES - 1);
        for (int i = 0; i < k; ++i) {
            float m = key[0];
#pragma unroll
            for (int s = 1; s < SLOTS; ++s) m = fmaxf(m, key[s]);
            const float best = team_max<LANES>(m);
            const unsigned who = __ballot_sync(kAll, m == best) >> base;
            bool mine = best > kMinusInf && l == __ffs(who) - 1;
#pragma unroll
            for (int s = 0; s < SLOTS; ++s)
                if (mine && key[s] == best) {
                    bench.chosen[i] = l * SLOTS + s;
                    bench.chosen_score[i] = score[s];
                    key[s] = kMinusInf;
                    mine = false;
                }
        }
    }
    __syncwarp();
}

// The chosen expert's logit, as values() gives it; -inf for an empty slot.
template <bool BF16>
__device__ __forceinline__ float logit_of(const void* row, int id) {
    if (id < 0) return kMinusInf;
    float x;
    if constexpr (BF16)
        x = __uint_as_float(static_cast<uint32_t>(ld_ro(static_cast<const uint16_t*>(row) + id)) << 16);
    else
        x = ld_ro(static_cast<const float*>(row) + id);
    return x > kMinusInf ? fminf(x, kLargest) : kMinusInf;
}

// A score up to a factor that all chosen experts share, `lead` their largest
// score_lead: exp(x - lead), times 1 / (1 + exp(-|x|)) for the sigmoid.  Of order
// one for the largest, however small the scores are.
__device__ __forceinline__ float score_lead(float x, bool sigmoid) {
    return sigmoid ? fminf(x, 0.0f) : x;
}
__device__ __forceinline__ float score_ratio(float x, bool sigmoid, float lead) {
    if (!(x > kMinusInf)) return 0.0f;
    const float e = expf(score_lead(x, sigmoid) - lead);
    return sigmoid ? e * rcp_approx(1.0f + expf(-fabsf(x))) : e;
}

template <int SLOTS, int LANES, bool BF16>
__global__ void __launch_bounds__(kThreads)
    route_topk_kernel(const void* __restrict__ logits, const float* __restrict__ bias,
                      int32_t* __restrict__ ids, float* __restrict__ weights,
                      int32_t* __restrict__ counts, int64_t T, int64_t ld, RouteShape sh,
                      bool wide, int group_lanes) {
    constexpr int kTokens = 32 / LANES;  // of a warp
    constexpr int kPitch = SLOTS + 4;    // of a lane's biases: vectors in different banks
    extern __shared__ __align__(16) float shared[];
    __shared__ Bench benches[kWarps * kTokens];
    __shared__ __align__(16) float biases[LANES * kPitch];
    grid_dependency_launch();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int l = lane % LANES, team = warp * kTokens + lane / LANES;
    Bench& bench = benches[team];
    int32_t* tally = reinterpret_cast<int32_t*>(shared);               // [E], when counts are wanted
    float* keys = shared + (counts ? sh.E : 0) + team * (sh.E + 32);   // when group_lanes == 0
    if (counts)
        for (int e = threadIdx.x; e < sh.E; e += kThreads) tally[e] = 0;
    const int64_t step = static_cast<int64_t>(gridDim.x) * kWarps * kTokens;
    int64_t t = static_cast<int64_t>(blockIdx.x) * kWarps * kTokens + team;
    grid_dependency_wait();
    // a bias of NaN takes its expert out as -inf does
    for (int e = threadIdx.x; e < LANES * SLOTS; e += kThreads) {
        const float b = bias && e < sh.E ? ld_ro(bias + e) : 0.0f;
        biases[e / SLOTS * kPitch + e % SLOTS] = b > kMinusInf ? b : kMinusInf;
    }
    __syncthreads();
    Raw<SLOTS, BF16> raw;
    raw.clear();
    if (t < T) raw.load(row_of<BF16>(logits, t, ld), l, sh.E, wide);
    // a warp's tokens go together: the first lane's token says whether there is one
    for (int64_t t0 = t - lane / LANES; t0 < T; t0 += step, t += step) {
        float x[SLOTS], p[SLOTS];
        raw.values(x);
        if (t + step < T) raw.load(row_of<BF16>(logits, t + step, ld), l, sh.E, wide);
        scores_of<SLOTS, LANES>(x, sh.sigmoid, p);
#pragma unroll
        for (int s = 0; s < SLOTS; s += 4) {
            const float4 b = *reinterpret_cast<const float4*>(biases + l * kPitch + s);
            x[s] = x[s] > kMinusInf ? p[s] + b.x : kMinusInf;
            x[s + 1] = x[s + 1] > kMinusInf ? p[s + 1] + b.y : kMinusInf;
            x[s + 2] = x[s + 2] > kMinusInf ? p[s + 2] + b.z : kMinusInf;
            x[s + 3] = x[s + 3] > kMinusInf ? p[s + 3] + b.w : kMinusInf;
        }
        if (sh.groups > 1) keep_groups<SLOTS, LANES>(x, sh, l, group_lanes, keys);
        bench.clear<LANES>(l);
        __syncwarp();
        choose<SLOTS, LANES>(x, p, sh.k, l, bench);

        float total = 0.0f;
        for (int i = l; i < sh.k; i += LANES) total += bench.chosen_score[i];
        total = team_sum<LANES>(total);
        // Renormalised weights are ratios, which hold where the scores underflow: once
        // more from the logits.  (A row's path does not depend on its neighbours'.)
        const bool tiny = sh.renorm && total < kTinyTotal && t < T && bench.chosen[0] >= 0;
        if (__any_sync(kAll, tiny)) {
            const void* row = row_of<BF16>(logits, t, ld);
            const int from = tiny ? l : sh.k;
            float lead = kMinusInf, again = 0.0f;
            for (int i = from; i < sh.k; i += LANES)
                lead = fmaxf(lead, score_lead(logit_of<BF16>(row, bench.chosen[i]), sh.sigmoid));
            lead = team_max<LANES>(lead);
            for (int i = from; i < sh.k; i += LANES) {
                const float part =
                    score_ratio(logit_of<BF16>(row, bench.chosen[i]), sh.sigmoid, lead);
                bench.chosen_score[i] = part;  // read by this lane alone
                again += part;
            }
            again = team_sum<LANES>(again);
            if (tiny) total = again;
        }
        if (t < T)
            for (int i = l; i < sh.k; i += LANES) {
                const int id = bench.chosen[i];
                float w = bench.chosen_score[i];
                if (sh.renorm) w = total > 0.0f ? __fdiv_rn(w, total) : 0.0f;
                st_plain(ids + t * sh.k + i, id);
                st_plain(weights + t * sh.k + i, w * sh.scale);
                if (counts && id >= 0) atomicAdd(tally + id, 1);
            }
        __syncwarp();
    }
    if (counts) {
        __syncthreads();
        for (int e = threadIdx.x; e < sh.E; e += kThreads)
            if (tally[e]) atomic_add_count(counts + e, tally[e]);
    }
}

// One output row from the warp's copy in shared memory, as 16-byte vectors where
// the rows allow it.
template <bool BF16>
__device__ __forceinline__ void store_row(void* out, const float* row, int E, int lane, bool wide) {
    constexpr int kVec = BF16 ? 8 : 4;
    if (wide) {
        for (int e = lane * kVec; e < E; e += 32 * kVec) {
            uint4* to = static_cast<uint4*>(out) + e / kVec;
            const float4 a = *reinterpret_cast<const float4*>(row + e);
            if constexpr (BF16) {
                const float4 b = *reinterpret_cast<const float4*>(row + e + 4);
                const float v[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
                st_stream(to, pack8_bf16(v));
            } else {
                st_stream(to, make_uint4(__float_as_uint(a.x), __float_as_uint(a.y),
                                         __float_as_uint(a.z), __float_as_uint(a.w)));
            }
        }
        return;
    }
    for (int e = lane; e < E; e += 32) {
        if constexpr (BF16)
            st_plain(static_cast<uint16_t*>(out) + e,
                     static_cast<uint16_t>(pack_bf16x2(row[e], 0.0f)));
        else
            st_plain(static_cast<float*>(out) + e, row[e]);
    }
}

// Gradient of the lane's chosen logit from a = scale * dweight.  A single
// renormalised expert has r = 1 exactly, and the gradient 0.
__device__ __forceinline__ float chosen_grad(float a, float x, const RouteShape& sh) {
    if (!sh.renorm) {  // the sigmoid: s (1 - s), without cancellation
        const float q = expf(-fabsf(x)), r = rcp_approx(1.0f + q);
        return a * q * r * r;
    }
    const float part = score_ratio(x, sh.sigmoid, team_max<32>(score_lead(x, sh.sigmoid)));
    const float total = warp_sum(part);
    const float share = total > 0.0f ? __fdiv_rn(part, total) : 0.0f;
    const float d = (a - warp_sum(a * share)) * share;
    if (!sh.sigmoid) return d;
    const float q = expf(-fabsf(x)), r = rcp_approx(1.0f + q);
    return d * (x > 0.0f ? q * r : r);  // 1 - s
}

// Adds v to row[id] for every lane with id >= 0; an id given more than once adds
// up in the order of its slots.
__device__ __forceinline__ void scatter(float* row, int id, float v, int lane) {
    const unsigned same = __match_any_sync(kAll, id);
    float sum = 0.0f;
    unsigned rest = same;
    while (__any_sync(kAll, rest)) {
        const int from = rest ? __ffs(rest) - 1 : lane;
        const float x = __shfl_sync(kAll, v, from);
        if (rest) sum += x;
        rest &= rest - 1;
        if (__all_sync(kAll, id < 0 || !rest)) break;
    }
    if (id >= 0 && lane == __ffs(same) - 1) row[id] += sum;
}

// Floats of a warp's row in shared memory: all lanes' slots, or E rounded up to
// whole 16-byte vectors of bf16 where no slots are written (slots 0).
__host__ __device__ constexpr int row_length(int E, int slots) {
    return slots ? (slots < 4 ? (32 * slots + 7) / 8 * 8 : 32 * slots) : (E + 7) / 8 * 8;
}

// The lane's slots into the warp's row, as vectors where there are four or more.
template <int SLOTS>
__device__ __forceinline__ void put_row(float* row, int lane, const float (&v)[SLOTS]) {
    float* to = row + lane * SLOTS;
    if constexpr (SLOTS >= 4) {
#pragma unroll
        for (int s = 0; s < SLOTS; s += 4)
            *reinterpret_cast<float4*>(to + s) = make_float4(v[s], v[s + 1], v[s + 2], v[s + 3]);
    } else {
#pragma unroll
        for (int s = 0; s < SLOTS; ++s) to[s] = v[s];
    }
}

// CHOSEN: only the chosen logits count (the sigmoid, renormalised weights).
template <int SLOTS, bool BF16, bool CHOSEN>
__global__ void __launch_bounds__(kThreads)
    route_backward_kernel(const void* __restrict__ logits, const int32_t* __restrict__ ids,
                          const float* __restrict__ dweights, void* __restrict__ dlogits,
                          int64_t T, int64_t ld, RouteShape sh, bool wide, bool wide_out) {
    extern __shared__ __align__(16) float shared[];
    grid_dependency_launch();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int length = row_length(sh.E, CHOSEN ? 0 : SLOTS);
    float* row = shared + warp * length;
    const int64_t step = static_cast<int64_t>(gridDim.x) * kWarps;
    int64_t t = static_cast<int64_t>(blockIdx.x) * kWarps + warp;
    // the slot's id (one outside [0, E) is an empty slot) and gradient
    int next_id = -1;
    float next_a = 0.0f;
    Raw<SLOTS, BF16> raw;
    raw.clear();
    const auto load = [&](int64_t at) {
        if (at >= T) return;
        if constexpr (!CHOSEN) raw.load(row_of<BF16>(logits, at, ld), lane, sh.E, wide);
        if (lane < sh.k) {
            next_id = ld_ro(ids + at * sh.k + lane);
            next_a = ld_ro(dweights + at * sh.k + lane);
        }
    };
    grid_dependency_wait();
    load(t);
    for (; t < T; t += step) {
        const int id = next_id >= 0 && next_id < sh.E ? next_id : -1;
        float a = id >= 0 ? sh.scale * next_a : 0.0f;
        float d = 0.0f;  // what the chosen expert's logit gets beside the row's share
        if constexpr (CHOSEN) {
            const float x = logit_of<BF16>(row_of<BF16>(logits, t, ld), id);
            if (x == kMinusInf) a = 0.0f;  // an absent expert: an empty slot
            load(t + step);
            for (int e = lane * 4; e < length; e += 128)
                *reinterpret_cast<float4*>(row + e) = make_float4(0.f, 0.f, 0.f, 0.f);
            d = chosen_grad(a, x, sh);
        } else {
            // dx_e = s_e (a_e - dot): -s_e dot for all, s_e a_e for the chosen
            float x[SLOTS], p[SLOTS];
            raw.values(x);
            load(t + step);
            scores_of<SLOTS, 32>(x, false, p);
            put_row<SLOTS>(row, lane, p);
            __syncwarp();
            const float score = id >= 0 ? row[id] : 0.0f;
            d = score > 0.0f ? a * score : 0.0f;  // an absent expert: an empty slot
            const float dot = warp_sum(d);
#pragma unroll
            for (int s = 0; s < SLOTS; ++s) p[s] *= -dot;
            __syncwarp();
            put_row<SLOTS>(row, lane, p);
        }
        __syncwarp();
        scatter(row, id, d, lane);
        __syncwarp();
        store_row<BF16>(static_cast<char*>(dlogits) + t * sh.E * (BF16 ? 2 : 4), row, sh.E, lane,
                        wide_out);
        __syncwarp();
    }
}

// The backward's registers for E logits a lane: the next power of two of E / 32.
template <typename F>
cudaError_t with_slots(int E, F&& f) {
    using std::integral_constant;
    if (E <= 32) return f(integral_constant<int, 1>());
    if (E <= 64) return f(integral_constant<int, 2>());
    if (E <= 128) return f(integral_constant<int, 4>());
    if (E <= 256) return f(integral_constant<int, 8>());
    if (E <= 512) return f(integral_constant<int, 16>());
    return f(integral_constant<int, 32>());
}
// The forward's slots and lanes a token.  Fewer lanes share a warp's instructions
// among more tokens, but the bound that `choose` starts from, the k-th largest of
// the lanes' maxima, is near only while the searched experts fill 2 k lanes: the
// fewest lanes, of up to 16 logits each, of which that holds.  Up to 32 experts
// all of them may be gathered.  65536 tokens, 8 of 256: 38 us with 16 lanes, 53 us
// with 32; 16 of 256: 97 us and 54 us; 8 of 64: 28 us with 8, 21 us with 16.
template <typename F>
cudaError_t with_lanes(const RouteShape& sh, F&& f) {
    using std::integral_constant;
    constexpr integral_constant<int, 4> c4;
    constexpr integral_constant<int, 8> c8;
    constexpr integral_constant<int, 16> c16;
    constexpr integral_constant<int, 32> c32;
    const int E = sh.E;
    // whether the searched experts fill 2 k lanes, `slots` each
    const auto fill = [&](int slots) {
        return E * sh.topk_groups >= 2 * sh.k * slots * sh.groups;
    };
    if (E <= 32) return f(c4, c8);
    if (E <= 64) return fill(8) ? f(c8, c8) : f(c4, c16);
    if (E <= 128) return fill(16) ? f(c16, c8) : fill(8) ? f(c8, c16) : f(c4, c32);
    if (E <= 256) return fill(16) ? f(c16, c16) : f(c8, c32);
    if (E <= 512) return f(c16, c32);
    return f(c32, c32);
}

}  // namespace

cudaError_t launch_route_topk(const void* logits, const float* bias, int32_t* ids, float* weights,
                              int32_t* counts, int64_t T, int64_t ld, const RouteShape& sh,
                              cudaStream_t stream) {
    return with_lanes(sh, [&](auto slots, auto lanes) {
        constexpr int S = decltype(slots)::value, L = decltype(lanes)::value;
        constexpr int kTokens = kWarps * 32 / L;  // of a CTA
        auto* k = sh.bf16 ? &route_topk_kernel<S, L, true> : &route_topk_kernel<S, L, false>;
        const bool wide = sh.bf16 ? wide_rows<S, true>(logits, ld, sh.E)
                                  : wide_rows<S, false>(logits, ld, sh.E);
        // lanes of a group, when groups are runs of a power of two of them
        const int per = sh.E / sh.groups;
        int group_lanes = per % S == 0 ? per / S : 0;
        if (group_lanes & (group_lanes - 1)) group_lanes = 0;
        const size_t smem =
            4u * ((counts ? sh.E : 0) + (sh.groups > 1 && !group_lanes ? kTokens * (sh.E + 32) : 0));
        const int grid = persistent_grid(reinterpret_cast<const void*>(k), kThreads, smem,
                                         (T + kTokens - 1) / kTokens);
        if (const cudaError_t e = upload_checks(stream)) return e;
        return launch_pdl(k, grid, kThreads, smem, stream, true, logits, bias, ids, weights,
                          counts, T, ld, sh, wide, group_lanes);
    });
}

cudaError_t launch_route_topk_backward(const void* logits, const int32_t* ids,
                                       const float* dweights, void* dlogits, int64_t T, int64_t ld,
                                       const RouteShape& sh, cudaStream_t stream) {
    const auto launch = [&](auto* k, int slots, bool wide) {
        const int64_t item = sh.bf16 ? 2 : 4;
        const bool wide_out =
            reinterpret_cast<uintptr_t>(dlogits) % 16 == 0 && sh.E * item % 16 == 0;
        const size_t smem = 4u * row_length(sh.E, slots) * kWarps;
        const int grid = persistent_grid(reinterpret_cast<const void*>(k), kThreads, smem,
                                         (T + kWarps - 1) / kWarps);
        if (const cudaError_t e = upload_checks(stream)) return e;
        return launch_pdl(k, grid, kThreads, smem, stream, true, logits, ids, dweights, dlogits, T,
                          ld, sh, wide, wide_out);
    };
    // these gradients read the chosen logits alone
    if (sh.sigmoid || sh.renorm)
        return sh.bf16 ? launch(&route_backward_kernel<1, true, true>, 0, false)
                       : launch(&route_backward_kernel<1, false, true>, 0, false);
    return with_slots(sh.E, [&](auto slots) {
        constexpr int S = decltype(slots)::value;
        return sh.bf16 ? launch(&route_backward_kernel<S, true, false>, S,
                                wide_rows<S, true>(logits, ld, sh.E))
                       : launch(&route_backward_kernel<S, false, false>, S,
                                wide_rows<S, false>(logits, ld, sh.E));
    });
}

}  // namespace tkq
