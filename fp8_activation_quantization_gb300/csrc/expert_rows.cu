// expert_rows.cu -- tokens in the order of their experts and back: the places of
// the routed pairs (tkq_expert_order), their rows gathered with or without a cast
// (tkq_expert_gather), summed back for each token (tkq_expert_reduce), and the
// gradient of that sum (tkq_expert_reduce_backward).
//
// A pair p = t k + j is token t's j-th expert.  Every kernel that moves rows walks
// tokens, not rows: a token's row is read once however many experts it goes to, and
// its sum needs no atomics.  slots[p] says where a pair's row is; a slot outside
// [0, R) is an empty one.
#include <cooperative_groups.h>
#include <cuda_runtime.h>

#include "tkq_device.cuh"
#include "tkq_internal.h"

namespace cg = cooperative_groups;

namespace tkq {
namespace {

constexpr unsigned kAll = 0xffffffffu;

// ---------------------------------------------------------------------------
// places
// ---------------------------------------------------------------------------
// A stable counting sort in one launch of one cluster: a warp counts the experts
// of its run of pairs, the warps' counts are added up within the CTA, the CTAs'
// read through distributed shared memory, and the warp then walks its run again,
// 32 pairs at a time, the lanes of one expert in pair order, so that equal experts
// keep the order of their pairs and the result does not depend on the launch.  A cluster
// of at most eight CTAs (the portable size) replaces the second launch and the workspace
// that a grid of CTAs would need; it is bound by the latency of its steps, not by the few
// bytes it moves, and from 8192 pairs on, with all eight CTAs at work, its time grows with
// their number: 65536 pairs 9 to 11 us, 131072 16, a million 89.  Each lane asks for kBatch
// of its ids at once.
constexpr int kOrderThreads = 1024;
constexpr int kOrderWarps = kOrderThreads / 32;
constexpr int kOrderMaxExperts = 1024;
constexpr int kBatch = 8;

struct OrderSmem {
    int total[kOrderMaxExperts];      // pairs of each expert in this CTA
    int start[kOrderMaxExperts + 1];  // first row of each expert
    int below[kOrderMaxExperts];      // pairs of it in the CTAs before this one, then first place of this CTA's
    int all[kOrderMaxExperts];        // pairs of each expert in all CTAs
    int warp_sum[kOrderWarps];
};

// CLUSTER: more than one CTA.
template <bool CLUSTER>
__global__ void __launch_bounds__(kOrderThreads, 1)
    order_kernel(const int32_t* __restrict__ ids, int32_t* __restrict__ slots,
                 int32_t* __restrict__ rows, int32_t* __restrict__ offsets, int P, int E, int align,
                 int R) {
    extern __shared__ int counts[];  // [kOrderWarps][E]: a warp's pairs of each expert, then their places
    __shared__ OrderSmem sm;
    cg::cluster_group cluster = cg::this_cluster();
    const int ctas = CLUSTER ? static_cast<int>(cluster.num_blocks()) : 1;
    const int rank = CLUSTER ? static_cast<int>(cluster.block_rank()) : 0;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int bits = 32 - __clz(E - 1);  // of an expert's number

    // this warp's run of pairs, a whole number of 32s
    const int per_warp = ((P + ctas * kOrderWarps - 1) / (ctas * kOrderWarps) + 31) / 32 * 32;
    const int64_t lo = static_cast<int64_t>(rank * kOrderWarps + warp) * per_warp;
    const int64_t hi = lo + per_warp < P ? lo + per_warp : P;
    const auto load = [&](int64_t p0, int (&id)[kBatch]) {
#pragma unroll
        for (int b = 0; b < kBatch; ++b) {
            const int64_t p = p0 + b * 32 + lane;
            id[b] = p < hi ? ld_ro(ids + p) : -1;
            if (id[b] < 0 || id[b] >= E) id[b] = -1;
        }
    };
    int id[kBatch];  // of the first batch, kept for the second walk
    load(lo, id);

    for (int i = threadIdx.x; i < kOrderWarps * E; i += kOrderThreads) counts[i] = 0;
    __syncthreads();
    int* mine = counts + warp * E;
    for (int64_t p0 = lo; p0 < hi; p0 += 32 * kBatch) {
        int next[kBatch];
        if (p0 > lo) load(p0, next);
#pragma unroll
        for (int b = 0; b < kBatch; ++b) {
            if (p0 + b * 32 >= hi) break;
            const int e = p0 > lo ? next[b] : id[b];
            if (e >= 0) atomicAdd(&mine[e], 1);
        }
    }
    __syncthreads();
    // counts[w][e]: pairs of e in the warps before w
    const int e = threadIdx.x;  // E <= kOrderThreads
    int n = 0;
    if (e < E) {
#pragma unroll 8
        for (int w = 0; w < kOrderWarps; ++w) {
            const int c = counts[w * E + e];
            counts[w * E + e] = n;
            n += c;
        }
    }
    int below = 0, all = n;
    if constexpr (CLUSTER) {
        if (e < E) sm.total[e] = n;
        cluster.sync();
        all = 0;
        if (e < E)
            for (int c = 0; c < ctas; ++c) {
                const int m = *cluster.map_shared_rank(&sm.total[e], c);
                if (c < rank) below += m;
                all += m;
            }
        // the other CTAs have read this one's counts before it can leave
        cluster.sync();
    }
    const int rounded = (all + align - 1) / align * align;
    int scan = rounded;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int m = __shfl_up_sync(kAll, scan, o);
        if (lane >= o) scan += m;
    }
    if (lane == 31) sm.warp_sum[warp] = scan;
    __syncthreads();
    if (warp == 0) {
        int v = sm.warp_sum[lane];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int m = __shfl_up_sync(kAll, v, o);
            if (lane >= o) v += m;
        }
        sm.warp_sum[lane] = v;
    }
    __syncthreads();
    const int incl = scan + (warp ? sm.warp_sum[warp - 1] : 0);
    if (e < E) {
        sm.start[e] = incl - rounded;
        sm.below[e] = incl - rounded + below;
        sm.all[e] = all;
        if (e == E - 1) sm.start[E] = incl;
        if (rank == 0) {
            st_plain(offsets + e, incl - rounded);
            if (e == E - 1) st_plain(offsets + E, incl);
        }
    }
    __syncthreads();

    for (int64_t p0 = lo; p0 < hi; p0 += 32 * kBatch) {
        int next[kBatch];
        if (p0 > lo) load(p0, next);
#pragma unroll
        for (int b = 0; b < kBatch; ++b) {
            const int64_t p = p0 + b * 32 + lane;
            if (p0 + b * 32 >= hi) break;
            const int x = p0 > lo ? next[b] : id[b];
            const unsigned same = lanes_of_value(x, bits, __ballot_sync(kAll, x >= 0));
            int at = 0;
            if (x >= 0) at = mine[x];
            __syncwarp();
            if (x >= 0 && lane == __ffs(same) - 1) mine[x] = at + __popc(same);
            __syncwarp();
            if (p < hi) {
                int slot = -1;
                if (x >= 0) {
                    slot = sm.below[x] + at + __popc(same & ((1u << lane) - 1u));
                    st_plain(rows + slot, static_cast<int32_t>(p));
                }
                st_plain(slots + p, slot);
            }
        }
    }
    // rows without a pair: behind each expert's and behind the last one's
    for (int x = rank * kOrderWarps + warp; x < E; x += ctas * kOrderWarps)
        for (int64_t r = static_cast<int64_t>(sm.start[x]) + sm.all[x] + lane; r < sm.start[x + 1]; r += 32)
            st_plain(rows + r, -1);
    for (int64_t r = static_cast<int64_t>(sm.start[E]) + rank * kOrderThreads + threadIdx.x; r < R;
         r += ctas * kOrderThreads)
        st_plain(rows + r, -1);
}

// ---------------------------------------------------------------------------
// rows to their experts
// ---------------------------------------------------------------------------
// The input is one flat sequence of 128-channel groups, as for the plain cast: eight
// lanes take a group, a lane 16 consecutive values, cast once and stored k times.  Memory
// bounds it, four bytes in five written: 8192 tokens of 4096 channels cast to 8 rows each
// in 66 to 68 us, 5.1 TB/s, 5.4 with the rows that pad 64 experts' to groups of 128 (61 us
// without those); copied as bf16 115, as codes 59.  Bulk copies in and, for each row, out of
// shared memory took 74.
// Form: what a row is and becomes.
enum GatherForm { kGatherBf16, kGatherCast, kGatherCodes };
constexpr int kGatherThreads = 256;
constexpr int kGatherWarps = kGatherThreads / 32;

struct GatherArgs {
    const uint4* x;          // [T, C] bf16, or codes
    const float* x_sf;       // [T, G], codes
    const int32_t* slots;    // [T, k]
    const int32_t* rows;     // [R]
    const int32_t* offsets;  // [E + 1]
    const float* weights;    // [T, k] or null
    uint4* out;              // [R, C]
    float* out_sf;           // [R, G]
    float* row_weights;      // [R] or null
    int64_t n_groups;        // T * G
    int G, k, E, R;
};

// Zeros in the rows that have no pair: those that pad an expert's, behind its last one; a
// cast row of zeros has the smallest scale.  kPadParts warps take an expert, each every
// kPadParts-th of its rows, looking at 32 rows at a time from the end on until none of them
// is padding.  (All rows looked at in turn, and cleared by the warp that met them, took 12
// of 73 us for 8192 tokens cast to 8 rows each of 64 experts.)
constexpr int kPadParts = 8;
template <int BYTES>
__device__ __forceinline__ void clear_padding(const int32_t* rows, const int32_t* offsets, int E, int R,
                                              int G, uint4* out, float* out_sf, float zero_scale,
                                              float* row_weights, int64_t warp, int64_t warps) {
    const int lane = threadIdx.x & 31;
    const int vecs = G * 128 * BYTES / 16;
    for (int64_t task = warp; task < static_cast<int64_t>(E) * kPadParts; task += warps) {
        const int e = static_cast<int>(task / kPadParts), part = static_cast<int>(task % kPadParts);
        int begin = ld_ro(offsets + e), end = ld_ro(offsets + e + 1);
        begin = begin < 0 ? 0 : begin;
        end = end > R ? R : end;
        for (int64_t r0 = static_cast<int64_t>(end) - 32; r0 > static_cast<int64_t>(begin) - 32; r0 -= 32) {
            const int64_t r = r0 + lane;
            const bool pad = r >= begin && ld_ro(rows + r) < 0;
            const unsigned all = __ballot_sync(kAll, pad);
            if (!all) break;
            const bool mine = pad && (r & (kPadParts - 1)) == part;
            if (mine && row_weights) st_plain(row_weights + r, 0.0f);
            for (unsigned m = __ballot_sync(kAll, mine); m; m &= m - 1) {
                const int64_t row = r0 + __ffs(m) - 1;
                for (int v = lane; v < vecs; v += 32) st_stream(out + row * vecs + v, make_uint4(0, 0, 0, 0));
                if (out_sf)
                    for (int g = lane; g < G; g += 32) st_plain(out_sf + row * G + g, zero_scale);
            }
        }
    }
}

template <int FORM, int FMT>
__global__ void __launch_bounds__(kGatherThreads, 5) gather_kernel(const GatherArgs a) {
    const int lane = threadIdx.x & 31;
    const int sub = lane >> 3, j8 = lane & 7;
    const int64_t step = static_cast<int64_t>(gridDim.x) * kGatherWarps;
    const int64_t first = static_cast<int64_t>(blockIdx.x) * kGatherWarps + (threadIdx.x >> 5);
    const int64_t units = (a.n_groups + 3) / 4;
    constexpr int kVecs = FORM == kGatherCodes ? 1 : 2;  // 16-byte vectors of a lane
    // token and group of this lane's group, advanced by the fixed stride
    int64_t t = (first * 4 + sub) / a.G;
    int g = static_cast<int>(first * 4 + sub - t * a.G);
    const int64_t dt = step * 4 / a.G;
    const int dg = static_cast<int>(step * 4 - dt * a.G);

    // a unit's values, and the slots of its tokens: lane j of a group's eight holds those of
    // experts j, j + 8, ...
    uint4 q[kVecs];
    float sf = 0.0f;
    int slot = -1;
    const auto slot_of = [&](int64_t token, int j) {
        const int s = j < a.k ? ld_ro(a.slots + token * a.k + j) : -1;
        return static_cast<unsigned>(s) < static_cast<unsigned>(a.R) ? s : -1;
    };
    const auto load = [&](int64_t u, int64_t token) {
        slot = -1;
        if (u < units && u * 4 + sub < a.n_groups) {
#pragma unroll
            for (int v = 0; v < kVecs; ++v) q[v] = ld_stream(a.x + (u * 32 + lane) * kVecs + v);
            if constexpr (FORM == kGatherCodes) sf = ld_ro(a.x_sf + u * 4 + sub);
            slot = slot_of(token, j8);
        }
    };
#pragma unroll
    for (int v = 0; v < kVecs; ++v) q[v] = make_uint4(0, 0, 0, 0);
    load(first, t);
    float zero_scale = 0.0f, inv;
    if constexpr (FORM == kGatherCast) group_scale<FMT>(0.0f, zero_scale, inv);
    clear_padding<FORM == kGatherBf16 ? 2 : 1>(a.rows, a.offsets, a.E, a.R, a.G, a.out,
                                               FORM == kGatherBf16 ? nullptr : a.out_sf, zero_scale,
                                               a.row_weights, first, step);
    for (int64_t u = first; u < units; u += step) {
        const bool live = u * 4 + sub < a.n_groups;
        const int64_t token = t;
        const int group = g;
        t += dt;
        g += dg;
        if (g >= a.G) {
            g -= a.G;
            ++t;
        }
        int slots8 = slot;
        constexpr int kOut = FORM == kGatherBf16 ? 2 : 1;
        uint4 o[kOut];
        float scale = 0.0f;
        if constexpr (FORM == kGatherCast) {
            float v[16];
            unpack8(q[0], v);
            unpack8(q[1], v + 8);
            load(u + step, t);
            float m = fmaxf(absmax8(v), absmax8(v + 8));
            m = fmaxf(m, __shfl_xor_sync(kAll, m, 1));
            m = fmaxf(m, __shfl_xor_sync(kAll, m, 2));
            m = fmaxf(m, __shfl_xor_sync(kAll, m, 4));
            float inv;
            group_scale<FMT>(m, scale, inv);
            const uint2 c0 = quantize8<FMT>(v, scale, inv), c1 = quantize8<FMT>(v + 8, scale, inv);
            o[0] = make_uint4(c0.x, c0.y, c1.x, c1.y);
        } else {
#pragma unroll
            for (int v = 0; v < kVecs; ++v) o[v] = q[v];
            scale = sf;
            load(u + step, t);
        }
        for (int j0 = 0; j0 < a.k; j0 += 8) {
            if (j0) slots8 = live ? slot_of(token, j0 + j8) : -1;
            const int most = a.k - j0 < 8 ? a.k - j0 : 8;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                if (j >= most) break;
                const int s = __shfl_sync(kAll, slots8, (lane & 24) | j);
                if (s < 0) continue;
                uint4* to = a.out + ((static_cast<int64_t>(s) * a.G + group) * 8 + j8) * kOut;
                if constexpr (kOut == 2) {
                    // whole sectors: two stores of 16 bytes took 167 us where this takes 119 (8192 x 4096, 8 each)
                    const uint32_t w[8] = {o[0].x, o[0].y, o[0].z, o[0].w, o[1].x, o[1].y, o[1].z, o[1].w};
                    st_sector(to, w);
                } else {
                    st_stream(to, o[0]);
                    if (j8 == j) st_plain(a.out_sf + static_cast<int64_t>(s) * a.G + group, scale);
                }
            }
            if (a.row_weights && group == 0 && slots8 >= 0)
                st_plain(a.row_weights + slots8, ld_ro(a.weights + token * a.k + j0 + j8));
        }
    }
}

// ---------------------------------------------------------------------------
// rows back to their tokens
// ---------------------------------------------------------------------------
// Half a warp takes 128 channels of a token, a lane eight of them, and adds up the
// token's rows in the order of its experts, so a sum repeats bit for bit.  The loads
// of up to eight rows are in flight at once: 8192 tokens of 8 rows of 4096 channels in
// 90 to 94 us, 6.4 TB/s, bound by memory; to fp32 sums 120 us, 5.6 TB/s.
constexpr int kReduceThreads = 256;
constexpr int kReduceDepth = 8;

struct ReduceArgs {
    const uint4* y;           // bf16 [R, C]
    const int32_t* slots;     // [T, k]
    const float* weights;     // [T, k] or null
    const float* row_values;  // [R] or null
    void* out;                // [T, C] bf16 or fp32
    float* values;            // [T, k]
    int64_t n_groups;         // T * G
    int G, k, R;
};

template <bool WEIGHTED, bool F32>
__global__ void __launch_bounds__(kReduceThreads) reduce_kernel(const ReduceArgs a) {
    const int l16 = threadIdx.x & 15;
    const int64_t step = static_cast<int64_t>(gridDim.x) * (kReduceThreads / 16);
    int64_t u = static_cast<int64_t>(blockIdx.x) * (kReduceThreads / 16) + (threadIdx.x >> 4);
    int64_t t = u / a.G;
    int g = static_cast<int>(u - t * a.G);
    const int64_t dt = step / a.G;
    const int dg = static_cast<int>(step - dt * a.G);
    for (; u < a.n_groups; u += step) {
        const int32_t* sl = a.slots + t * a.k;
        float acc[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) acc[i] = 0.0f;
        for (int j0 = 0; j0 < a.k; j0 += kReduceDepth) {
            uint4 q[kReduceDepth];
            float w[kReduceDepth];
#pragma unroll
            for (int j = 0; j < kReduceDepth; ++j) {
                const int s = j0 + j < a.k ? ld_ro(sl + j0 + j) : -1;
                const bool live = static_cast<unsigned>(s) < static_cast<unsigned>(a.R);
                q[j] = make_uint4(0, 0, 0, 0);
                w[j] = 0.0f;
                if (live) {
                    q[j] = ld_stream(a.y + (static_cast<int64_t>(s) * a.G + g) * 16 + l16);
                    w[j] = WEIGHTED ? ld_ro(a.weights + t * a.k + j0 + j) : 1.0f;
                }
            }
#pragma unroll
            for (int j = 0; j < kReduceDepth; ++j) {
                float v[8];
                unpack8(q[j], v);
#pragma unroll
                for (int i = 0; i < 8; ++i) acc[i] = WEIGHTED ? fmaf(w[j], v[i], acc[i]) : acc[i] + v[i];
            }
        }
        if constexpr (F32) {
            float4* o = static_cast<float4*>(a.out) + (u * 16 + l16) * 2;
            st_plain(o, make_float4(acc[0], acc[1], acc[2], acc[3]));
            st_plain(o + 1, make_float4(acc[4], acc[5], acc[6], acc[7]));
        } else {
            st_stream(static_cast<uint4*>(a.out) + u * 16 + l16, pack8_bf16(acc));
        }
        if (a.values && g == 0)
            for (int j = l16; j < a.k; j += 16) {
                const int s = ld_ro(sl + j);
                const bool live = static_cast<unsigned>(s) < static_cast<unsigned>(a.R);
                st_plain(a.values + t * a.k + j, live ? ld_ro(a.row_values + s) : 0.0f);
            }
        t += dt;
        g += dg;
        if (g >= a.G) {
            g -= a.G;
            ++t;
        }
    }
}

// ---------------------------------------------------------------------------
// gradient of the weighted sum
// ---------------------------------------------------------------------------
// A CTA takes a token, half a warp 128 of its channels at a time: dy of each of the
// token's rows is w times dout, and dw of each the sum over the channels of dout times
// the row.  A lane keeps kGradDepth of those sums while it walks its channels; they are
// added up within the warp and, in the order of the warps, within the CTA.  8192 tokens
// of 8 rows of 4096 channels: 186 us, 6.1 TB/s, bound by memory (half of it writes); with
// bf16 rows 122 registers, four CTAs an SM, hold more loads (at most 56: 192 us), with a
// cast 80, six CTAs (153: 187 us, 80: 149).
// FMT: an FP8 format, or 2 for bf16 rows.
constexpr int kGradThreads = 128;
constexpr int kGradDepth = 8;

struct GradArgs {
    const uint4* dout;        // bf16 [T, C]
    const uint4* y;           // bf16 [R, C]
    const int32_t* slots;     // [T, k]
    const int32_t* rows;      // [R]
    const int32_t* offsets;   // [E + 1]
    const float* weights;     // [T, k]
    void* dy;                 // [R, C] bf16 or codes
    float* dy_sf;             // [R, G], codes
    float* dweights;          // [T, k]
    int64_t T;
    int G, k, E, R;
};

template <int FMT>
__global__ void __launch_bounds__(kGradThreads, FMT == 2 ? 1 : 6) reduce_backward_kernel(const GradArgs a) {
    __shared__ float part[kGradThreads / 32][kGradDepth];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int half = threadIdx.x >> 4, l16 = threadIdx.x & 15;
    for (int64_t t = blockIdx.x; t < a.T; t += gridDim.x) {
        for (int j0 = 0; j0 < a.k; j0 += kGradDepth) {
            int s[kGradDepth];
            float w[kGradDepth], dot[kGradDepth];
#pragma unroll
            for (int j = 0; j < kGradDepth; ++j) {
                s[j] = -1;
                w[j] = dot[j] = 0.0f;
                if (j0 + j < a.k) {
                    s[j] = ld_ro(a.slots + t * a.k + j0 + j);
                    if (static_cast<unsigned>(s[j]) >= static_cast<unsigned>(a.R)) s[j] = -1;
                    if (s[j] >= 0) w[j] = ld_ro(a.weights + t * a.k + j0 + j);
                }
            }
            // all lanes of a warp stay in the loop: the cast's maximum is shuffled
            for (int g0 = 0; g0 < a.G; g0 += kGradThreads / 16) {
                const int g = g0 + half;
                const bool live = g < a.G;
                float d[8];
                uint4 q = make_uint4(0, 0, 0, 0);
                if (live) q = ld_stream(a.dout + (t * a.G + g) * 16 + l16);
                unpack8(q, d);
                uint4 r[kGradDepth];
#pragma unroll
                for (int j = 0; j < kGradDepth; ++j) {
                    r[j] = make_uint4(0, 0, 0, 0);
                    if (live && s[j] >= 0)
                        r[j] = ld_stream(a.y + (static_cast<int64_t>(s[j]) * a.G + g) * 16 + l16);
                }
                float m = 0.0f;
                if constexpr (FMT != 2) {
                    m = absmax8(d);
#pragma unroll
                    for (int o = 1; o < 16; o <<= 1) m = fmaxf(m, __shfl_xor_sync(kAll, m, o));
                }
#pragma unroll
                for (int j = 0; j < kGradDepth; ++j) {
                    float v[8], e[8];
                    unpack8(r[j], v);
#pragma unroll
                    for (int i = 0; i < 8; ++i) dot[j] = fmaf(d[i], v[i], dot[j]);
                    if (!live || s[j] < 0) continue;
#pragma unroll
                    for (int i = 0; i < 8; ++i) e[i] = w[j] * d[i];
                    const int64_t at = static_cast<int64_t>(s[j]) * a.G + g;
                    if constexpr (FMT == 2) {
                        st_stream(static_cast<uint4*>(a.dy) + at * 16 + l16, pack8_bf16(e));
                    } else {
                        // rounding is monotone, so the largest product is that of the largest value
                        float scale, inv;
                        group_scale<FMT>(fabsf(w[j]) * m, scale, inv);
                        st_stream(static_cast<uint2*>(a.dy) + at * 16 + l16, quantize8<FMT>(e, scale, inv));
                        if (l16 == 0) st_plain(a.dy_sf + at, scale);
                    }
                }
            }
#pragma unroll
            for (int j = 0; j < kGradDepth; ++j) {
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) dot[j] += __shfl_xor_sync(kAll, dot[j], o);
                if (lane == 0) part[warp][j] = dot[j];
            }
            __syncthreads();
            if (threadIdx.x < kGradDepth && j0 + static_cast<int>(threadIdx.x) < a.k) {
                const int64_t p = t * a.k + j0 + threadIdx.x;
                float v = 0.0f;
                // an empty slot has no gradient, whatever dout holds
                if (static_cast<unsigned>(ld_ro(a.slots + p)) < static_cast<unsigned>(a.R))
                    for (int x = 0; x < kGradThreads / 32; ++x) v += part[x][threadIdx.x];
                st_plain(a.dweights + p, v);
            }
            __syncthreads();
        }
    }
    float zero_scale = 0.0f, inv;
    if constexpr (FMT != 2) group_scale<FMT>(0.0f, zero_scale, inv);
    clear_padding<FMT == 2 ? 2 : 1>(a.rows, a.offsets, a.E, a.R, a.G, static_cast<uint4*>(a.dy),
                                    FMT == 2 ? nullptr : a.dy_sf, zero_scale, nullptr,
                                    static_cast<int64_t>(blockIdx.x) * (kGradThreads / 32) + warp,
                                    static_cast<int64_t>(gridDim.x) * (kGradThreads / 32));
}

template <typename K, typename A>
cudaError_t launch_rows(K kernel, int threads, int64_t blocks, const A& a, cudaStream_t stream) {
    const int grid = persistent_grid(reinterpret_cast<const void*>(kernel), threads, 0, blocks);
    if (const cudaError_t e = upload_checks(stream)) return e;
    kernel<<<grid, threads, 0, stream>>>(a);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_expert_order(const int32_t* ids, int32_t* slots, int32_t* rows, int32_t* offsets,
                                int64_t P, int E, int align, int64_t R, cudaStream_t stream) {
    // CTAs of the cluster: as many as leave each warp 32 pairs.  (256 experts, four times as
    // many pairs a CTA: 9.9 instead of 7.9 us for 4096 pairs, 10.6 instead of 7.7 for 8192.)
    const int64_t per_cta = kOrderWarps * 32;
    int ctas = 1;
    while (ctas < 8 && ctas * per_cta < P) ctas *= 2;
    const size_t smem = static_cast<size_t>(kOrderWarps) * E * sizeof(int);
    auto* k = ctas > 1 ? &order_kernel<true> : &order_kernel<false>;
    persistent_grid(reinterpret_cast<const void*>(k), kOrderThreads, smem, 1);  // allows the shared memory
    if (const cudaError_t e = upload_checks(stream)) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(ctas);
    cfg.blockDim = dim3(kOrderThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = ctas;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = ctas > 1 ? 1 : 0;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, k, ids, slots, rows, offsets, static_cast<int>(P), E,
                                             align, static_cast<int>(R));
    return e != cudaSuccess ? e : cudaGetLastError();
}

cudaError_t launch_expert_gather(const ExpertGather& p, cudaStream_t stream) {
    GatherArgs a = {};
    a.x = static_cast<const uint4*>(p.x);
    a.x_sf = p.x_sf;
    a.slots = p.slots;
    a.rows = p.rows;
    a.offsets = p.offsets;
    a.weights = p.weights;
    a.out = static_cast<uint4*>(p.out);
    a.out_sf = p.out_sf;
    a.row_weights = p.row_weights;
    a.G = static_cast<int>(p.C / 128);
    a.k = p.k;
    a.E = p.E;
    a.R = static_cast<int>(p.R);
    a.n_groups = p.T * a.G;
    const int64_t blocks = ((a.n_groups + 3) / 4 + kGatherWarps - 1) / kGatherWarps +
                           (p.E * kPadParts + kGatherWarps - 1) / kGatherWarps;
    if (p.form == 0) return launch_rows(&gather_kernel<kGatherBf16, kFmtE4M3>, kGatherThreads, blocks, a, stream);
    if (p.form == 2) return launch_rows(&gather_kernel<kGatherCodes, kFmtE4M3>, kGatherThreads, blocks, a, stream);
    return p.fmt == kFmtE4M3
               ? launch_rows(&gather_kernel<kGatherCast, kFmtE4M3>, kGatherThreads, blocks, a, stream)
               : launch_rows(&gather_kernel<kGatherCast, kFmtE5M2>, kGatherThreads, blocks, a, stream);
}

cudaError_t launch_expert_reduce(const void* y, const int32_t* slots, const float* weights,
                                 const float* row_values, void* out, float* values, int64_t T, int64_t C,
                                 int k, int64_t R, bool out_f32, cudaStream_t stream) {
    ReduceArgs a = {};
    a.y = static_cast<const uint4*>(y);
    a.slots = slots;
    a.weights = weights;
    a.row_values = row_values;
    a.out = out;
    a.values = values;
    a.G = static_cast<int>(C / 128);
    a.k = k;
    a.R = static_cast<int>(R);
    a.n_groups = T * a.G;
    const int64_t blocks = (a.n_groups + kReduceThreads / 16 - 1) / (kReduceThreads / 16);
    if (weights)
        return out_f32 ? launch_rows(&reduce_kernel<true, true>, kReduceThreads, blocks, a, stream)
                       : launch_rows(&reduce_kernel<true, false>, kReduceThreads, blocks, a, stream);
    return out_f32 ? launch_rows(&reduce_kernel<false, true>, kReduceThreads, blocks, a, stream)
                   : launch_rows(&reduce_kernel<false, false>, kReduceThreads, blocks, a, stream);
}

cudaError_t launch_expert_reduce_backward(const ExpertReduceGrad& p, cudaStream_t stream) {
    GradArgs a = {};
    a.dout = static_cast<const uint4*>(p.dout);
    a.y = static_cast<const uint4*>(p.y);
    a.slots = p.slots;
    a.rows = p.rows;
    a.offsets = p.offsets;
    a.weights = p.weights;
    a.dy = p.dy;
    a.dy_sf = p.dy_sf;
    a.dweights = p.dweights;
    a.T = p.T;
    a.G = static_cast<int>(p.C / 128);
    a.k = p.k;
    a.E = p.E;
    a.R = static_cast<int>(p.R);
    const int64_t pads = p.E * kPadParts / (kGradThreads / 32);
    const int64_t blocks = p.T > pads ? p.T : pads;
    if (p.fmt == kFmtE4M3)
        return launch_rows(&reduce_backward_kernel<kFmtE4M3>, kGradThreads, blocks, a, stream);
    if (p.fmt == kFmtE5M2)
        return launch_rows(&reduce_backward_kernel<kFmtE5M2>, kGradThreads, blocks, a, stream);
    return launch_rows(&reduce_backward_kernel<2>, kGradThreads, blocks, a, stream);
}

}  // namespace tkq
