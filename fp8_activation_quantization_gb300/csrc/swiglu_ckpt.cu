// swiglu_ckpt.cu -- the SwiGLU with an 8-bit checkpoint of its input, and its
// backward from that checkpoint.
//
// Forward: one read of the bf16 [T, 2H] gate|up matrix gives
//   y = silu(g) * u [* w]  cast per token (codes, scales: swiglu_flat.cu), and
//   the checkpoint, the per-token cast of [g | u] itself (exact quotients:
//   bit for bit what token_cast.cu writes for the same matrix).
// Backward, with g, u = code * scale in binary32, d = dy, s = 1 / (1 + exp(-g)):
//   dg = d u s (1 + g (1 - s)) [w]      du = d g s [w]
//   dw[t] = sum_c d g s u               y  = g s u [w]
// The gradients leave as bf16 or cast per token; dw is the gradient of the
// routing weight and y the forward's output again, for the weight gradient of
// the product that follows.
//
// Bytes for each element of y: forward 4 in, 1 + 2 out; backward 2 + 2 in,
// 4 (bf16) or 2 out and 2 for y; scales add 1 / 32 for each cast matrix.
// Measured at 65536 x 2048: forward 156 us (6.1 TB/s, 91 % of a copy's rate);
// backward with FP8 gradients, dw and y 185 us (5.9 TB/s, 88 %), where the ALU
// pipe (conversions, maxima) is as busy as memory; with bf16 gradients and dw 187 us
// (87 %), with y too 254 us (79 %).  Each thread has the registers that its CTAs an
// SM leave it (64 and 80), for which the forward spills one to three values, the
// backward with y two to eight.
#include <type_traits>

#include <cuda_runtime.h>

#include "tkq_device.cuh"
#include "tkq_flat.cuh"
#include "tkq_internal.h"

namespace tkq {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr unsigned kAll = 0xffffffffu;
constexpr int kBf16Out = 2;  // in the place of an FP8 format: the gradients leave as bf16
// Units in flight, the current one among them.  Backward, 65536 x 2048: bf16
// gradients 201 us with two, 186 us with three; FP8 gradients and y 186 us with
// two, 196 us with three; four are no better for either.
constexpr int kSaveDepth = 3;
template <int OUT>
constexpr int kRestoreDepth = OUT == kBf16Out ? 3 : 2;

// Largest value of the eight lanes that share a group.
__device__ __forceinline__ float group_max(float m) {
    m = fmaxf(m, __shfl_xor_sync(kAll, m, 1));
    m = fmaxf(m, __shfl_xor_sync(kAll, m, 2));
    return fmaxf(m, __shfl_xor_sync(kAll, m, 4));
}
__device__ __forceinline__ float absmax16(const float* v) {
    return fmaxf(absmax8(v), absmax8(v + 8));
}

// ---------------------------------------------------------------------------
// forward
// ---------------------------------------------------------------------------
// The flat stream of swiglu_flat.cu: a warp takes units of four groups of y
// (lane l: 16 channels of group 4u + l / 8) and reads the 32-byte runs of
// gate and up; the same registers give the two checkpoint groups and the group
// of y.  The next two units are in flight as asynchronous copies into shared
// memory (`Run`), which costs no registers: 64 a thread, four CTAs an SM, 156 us
// at 65536 x 2048; with the next unit's loads in registers and three CTAs 168 us.

// Scales of two groups (a gate's and an up's) that eight lanes share: lanes
// 0 - 3 end with the first one's maximum, 4 - 7 with the second's, so one scale
// is computed for both; a lane then takes both from its two halves.
template <int FMT>
struct TwoScales {
    float sc, inv;  // this lane's half's

    __device__ __forceinline__ TwoScales(float m0, float m1, int k, bool pow2) {
        const bool hi = k & 4;
        float m = fmaxf(hi ? m1 : m0, __shfl_xor_sync(kAll, hi ? m0 : m1, 4));
        m = fmaxf(m, __shfl_xor_sync(kAll, m, 1));
        m = fmaxf(m, __shfl_xor_sync(kAll, m, 2));
        group_scale<FMT>(m, sc, inv);
        if (pow2) pow2_scale(sc, inv);
    }
    static __device__ __forceinline__ float of(float mine, int lane, int which) {
        return __shfl_sync(kAll, mine, (lane & ~7) + 4 * which);
    }
};

// Codes of one lane's 16 values with the exact quotient.
template <int FMT>
__device__ __forceinline__ uint4 codes16(const float* v, float sc, float inv) {
    const uint2 lo = quantize8<FMT>(v, sc, inv), hi = quantize8<FMT>(v + 8, sc, inv);
    return make_uint4(lo.x, lo.y, hi.x, hi.y);
}
// Codes of the products by the rounded reciprocal.
template <int FMT>
__device__ __forceinline__ uint4 codes16_mul(const float* v, float inv) {
    const uint2 lo = quantize8_mul<FMT>(v, inv), hi = quantize8_mul<FMT>(v + 8, inv);
    return make_uint4(lo.x, lo.y, hi.x, hi.y);
}

// A bf16 run of a group is 16 vectors of 8 channels, of which lane k of the
// group computes on vectors 2k and 2k + 1.  It is copied in the coalesced order
// (lane k: vectors k and k + 8) and stored with the halves interleaved, vector
// v at v ^ (v >> 3), so that neither the copies nor the reads of a quarter warp
// meet in a bank.  The warp's lanes exchange vectors, hence the __syncwarp
// between a wait and the reads; the same one lets the slots read an iteration
// ago be overwritten.
template <int DEPTH>
struct Run {
    uint4 vec[DEPTH][kThreads * 2];

    __device__ __forceinline__ void copy(int stage, int tid, const uint4* run) {
        const int k = tid & 7;
        uint4* v = vec[stage] + (tid >> 3) * 16;
        cp_async16(v + k, run + k);
        cp_async16(v + ((k + 8) ^ 1), run + k + 8);
    }
    __device__ __forceinline__ void read(int stage, int tid, float* out) const {
        const int k = tid & 7, at = 2 * k ^ (k >> 2);
        const uint4* v = vec[stage] + (tid >> 3) * 16;
        unpack8(v[at], out);
        unpack8(v[at ^ 1], out + 8);
    }
};

struct SaveSlots {
    Run<kSaveDepth> g, u;
    float w[kSaveDepth][kThreads];
};

// SFX: a scale layout other than row-major fp32.
template <int FMT, int CKPT, bool SFX>
__global__ void __launch_bounds__(kThreads, 4)
    swiglu_save_kernel(const uint4* __restrict__ x, const float* __restrict__ w,
                       uint4* __restrict__ out, void* __restrict__ sf, SfLayout lay,
                       uint4* __restrict__ ckpt, float* __restrict__ ckpt_sf, int64_t H,
                       int64_t n_groups, int64_t n_walk) {
    extern __shared__ char shared[];
    SaveSlots& slots = *reinterpret_cast<SaveSlots*>(shared);
    grid_dependency_launch();
    const int tid = threadIdx.x, lane = tid & 31;
    const int sub = lane >> 3, k = lane & 7;
    const int GH = static_cast<int>(H / 128);
    const int64_t units = (n_walk + 3) / 4;
    const int64_t step = static_cast<int64_t>(gridDim.x) * kWarps;
    Walk cur(static_cast<int64_t>(blockIdx.x) * kWarps + (tid >> 5), sub, step, GH);
    Walk next = cur;
    const auto fetch = [&](int stage) {
        if (next.u < units && next.g < n_groups) {
            const uint4* pg = x + next.t * (H / 4) + next.j * 16;
            slots.g.copy(stage, tid, pg);
            slots.u.copy(stage, tid, pg + H / 8);
            if (w) cp_async4(&slots.w[stage][tid], w + next.t);
        }
        cp_async_commit();
        next.next(step);
    };
    grid_dependency_wait();
    for (int d = 0; d < kSaveDepth - 1; ++d) fetch(d);
    int stage = 0, ahead = kSaveDepth - 1;
    while (cur.u < units) {
        cp_async_wait(kSaveDepth - 1);
        __syncwarp();
        fetch(ahead);
        const int64_t g = cur.g, t = cur.t;
        const int j = cur.j;
        const bool live = g < n_groups;
        float gv[16], uv[16];
        slots.g.read(stage, tid, gv);
        slots.u.read(stage, tid, uv);
        const float wt = w ? slots.w[stage][tid] : 1.0f;
        stage = stage + 1 == kSaveDepth ? 0 : stage + 1;
        ahead = ahead + 1 == kSaveDepth ? 0 : ahead + 1;
        cur.next(step);

        uint4* pc = ckpt + t * (H / 8) + j * 8 + k;
        const TwoScales<CKPT> own(absmax16(gv), absmax16(uv), k, false);
        const uint4 cg = codes16<CKPT>(gv, own.of(own.sc, lane, 0), own.of(own.inv, lane, 0));
        if (live) st_stream(pc, cg);
        const uint4 cu = codes16<CKPT>(uv, own.of(own.sc, lane, 1), own.of(own.inv, lane, 1));
        if (live) st_stream(pc + H / 16, cu);
        if (live && (k & 3) == 0) st_stream(ckpt_sf + t * 2 * GH + j + (k ? GH : 0), own.sc);
#pragma unroll
        for (int e = 0; e < 16; e += 2) {
            // the product by 1 of a row without a weight changes nothing
            const float2 y = mul2(swiglu2(make_float2(gv[e], gv[e + 1]), make_float2(uv[e], uv[e + 1])),
                                  make_float2(wt, wt));
            gv[e] = y.x;
            gv[e + 1] = y.y;
        }
        float sc, inv;
        group_scale<FMT>(group_max(absmax16(gv)), sc, inv);
        if (SFX && (lay.flags & (kSfRoundPow2 | kSfPacked))) pow2_scale(sc, inv);
        if (live) st_stream(out + g * 8 + k, codes16_mul<FMT>(gv, inv));
        if (k == 0) {
            if constexpr (SFX)
                store_scale(sf, lay, t, live, j, sc);
            else if (live)
                st_stream(static_cast<float*>(sf) + g, sc);
        }
    }
}

// ---------------------------------------------------------------------------
// backward
// ---------------------------------------------------------------------------
// A row belongs to `team` consecutive warps of a CTA (1, 2, 4 or 8), which take
// its units of four groups in turn, so that dw[t] is one lane's running sum,
// five shuffles and, for teams of several warps, one exchange through shared
// memory, always in the same order.  Rows of one or two groups go four or two
// (`pack`) to a warp, so that its lanes are filled.
template <int CKPT>
__device__ __forceinline__ void decode16(const uint4& q, float s, float* v) {
    decode4<CKPT>(q.x, v);
    decode4<CKPT>(q.y, v + 4);
    decode4<CKPT>(q.z, v + 8);
    decode4<CKPT>(q.w, v + 12);
#pragma unroll
    for (int e = 0; e < 16; e += 2) {
        const float2 r = mul2(make_float2(v[e], v[e + 1]), make_float2(s, s));
        v[e] = r.x;
        v[e + 1] = r.y;
    }
}

// silu(g) and its slope s (1 + g (1 - s)) = s + silu(g) (1 - s) for two values.
// 1 - s is taken as it stands: it is exact for g << 0, and for g > 0 its
// rounding adds at most |g| u to a slope near 1.
__device__ __forceinline__ void silu_and_slope2(float2 g, float2& silu, float2& slope) {
    const float2 t = mul2(g, make_float2(-1.4426950408889634f, -1.4426950408889634f));
    const float2 den = add2(make_float2(1.0f, 1.0f), make_float2(ex2_approx(t.x), ex2_approx(t.y)));
    const float2 s = make_float2(rcp_approx(den.x), rcp_approx(den.y));
    silu = mul2(g, s);
    const float2 rest = fma2(s, make_float2(-1.0f, -1.0f), make_float2(1.0f, 1.0f));
    slope = fma2(silu, rest, s);
}

// One lane's place in its warp's walk: row t and first block u0 of the unit.
struct RowWalk {
    int64_t t;
    int u0;
    __device__ __forceinline__ void next(int member, int team, int GH, int64_t rows) {
        u0 += team * 4;
        if (u0 >= GH) {
            u0 = member * 4;
            t += rows;
        }
    }
};

template <int DEPTH>
struct RestoreSlots {
    uint4 code[DEPTH][2][kThreads];  // a lane's own codes and scales of g and u
    float scale[DEPTH][2][kThreads];
    Run<DEPTH> dy;
};

template <int CKPT, int OUT, bool Y, bool SFX>
__global__ void __launch_bounds__(kThreads, 3)
    swiglu_restore_kernel(const uint4* __restrict__ ckpt, const float* __restrict__ ckpt_sf,
                          const uint4* __restrict__ dy, const float* __restrict__ w,
                          void* __restrict__ dx, void* __restrict__ dx_sf, SfLayout lay,
                          uint4* __restrict__ y, float* __restrict__ dw, int64_t T,
                          int64_t rows_walk, int64_t H, int team) {
    extern __shared__ char shared[];
    constexpr int kDepth = kRestoreDepth<OUT>;
    auto& slots = *reinterpret_cast<RestoreSlots<kDepth>*>(shared);
    __shared__ float part[kWarps];
    grid_dependency_launch();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int sub = lane >> 3, k = lane & 7;
    const int GH = static_cast<int>(H / 128);
    const int member = warp & (team - 1);      // the warp's place in its team
    const int teams = kWarps / team;           // (packs of) rows a CTA takes at a time
    const int pack = GH == 1 ? 4 : GH == 2 ? 2 : 1;
    const int j0 = pack > 1 ? sub % GH : sub;     // the lane's group in a unit,
    const int in_pack = pack > 1 ? sub / GH : 0;  // its row in a pack
    const int64_t step = static_cast<int64_t>(gridDim.x) * teams;
    // units of the rows that hold data; a member of a team that is larger than
    // the row's units has none
    const int64_t first = (static_cast<int64_t>(blockIdx.x) * teams + warp / team) * pack + in_pack;
    RowWalk ahead = {first, member * 4};
    if (ahead.u0 >= GH) ahead.t = T;
    const auto fetch = [&](int stage) {
        const int j = ahead.u0 + j0;
        if (ahead.t < T && j < GH) {
            // a row of codes, and one of dy, is H / 8 pieces, one of scales H / 64
            const int64_t row = ahead.t * (H / 8);
            const uint4* pg = ckpt + row + (j * 8 + k);
            cp_async16(&slots.code[stage][0][tid], pg);
            cp_async16(&slots.code[stage][1][tid], pg + H / 16);
            slots.dy.copy(stage, tid, dy + row + j * 16);
            const float* ps = ckpt_sf + (row >> 3) + j;
            cp_async4(&slots.scale[stage][0][tid], ps);
            cp_async4(&slots.scale[stage][1][tid], ps + GH);
        }
        cp_async_commit();
        ahead.next(member, team, GH, step * pack);
    };
    grid_dependency_wait();
    for (int d = 0; d < kDepth - 1; ++d) fetch(d);
    int stage = 0, free_stage = kDepth - 1;
    const auto weight = [&](int64_t t) { return w && t < T ? ld_ro(w + t) : 1.0f; };
    float w_next = weight(first);
    int64_t t = first;
    for (int64_t t0 = static_cast<int64_t>(blockIdx.x) * teams * pack; t0 < rows_walk;
         t0 += step * pack, t += step * pack) {
        const float wt = w_next;
        w_next = weight(t + step * pack);
        const bool row = t < T;
        float2 dot = make_float2(0.0f, 0.0f);
        // the row's first piece of codes (and of y), and of bf16 gradients
        const int64_t row_at = t * (H / 8);
        for (int u0 = member * 4; u0 < GH; u0 += team * 4) {
            cp_async_wait(kDepth - 1);
            __syncwarp();
            fetch(free_stage);
            const int j = u0 + j0;
            const bool in_row = j < GH && t < rows_walk, live = row && j < GH;
            // a group without data computes on what its slots hold; nothing of it is used
            float gv[16], uv[16], dv[16];
            decode16<CKPT>(slots.code[stage][0][tid], slots.scale[stage][0][tid], gv);
            decode16<CKPT>(slots.code[stage][1][tid], slots.scale[stage][1][tid], uv);
            slots.dy.read(stage, tid, dv);
            stage = stage + 1 == kDepth ? 0 : stage + 1;
            free_stage = free_stage + 1 == kDepth ? 0 : free_stage + 1;
            float2 unit_dot = make_float2(0.0f, 0.0f);
            [[maybe_unused]] uint32_t yv[8];
#pragma unroll
            for (int e = 0; e < 16; e += 2) {
                const float2 g = make_float2(gv[e], gv[e + 1]);
                const float2 u = make_float2(uv[e], uv[e + 1]);
                const float2 d = make_float2(dv[e], dv[e + 1]);
                const float2 wd = mul2(d, make_float2(wt, wt));
                float2 silu, slope;
                silu_and_slope2(g, silu, slope);
                const float2 s = mul2(silu, u);
                unit_dot = fma2(d, s, unit_dot);
                const float2 dg = mul2(mul2(wd, u), slope), du = mul2(wd, silu);
                gv[e] = dg.x;
                gv[e + 1] = dg.y;
                uv[e] = du.x;
                uv[e + 1] = du.y;
                if constexpr (Y) {
                    const float2 v = mul2(s, make_float2(wt, wt));
                    yv[e / 2] = pack_bf16x2(v.x, v.y);
                }
            }
            if (live) dot = add2(dot, unit_dot);
            if constexpr (Y) {
                if (live) {
                    uint4* py = y + row_at + (j * 16 + k * 2);
                    st_stream(py, make_uint4(yv[0], yv[1], yv[2], yv[3]));
                    st_stream(py + 1, make_uint4(yv[4], yv[5], yv[6], yv[7]));
                }
            }
            if constexpr (OUT == kBf16Out) {
                if (live) {
                    uint4* p = static_cast<uint4*>(dx) + 2 * row_at + (j * 16 + k * 2);
                    st_stream(p, pack8_bf16(gv));
                    st_stream(p + 1, pack8_bf16(gv + 8));
                    st_stream(p + H / 8, pack8_bf16(uv));
                    st_stream(p + H / 8 + 1, pack8_bf16(uv + 8));
                }
            } else {
                const TwoScales<OUT> two(absmax16(gv), absmax16(uv), k,
                                         SFX && (lay.flags & (kSfRoundPow2 | kSfPacked)));
                const uint4 cg = codes16_mul<OUT>(gv, two.of(two.inv, lane, 0));
                const uint4 cu = codes16_mul<OUT>(uv, two.of(two.inv, lane, 1));
                if (live) {
                    uint4* p = static_cast<uint4*>(dx) + row_at + (j * 8 + k);
                    st_stream(p, cg);
                    st_stream(p + H / 16, cu);
                }
                if ((k & 3) == 0 && in_row) {
                    const int group = j + (k ? GH : 0);
                    if constexpr (SFX)
                        store_scale(dx_sf, lay, t, live, group, two.sc);
                    else if (live)
                        st_stream(static_cast<float*>(dx_sf) + (row_at >> 3) + group, two.sc);
                }
            }
        }
        if (dw) {
            float sum = dot.x + dot.y;
            for (int o = 16 / pack; o > 0; o >>= 1) sum += __shfl_xor_sync(kAll, sum, o);
            if (team > 1) {
                __syncthreads();  // the sums of the rows before have been read
                if (lane == 0) part[warp] = sum;
                __syncthreads();
                sum = 0.0f;
                for (int i = 0; i < team; ++i) sum += part[warp - member + i];
            }
            if (lane % (32 / pack) == 0 && member == 0 && row) st_plain(dw + t, sum);
        }
    }
}

SfLayout layout_of(unsigned flags, int64_t T, int64_t groups) {
    SfLayout lay;
    lay.flags = flags;
    lay.groups = static_cast<int>(groups);
    lay.words = (lay.groups + 3) / 4;
    lay.rows4 = (T + 3) / 4 * 4;
    return lay;
}

template <typename F>
cudaError_t with_fmt(int fmt, F&& f) {
    if (fmt == kFmtE4M3) return f(std::integral_constant<int, kFmtE4M3>());
    return f(std::integral_constant<int, kFmtE5M2>());
}

}  // namespace

cudaError_t launch_swiglu_save(const void* x, const float* w, void* out, void* sf, void* ckpt,
                               float* ckpt_sf, int64_t T, int64_t H, int fmt, int ckpt_fmt,
                               unsigned sf_flags, cudaStream_t stream) {
    const SfLayout lay = layout_of(sf_flags, T, H / 128);
    const int64_t n_groups = T * lay.groups;
    const int64_t n_walk = (sf_flags & kSfColMajor) ? lay.rows4 * lay.groups : n_groups;
    const auto launch = [&](auto* k) {
        const int grid = persistent_grid(reinterpret_cast<const void*>(k), kThreads,
                                         sizeof(SaveSlots), ((n_walk + 3) / 4 + kWarps - 1) / kWarps);
        if (const cudaError_t e = upload_checks(stream)) return e;
        return launch_pdl(k, grid, kThreads, sizeof(SaveSlots), stream, true,
                          static_cast<const uint4*>(x), w, static_cast<uint4*>(out), sf, lay,
                          static_cast<uint4*>(ckpt), ckpt_sf, H, n_groups, n_walk);
    };
    return with_fmt(fmt, [&](auto f) {
        return with_fmt(ckpt_fmt, [&](auto c) {
            return sf_flags & ~kQReciprocal ? launch(&swiglu_save_kernel<f(), c(), true>)
                                            : launch(&swiglu_save_kernel<f(), c(), false>);
        });
    });
}

cudaError_t launch_swiglu_restore(const void* ckpt, const float* ckpt_sf, const void* dy,
                                  const float* w, void* dx, void* dx_sf, void* y, float* dw,
                                  int64_t T, int64_t H, int ckpt_fmt, int out_kind,
                                  unsigned sf_flags, cudaStream_t stream) {
    const SfLayout lay = layout_of(sf_flags, T, 2 * (H / 128));
    const int64_t rows = out_kind != kBf16Out && (sf_flags & kSfColMajor) ? lay.rows4 : T;
    // as many warps a row as it takes to give every SM some, up to its units
    const int64_t units = (H / 128 + 3) / 4;
    const int64_t packs = H == 128 ? (rows + 3) / 4 : H == 256 ? (rows + 1) / 2 : rows;
    int team = 1;
    while (team < kWarps && team < units && rows * team < int64_t{num_sms()} * 3 * kWarps) team *= 2;
    const auto launch = [&](auto* k, size_t smem) {
        const int grid = persistent_grid(reinterpret_cast<const void*>(k), kThreads, smem,
                                         (packs * team + kWarps - 1) / kWarps);
        if (const cudaError_t e = upload_checks(stream)) return e;
        return launch_pdl(k, grid, kThreads, smem, stream, true,
                          static_cast<const uint4*>(ckpt), ckpt_sf, static_cast<const uint4*>(dy),
                          w, dx, dx_sf, lay, static_cast<uint4*>(y), dw, T, rows, H, team);
    };
    const auto go = [&](auto c, auto o) {
        constexpr size_t smem = sizeof(RestoreSlots<kRestoreDepth<o()>>);
        if constexpr (o() != kBf16Out)
            if (sf_flags & ~kQReciprocal)
                return y ? launch(&swiglu_restore_kernel<c(), o(), true, true>, smem)
                         : launch(&swiglu_restore_kernel<c(), o(), false, true>, smem);
        return y ? launch(&swiglu_restore_kernel<c(), o(), true, false>, smem)
                 : launch(&swiglu_restore_kernel<c(), o(), false, false>, smem);
    };
    return with_fmt(ckpt_fmt, [&](auto c) {
        if (out_kind == kBf16Out) return go(c, std::integral_constant<int, kBf16Out>());
        return with_fmt(out_kind, [&](auto o) { return go(c, o); });
    });
}

}  // namespace tkq
