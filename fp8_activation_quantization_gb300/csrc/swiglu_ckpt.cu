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
// 4 (bf16) or 2 out and 2 for y; scales add 1 / 32 for each cast matrix.  Both
// are bound by memory.
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
// of y.
struct RawPair {
    uint4 g[2], u[2];
    float w;

    __device__ __forceinline__ void load(const uint4* x, const float* wt, int64_t t, int j, int k,
                                         int64_t H) {
        const uint4* pg = x + t * (H / 4) + j * 16 + k * 2;
        const uint4* pu = pg + H / 8;
        g[0] = ld_stream(pg);
        g[1] = ld_stream(pg + 1);
        u[0] = ld_stream(pu);
        u[1] = ld_stream(pu + 1);
        w = wt ? ld_ro(wt + t) : 1.0f;
    }
};

// Codes of one lane's 16 values with the exact quotient, and its group's scale.
template <int FMT>
__device__ __forceinline__ uint4 cast16(const float* v, float& sc) {
    float inv;
    group_scale<FMT>(group_max(absmax16(v)), sc, inv);
    const uint2 lo = quantize8<FMT>(v, sc, inv), hi = quantize8<FMT>(v + 8, sc, inv);
    return make_uint4(lo.x, lo.y, hi.x, hi.y);
}

template <int FMT, int CKPT>
__global__ void __launch_bounds__(kThreads, 3)
    swiglu_save_kernel(const uint4* __restrict__ x, const float* __restrict__ w,
                       uint4* __restrict__ out, void* __restrict__ sf, SfLayout lay,
                       uint4* __restrict__ ckpt, float* __restrict__ ckpt_sf, int64_t H,
                       int64_t n_groups, int64_t n_walk) {
    grid_dependency_launch();
    const int lane = threadIdx.x & 31;
    const int sub = lane >> 3, k = lane & 7;
    const int GH = static_cast<int>(H / 128);
    const int64_t units = (n_walk + 3) / 4;
    const int64_t step = static_cast<int64_t>(gridDim.x) * kWarps;
    Walk cur(static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5), sub, step, GH);
    grid_dependency_wait();
    RawPair in = {};
    if (cur.u < units && cur.g < n_groups) in.load(x, w, cur.t, cur.j, k, H);
    while (cur.u < units) {
        const int64_t g = cur.g, t = cur.t;
        const int j = cur.j;
        const bool live = g < n_groups;
        float gv[16], uv[16];
        unpack8(in.g[0], gv);
        unpack8(in.g[1], gv + 8);
        unpack8(in.u[0], uv);
        unpack8(in.u[1], uv + 8);
        const float wt = in.w;
        // the next unit's loads go out before this unit's arithmetic
        cur.next(step);
        if (cur.u < units && cur.g < n_groups) in.load(x, w, cur.t, cur.j, k, H);

        float sg, su;
        const uint4 cg = cast16<CKPT>(gv, sg);
        const uint4 cu = cast16<CKPT>(uv, su);
        float v[16];
#pragma unroll
        for (int e = 0; e < 16; e += 2) {
            float2 y = swiglu2(make_float2(gv[e], gv[e + 1]), make_float2(uv[e], uv[e + 1]));
            if (w) y = mul2(y, make_float2(wt, wt));
            v[e] = y.x;
            v[e + 1] = y.y;
        }
        float sc, inv;
        group_scale<FMT>(group_max(absmax16(v)), sc, inv);
        if (lay.flags & (kSfRoundPow2 | kSfPacked)) pow2_scale(sc, inv);
        if (live) {
            const uint2 lo = quantize8_mul<FMT>(v, inv), hi = quantize8_mul<FMT>(v + 8, inv);
            st_stream(out + g * 8 + k, make_uint4(lo.x, lo.y, hi.x, hi.y));
            uint4* pc = ckpt + t * (H / 8) + j * 8 + k;
            st_stream(pc, cg);
            st_stream(pc + H / 16, cu);
        }
        if (k == 0) {
            store_scale(sf, lay, t, live, j, sc);
            if (live) {
                st_stream(ckpt_sf + t * 2 * GH + j, sg);
                st_stream(ckpt_sf + t * 2 * GH + GH + j, su);
            }
        }
    }
}

// ---------------------------------------------------------------------------
// backward
// ---------------------------------------------------------------------------
// A row belongs to `team` consecutive warps of a CTA (1, 2, 4 or 8), which take
// its units of four groups in turn, so that dw[t] is one lane's running sum,
// five shuffles and, for teams of several warps, one exchange through shared
// memory, always in the same order.
struct RestoreIn {
    uint4 g, u, d[2];
    float sg, su;

    __device__ __forceinline__ void load(const uint4* ckpt, const float* ckpt_sf, const uint4* dy,
                                         int64_t t, int j, int k, int64_t H, int GH) {
        const uint4* pg = ckpt + t * (H / 8) + j * 8 + k;
        g = ld_stream(pg);
        u = ld_stream(pg + H / 16);
        const uint4* pd = dy + t * (H / 8) + j * 16 + k * 2;
        d[0] = ld_stream(pd);
        d[1] = ld_stream(pd + 1);
        sg = ld_ro(ckpt_sf + t * 2 * GH + j);
        su = ld_ro(ckpt_sf + t * 2 * GH + GH + j);
    }
};

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

// One half of the gradients (16 values of a lane): bf16, or cast per token.
// `live`: the group holds data; `owned`: its scale is this launch's to write
// (data, or the padding rows of the column-major layouts).
template <int OUT>
__device__ __forceinline__ void store_grad(void* dx, void* dx_sf, const SfLayout& lay, int64_t t,
                                           int j, int k, bool live, bool owned, const float* v) {
    if constexpr (OUT == kBf16Out) {
        if (!live) return;
        uint4* p = static_cast<uint4*>(dx) + (t * lay.groups + j) * 16 + k * 2;
        st_stream(p, pack8_bf16(v));
        st_stream(p + 1, pack8_bf16(v + 8));
    } else {
        float sc, inv;
        group_scale<OUT>(group_max(absmax16(v)), sc, inv);
        if (lay.flags & (kSfRoundPow2 | kSfPacked)) pow2_scale(sc, inv);
        if (live) {
            const uint2 lo = quantize8_mul<OUT>(v, inv), hi = quantize8_mul<OUT>(v + 8, inv);
            st_stream(static_cast<uint4*>(dx) + (t * lay.groups + j) * 8 + k,
                      make_uint4(lo.x, lo.y, hi.x, hi.y));
        }
        if (k == 0 && owned) store_scale(dx_sf, lay, t, live, j, sc);
    }
}

template <int CKPT, int OUT>
__global__ void __launch_bounds__(kThreads, 3)
    swiglu_restore_kernel(const uint4* __restrict__ ckpt, const float* __restrict__ ckpt_sf,
                          const uint4* __restrict__ dy, const float* __restrict__ w,
                          void* __restrict__ dx, void* __restrict__ dx_sf, SfLayout lay,
                          uint4* __restrict__ y, float* __restrict__ dw, int64_t T,
                          int64_t rows_walk, int64_t H, int team) {
    __shared__ float part[kWarps];
    grid_dependency_launch();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int sub = lane >> 3, k = lane & 7;
    const int GH = static_cast<int>(H / 128);
    const int member = warp & (team - 1);      // the warp's place in its team
    const int teams = kWarps / team;           // rows a CTA takes at a time
    grid_dependency_wait();
    for (int64_t t0 = static_cast<int64_t>(blockIdx.x) * teams; t0 < rows_walk;
         t0 += static_cast<int64_t>(gridDim.x) * teams) {
        const int64_t t = t0 + warp / team;
        float dot = 0.0f;
        if (t < rows_walk) {
            const bool row = t < T;
            const float wt = w && row ? ld_ro(w + t) : 1.0f;
            for (int u0 = member * 4; u0 < GH; u0 += team * 4) {
                const int j = u0 + sub;
                const bool in_row = j < GH, live = row && in_row;
                RestoreIn in = {};
                if (live) in.load(ckpt, ckpt_sf, dy, t, j, k, H, GH);
                float gv[16], uv[16], dv[16];
                decode16<CKPT>(in.g, in.sg, gv);
                decode16<CKPT>(in.u, in.su, uv);
                unpack8(in.d[0], dv);
                unpack8(in.d[1], dv + 8);
                float yv[16];
#pragma unroll
                for (int e = 0; e < 16; e += 2) {
                    const float2 g = make_float2(gv[e], gv[e + 1]);
                    const float2 u = make_float2(uv[e], uv[e + 1]);
                    const float2 d = make_float2(dv[e], dv[e + 1]);
                    float2 dg, du;
                    swiglu_grad2(g, u, d, dg, du);
                    // d silu(g) u is du u
                    const float2 c = mul2(du, u);
                    dot += c.x + c.y;
                    if (y) {
                        float2 v = swiglu2(g, u);
                        if (w) v = mul2(v, make_float2(wt, wt));
                        yv[e] = v.x;
                        yv[e + 1] = v.y;
                    }
                    if (w) {
                        dg = mul2(dg, make_float2(wt, wt));
                        du = mul2(du, make_float2(wt, wt));
                    }
                    gv[e] = dg.x;
                    gv[e + 1] = dg.y;
                    uv[e] = du.x;
                    uv[e + 1] = du.y;
                }
                store_grad<OUT>(dx, dx_sf, lay, t, j, k, live, in_row, gv);
                store_grad<OUT>(dx, dx_sf, lay, t, GH + j, k, live, in_row, uv);
                if (y && live) {
                    uint4* py = y + t * (H / 8) + j * 16 + k * 2;
                    st_stream(py, pack8_bf16(yv));
                    st_stream(py + 1, pack8_bf16(yv + 8));
                }
            }
        }
        if (dw) {
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) dot += __shfl_xor_sync(kAll, dot, o);
            if (team > 1) {
                __syncthreads();  // the sums of the rows before have been read
                if (lane == 0) part[warp] = dot;
                __syncthreads();
                dot = 0.0f;
                for (int i = 0; i < team; ++i) dot += part[warp - member + i];
            }
            if (lane == 0 && member == 0 && t < T) st_plain(dw + t, dot);
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
    return with_fmt(fmt, [&](auto f) {
        return with_fmt(ckpt_fmt, [&](auto c) {
            auto* k = &swiglu_save_kernel<decltype(f)::value, decltype(c)::value>;
            const int grid = persistent_grid(reinterpret_cast<const void*>(k), kThreads, 0,
                                             ((n_walk + 3) / 4 + kWarps - 1) / kWarps);
            if (const cudaError_t e = upload_checks(stream)) return e;
            return launch_pdl(k, grid, kThreads, 0, stream, true, static_cast<const uint4*>(x), w,
                              static_cast<uint4*>(out), sf, lay, static_cast<uint4*>(ckpt),
                              ckpt_sf, H, n_groups, n_walk);
        });
    });
}

cudaError_t launch_swiglu_restore(const void* ckpt, const float* ckpt_sf, const void* dy,
                                  const float* w, void* dx, void* dx_sf, void* y, float* dw,
                                  int64_t T, int64_t H, int ckpt_fmt, int out_kind,
                                  unsigned sf_flags, cudaStream_t stream) {
    const SfLayout lay = layout_of(sf_flags, T, 2 * (H / 128));
    const int64_t rows = out_kind != kBf16Out && (sf_flags & kSfColMajor) ? lay.rows4 : T;
    auto go = [&](auto c, auto o) {
        auto* k = &swiglu_restore_kernel<decltype(c)::value, decltype(o)::value>;
        // as many warps a row as it takes to give every SM some, up to its units
        const int64_t units = (H / 128 + 3) / 4;
        int team = 1;
        while (team < kWarps && team < units && rows * team < int64_t{num_sms()} * 3 * kWarps)
            team *= 2;
        const int grid = persistent_grid(reinterpret_cast<const void*>(k), kThreads, 0,
                                         (rows * team + kWarps - 1) / kWarps);
        if (const cudaError_t e = upload_checks(stream)) return e;
        return launch_pdl(k, grid, kThreads, 0, stream, true, static_cast<const uint4*>(ckpt),
                          ckpt_sf, static_cast<const uint4*>(dy), w, dx, dx_sf, lay,
                          static_cast<uint4*>(y), dw, T, rows, H, team);
    };
    return with_fmt(ckpt_fmt, [&](auto c) {
        if (out_kind == kBf16Out) return go(c, std::integral_constant<int, kBf16Out>());
        return with_fmt(out_kind, [&](auto o) { return go(c, o); });
    });
}

}  // namespace tkq
