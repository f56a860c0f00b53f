// residual_norm.cu -- the norms before and after a block with the block's gate
// and residual scale, fused with the per-token cast, and their gradients.
//
// Forward, for each row (h the block's output, r the residual stream, a the
// residual scale; every factor in brackets is optional):
//   p  = 1 / sqrt(mean(h^2) + eps)
//   b  = h [p] [w_post] [sigmoid(gate)]
//   r' = r + a b
//   q  = 1 / sqrt(mean(r'^2) + eps)
//   x  = r' q [w_pre]           cast per token (exact quotient) and / or bf16
// Backward, with m = h [p], n = r' q, s = sigmoid(gate), dr' and dx given:
//   dr     = dr' + q (dx w_pre - n mean(dx w_pre n))      dw_pre  = sum_t dx n
//   e      = a dr
//   dgate  = e m w_post s (1 - s)                         dw_post = sum_t e s m
//   dh     = p (e s w_post - m mean(e s w_post m)),  or e s w_post without p
//
// One CTA per row, each thread with the same channels of every row: each tensor
// is read and written once.  A thread keeps its next rows in flight as
// 16-byte asynchronous copies into its own slots of shared memory (`Fifo`), so
// loads go on across the reductions' barriers and no other thread waits for
// them.  The stream r' is rounded to its type where it is stored; the norm that
// follows is taken of the binary32 value before that rounding.
//
// Both directions are bound by memory.  8192 x 7168, bf16 stream, gate: forward
// 87 us (6.1 TB/s, 91 % of a copy's rate), backward 162 us (5.8 TB/s, 87 %; moving
// its rows with one barrier each and no arithmetic takes 149 us).
#include <type_traits>

#include <cuda_runtime.h>

#include "residual_norm.cuh"

namespace tkq {
namespace {

// ---------------------------------------------------------------------------
// forward
// ---------------------------------------------------------------------------
// Codes and scales of a thread's vectors of ROWS rows; a group is half a warp's
// vectors of one row.  The lanes of a half warp split the groups they share
// among them on the way to the maxima, as CtaSum does, so the scales of all of
// them are computed, and stored, at once; each lane then takes every group's.
template <int FMT, int ROWS, int NV>
__device__ __forceinline__ void cast_rows(const ResidualNorm& a, const SfLayout& lay, int64_t t,
                                          int vecs, const float (&v)[ROWS][NV][8]) {
    constexpr int kGroups = ROWS * NV, kLanes = 16 / kGroups;  // 1, 2 or 4 groups
    const int lane = threadIdx.x & 31, half = lane & 15;
    float m[kGroups];
#pragma unroll
    for (int g = 0; g < kGroups; ++g) m[g] = absmax8(v[g / NV][g % NV]);
    float s = m[0];
    if constexpr (kGroups == 2) {
        const bool hi = lane & 8;
        s = fmaxf(hi ? m[1] : m[0], __shfl_xor_sync(kAll, hi ? m[0] : m[1], 8));
    } else if constexpr (kGroups == 4) {
        const bool hi = lane & 8, up = lane & 4;
        const float x = fmaxf(hi ? m[2] : m[0], __shfl_xor_sync(kAll, hi ? m[0] : m[2], 8));
        const float y = fmaxf(hi ? m[3] : m[1], __shfl_xor_sync(kAll, hi ? m[1] : m[3], 8));
        s = fmaxf(up ? y : x, __shfl_xor_sync(kAll, up ? x : y, 4));
    }
#pragma unroll
    for (int o = kLanes / 2; o > 0; o >>= 1) s = fmaxf(s, __shfl_xor_sync(kAll, s, o));
    float sc, inv;
    group_scale<FMT>(s, sc, inv);
    if (lay.flags & (kSfRoundPow2 | kSfPacked)) pow2_scale(sc, inv);
    const int mine = half / kLanes;
    const int64_t row = t + mine / NV;
    const int at = threadIdx.x + mine % NV * blockDim.x;
    if (half % kLanes == 0 && row < a.T && at < vecs)
        store_scale(a.sf, lay, row, true, at / 16, sc);
#pragma unroll
    for (int g = 0; g < kGroups; ++g) {
        const int from = (lane & 16) + g * kLanes;
        const float gs = __shfl_sync(kAll, sc, from), gi = __shfl_sync(kAll, inv, from);
        const int vec = threadIdx.x + g % NV * blockDim.x;
        if (vec < vecs && t + g / NV < a.T)
            st_stream(static_cast<uint2*>(a.out) + (t + g / NV) * vecs + vec,
                      quantize8<FMT>(v[g / NV][g % NV], gs, gi));
    }
}

// Three ways to hold a row, by its width (measured at T C = 59 - 67 million,
// bf16 stream, post-norm, gate and cast):
//   up to 4096 channels   one vector a thread, 64 registers, 1024 threads an SM:
//                         4096: 101 us, 159 us with the 128 registers below (one
//                         CTA an SM); 1024: 51 us, 58 us
//   up to 8192            two vectors, 128 registers: 7168: 87 us, 95 us with one
//                         vector and 896 threads; 5120: 73 us, 76 us
//   up to 16384           two vectors, 64 registers, the weights read again for
//                         each row: 16384: 137 us, 148 us with four and 512 threads
template <int NV, bool KEPT>
constexpr int kForwardThreads = NV == 2 && KEPT ? 512 : 1024;

// ROWS consecutive rows are taken at a time, so that their reductions share the
// barriers and the shuffles, and one row's arithmetic covers the other's
// latencies.  The usual call (Mode) has a block and a pre-norm.
template <int NV, bool KEPT, bool F32, bool POST, bool GATE, int ROWS, int MODE>
__global__ void __launch_bounds__(kForwardThreads<NV, KEPT>)
    residual_norm_kernel(const ResidualNorm a, const SfLayout lay, int64_t rows_walk, int fmt,
                         Fifo q8) {
    extern __shared__ uint4 fifo[];
    __shared__ CtaSum<ROWS, kForwardThreads<NV, KEPT>> cta_sum;
    grid_dependency_launch();
    constexpr bool WHOLE = MODE != kAny, EXACT = MODE == kExact;
    constexpr int kR = F32 ? 2 : 1;   // slots of r; then h, gate
    int turn = 0;
    const int tid = threadIdx.x, vecs = static_cast<int>(a.C / 8);
    const float inv_c = 1.0f / static_cast<float>(a.C);
    const int pitch = EXACT ? vecs : NV * blockDim.x, row_size = q8.slots * pitch;
    const bool has_h = WHOLE || a.h, pre = WHOLE || a.pre;
    const auto fetch_rows = [&](int64_t t0, int stage) {
#pragma unroll
        for (int k = 0; k < ROWS; ++k) {
            if (t0 + k >= a.T) break;
            uint4* s = fifo + (stage * ROWS + k) * row_size;
            const int64_t row = (t0 + k) * vecs;
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const Place<EXACT> at(i, pitch, vecs);
                uint4* to = s + at.slot;
                if (has_h) fetch<false>(to + kR * pitch, pitch, a.h, row + at.vec);
                fetch<F32>(to, pitch, a.r, row + at.vec);
                if constexpr (GATE) fetch<false>(to + (kR + 1) * pitch, pitch, a.gate, row + at.vec);
            }
        }
        cp_async_commit();
    };
    const int64_t step = static_cast<int64_t>(gridDim.x) * ROWS;
    const int64_t start = static_cast<int64_t>(blockIdx.x) * ROWS;
    grid_dependency_wait();
    for (int d = 0; d < q8.depth - 1; ++d) fetch_rows(start + d * step, d);
    Weights<NV, KEPT> w_post, w_pre;
    w_post.template init<EXACT>(a.w_post, a.res_scale, pitch, vecs);
    w_pre.template init<EXACT>(a.w_pre, 1.0f, pitch, vecs);
    int stage = 0, ahead = q8.depth - 1;
    for (int64_t t = start; t < rows_walk; t += step) {
        fetch_rows(t + (q8.depth - 1) * step, ahead);
        if (t + ROWS > a.T)  // the padding rows of the column-major scale layouts
            for (int64_t row = t < a.T ? a.T : t; row < rows_walk && row < t + ROWS; ++row)
                for (int j = tid; j < lay.groups; j += blockDim.x)
                    store_scale(a.sf, lay, row, false, j, 0.0f);
        if (t >= a.T) continue;
        const uint4* s = fifo + stage * ROWS * row_size;
        cp_async_wait(q8.depth);
        stage = stage + 1 == q8.depth ? 0 : stage + 1;
        ahead = ahead + 1 == q8.depth ? 0 : ahead + 1;
        // a row past the last one computes on what its slots hold and stores nothing
        float v[ROWS][NV][8];
        float sum[ROWS], p[ROWS];
        if constexpr (POST) {
#pragma unroll
            for (int k = 0; k < ROWS; ++k) {
                sum[k] = 0.0f;
#pragma unroll
                for (int i = 0; i < NV; ++i) {
                    const Place<EXACT> at(i, pitch, vecs);
                    values8<false>(s + k * row_size + kR * pitch + at.slot, pitch, v[k][i]);
                    float2 c = two(0.0f);
#pragma unroll
                    for (int e = 0; e < 8; e += 2) c = fma2(at2(v[k][i], e), at2(v[k][i], e), c);
                    sum[k] += at.live ? c.x + c.y : 0.0f;
                }
            }
            cta_sum(sum, turn);
#pragma unroll
            for (int k = 0; k < ROWS; ++k) {
                p[k] = rsqrtf(sum[k] * inv_c + a.eps);
                if (tid == 0 && a.rstd_post && t + k < a.T) st_plain(a.rstd_post + t + k, p[k]);
            }
        }
#pragma unroll
        for (int k = 0; k < ROWS; ++k) {
            sum[k] = 0.0f;
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const Place<EXACT> at(i, pitch, vecs);
                float* vi = v[k][i];
                const uint4* from = s + k * row_size + at.slot;
                float r[8];
                values8<F32>(from, pitch, r);
                if (has_h) {
                    float w[8], g[8];
                    if constexpr (!POST) values8<false>(from + kR * pitch, pitch, vi);
                    if constexpr (GATE) values8<false>(from + (kR + 1) * pitch, pitch, g);
                    w_post.get(i, at.vec, w);
#pragma unroll
                    for (int e = 0; e < 8; e += 2) {
                        float2 b = mul2(at2(w, e), at2(vi, e));
                        if constexpr (GATE) {
                            float2 rest;
                            b = mul2(b, sigmoid2(at2(g, e), rest));
                        }
                        put2(vi, e, POST ? fma2(b, two(p[k]), at2(r, e)) : add2(b, at2(r, e)));
                    }
                    if (at.live && (ROWS == 1 || t + k < a.T))
                        store8<F32>(a.r_out, (t + k) * vecs + at.vec, vi);
                } else {
#pragma unroll
                    for (int e = 0; e < 8; ++e) vi[e] = r[e];
                }
                float2 c = two(0.0f);
#pragma unroll
                for (int e = 0; e < 8; e += 2) c = fma2(at2(vi, e), at2(vi, e), c);
                sum[k] += at.live ? c.x + c.y : 0.0f;
            }
        }
        if (!pre) continue;
        cta_sum(sum, turn);
#pragma unroll
        for (int k = 0; k < ROWS; ++k) {
            const bool row = ROWS == 1 || t + k < a.T;
            const float q = rsqrtf(sum[k] * inv_c + a.eps);
            if (tid == 0 && a.rstd_pre && row) st_plain(a.rstd_pre + t + k, q);
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const Place<EXACT> at(i, pitch, vecs);
                float* vi = v[k][i];
                float w[8];
                w_pre.get(i, at.vec, w);
#pragma unroll
                for (int e = 0; e < 8; e += 2) put2(vi, e, mul2(mul2(at2(vi, e), two(q)), at2(w, e)));
                if (a.x_out && row && at.live)
                    st_stream(static_cast<uint4*>(a.x_out) + (t + k) * vecs + at.vec,
                              pack8_bf16(vi));
            }
        }
        if (!a.out) continue;
        if (fmt == kFmtE4M3)
            cast_rows<kFmtE4M3>(a, lay, t, vecs, v);
        else
            cast_rows<kFmtE5M2>(a, lay, t, vecs, v);
    }
}

}  // namespace

cudaError_t launch_residual_norm(const ResidualNorm& a, int fmt, unsigned sf_flags,
                                 cudaStream_t stream) {
    SfLayout lay;
    lay.flags = sf_flags;
    lay.groups = static_cast<int>(a.C / 128);
    lay.words = (lay.groups + 3) / 4;
    lay.rows4 = (a.T + 3) / 4 * 4;
    const int64_t rows = a.out && (sf_flags & kSfColMajor) ? lay.rows4 : a.T;
    const int slots = (a.r_f32 ? 2 : 1) + (a.h ? 1 : 0) + (a.gate ? 1 : 0);
    const int nv = a.C <= 4096 ? 1 : 2;
    const bool kept = a.C <= 8192;
    const int per_sm = nv == 1 ? kForwardThreads<1, true>
                       : kept  ? kForwardThreads<2, true>
                               : kForwardThreads<2, false>;
    const Shape one = shape_of(a.C, nv, per_sm, slots, 1);
    const Shape pair = shape_of(a.C, nv, per_sm, slots, 2);
    const auto launch = [&](auto* k, const Shape& s, int rows_at_once) {
        const int grid = persistent_grid(reinterpret_cast<const void*>(k), s.threads, s.smem,
                                         (rows + rows_at_once - 1) / rows_at_once);
        if (const cudaError_t e = upload_checks(stream)) return e;
        return launch_pdl(k, grid, s.threads, s.smem, stream, true, a, lay, rows, fmt, s.fifo);
    };
    return with_options(a.r_f32, a.post, a.gate, [&](auto f32, auto post, auto gate) {
        if (!kept)
            return launch(&residual_norm_kernel<2, false, f32(), post(), gate(), 1, kAny>, one, 1);
        return with_flag(nv == 2, [&](auto wide) {
            return with_mode(a.h && a.pre, one.exact, [&](auto mode) {
                constexpr int n = wide() ? 2 : 1;
                // two rows at a time once every SM has work for that and the next two fit
                if (a.T >= 4 * int64_t{num_sms()} && pair.fifo.depth >= 2)
                    return launch(
                        &residual_norm_kernel<n, true, f32(), post(), gate(), 2, mode()>, pair, 2);
                return launch(&residual_norm_kernel<n, true, f32(), post(), gate(), 1, mode()>, one,
                              1);
            });
        });
    });
}

}  // namespace tkq
