// residual_norm_backward.cu -- the gradients of residual_norm.cu (formulas there).
#include <type_traits>

#include <cuda_runtime.h>

#include "residual_norm.cuh"

namespace tkq {
namespace {

// ---------------------------------------------------------------------------
// backward
// ---------------------------------------------------------------------------
// One reduction a row.  With G = dr' + q dx w_pre, so that dr = G - q^2 m1 r'
// for the first mean m1 = S1 / C, and f = a w_post s, the sum that dh needs is
// linear in m1 and follows from sums over what the row brings along:
//   S1 = q sum dx w_pre r',  S2 = p sum f h G,  S3 = p sum f h r':
//   sum e w_post s m = S2 - q^2 m1 S3.
// G and r' stay in registers between the two passes (up to two vectors a
// thread), h and the gate are read from shared memory again.  The weight
// gradients are summed over a CTA's rows in registers and written as one
// partial row a CTA; sum_parts_kernel adds them up in order.
// The usual call (Mode) gives dr', dx and h.
//
// How a row is held, by its width (16 bytes a channel; measured at T C = 59 - 67
// million, bf16 stream, gate):
//   up to 4096 channels   one vector a thread, 512 threads of 128 registers:
//                         4096: 171 us, 278 us with the 72 registers below;
//                         2048: 165 us, 227 us
//   up to 7168, whole     one vector, 896 threads of 72 registers: 7168: 162 us,
//   warps, bf16 stream    174 us with two vectors and 448 threads of 128 registers;
//                         an fp32 stream needs more: 337 us, 241 us
//   up to 8192            two vectors, 512 threads of 128 registers
//   up to 16384           four, the stream and the weights not kept
struct BackwardKind {
    int nv, threads;
};
constexpr BackwardKind kNarrow = {1, 512}, kMiddle = {1, 896}, kWide = {2, 512}, kWidest = {4, 512};
template <int NV, int THREADS, bool F32, bool POST, bool GATE, int MODE>
__global__ void __launch_bounds__(THREADS)
    residual_norm_backward_kernel(const ResidualNormGrad a, Fifo q8) {
    extern __shared__ uint4 fifo[];
    __shared__ CtaSum<POST ? 3 : 1, THREADS> cta_sum;
    grid_dependency_launch();
    constexpr bool WHOLE = MODE != kAny, EXACT = MODE == kExact;
    constexpr int kS = F32 ? 2 : 1;   // slots of a stream: h, gate, dr, dx, r
    constexpr bool kKept = NV <= 2;
    const bool has_dr = WHOLE || a.dr, has_dx = WHOLE || a.dx, has_h = WHOLE || a.h;
    int turn = 0;
    const int tid = threadIdx.x, vecs = static_cast<int>(a.C / 8);
    const int pitch = EXACT ? vecs : NV * blockDim.x;
    const int at_gate = pitch;
    const int at_dr = ((has_h ? 1 : 0) + (GATE ? 1 : 0)) * pitch;
    const int at_dx = at_dr + (has_dr ? kS : 0) * pitch;
    const int at_r = at_dx + pitch;
    const float inv_c = 1.0f / static_cast<float>(a.C);
    const int stage_size = q8.slots * pitch;
    const auto fetch_row = [&](int64_t t, int stage) {
        if (t < a.T)
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const Place<EXACT> place(i, pitch, vecs);
                uint4* s = fifo + stage * stage_size + place.slot;
                const int64_t at = t * vecs + place.vec;
                if (has_dr) fetch<F32>(s + at_dr, pitch, a.dr, at);
                if (has_dx) {
                    fetch<false>(s + at_dx, pitch, a.dx, at);
                    fetch<F32>(s + at_r, pitch, a.r, at);
                }
                if (has_h) fetch<false>(s, pitch, a.h, at);
                if constexpr (GATE) fetch<false>(s + at_gate, pitch, a.gate, at);
            }
        cp_async_commit();
    };
    // dr', dx and r' of one vector, zeros for what is absent
    const auto stream = [&](const uint4* s, float* g, float* d, float* r) {
#pragma unroll
        for (int e = 0; e < 8; ++e) g[e] = d[e] = r[e] = 0.0f;
        if (has_dr) values8<F32>(s + at_dr, pitch, g);
        if (has_dx) {
            values8<false>(s + at_dx, pitch, d);
            values8<F32>(s + at_r, pitch, r);
        }
    };
    float acc_pre[NV][8] = {}, acc_post[NV][8] = {};
    grid_dependency_wait();
    for (int d = 0; d < q8.depth - 1; ++d)
        fetch_row(blockIdx.x + static_cast<int64_t>(d) * gridDim.x, d);
    Weights<NV, kKept> w_post, w_pre;
    w_post.template init<EXACT>(a.w_post, a.res_scale, pitch, vecs);
    w_pre.template init<EXACT>(a.w_pre, 1.0f, pitch, vecs);
    float p_next = 1.0f, q_next = 0.0f;
    const auto load_factors = [&](int64_t t) {
        if (POST && t < a.T) p_next = ld_ro(a.rstd_post + t);
        if (has_dx && t < a.T) q_next = ld_ro(a.rstd_pre + t);
    };
    load_factors(blockIdx.x);
    int stage = 0, ahead = q8.depth - 1;
    for (int64_t t = blockIdx.x; t < a.T; t += gridDim.x) {
        fetch_row(t + static_cast<int64_t>(q8.depth - 1) * gridDim.x, ahead);
        // the row's factors were loaded a row ago
        const float p = p_next, q = q_next;
        load_factors(t + gridDim.x);
        const uint4* s = fifo + stage * stage_size;
        cp_async_wait(q8.depth);
        stage = stage + 1 == q8.depth ? 0 : stage + 1;
        ahead = ahead + 1 == q8.depth ? 0 : ahead + 1;
        float g[kKept ? NV : 1][8], r[kKept ? NV : 1][8];
        float sum[POST ? 3 : 1] = {};
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const Place<EXACT> place(i, pitch, vecs);
            float* gi = g[kKept ? i : 0];
            float* ri = r[kKept ? i : 0];
            float d[8], w[8];
            stream(s + place.slot, gi, d, ri);
            float2 s1 = two(0.0f);
            if (has_dx) {
                w_pre.get(i, place.vec, w);
#pragma unroll
                for (int e = 0; e < 8; e += 2) {
                    const float2 dq = mul2(at2(d, e), two(q));
                    put2(acc_pre[i], e, fma2(dq, at2(ri, e), at2(acc_pre[i], e)));
                    const float2 dw = mul2(dq, at2(w, e));
                    s1 = fma2(dw, at2(ri, e), s1);
                    put2(gi, e, add2(dw, at2(gi, e)));
                }
            }
            sum[0] += place.live ? s1.x + s1.y : 0.0f;
            if constexpr (POST) {
                float2 s2 = two(0.0f), s3 = s2;
                float h[8], gt[8];
                values8<false>(s + place.slot, pitch, h);
                if constexpr (GATE) values8<false>(s + place.slot + at_gate, pitch, gt);
                w_post.get(i, place.vec, w);
#pragma unroll
                for (int e = 0; e < 8; e += 2) {
                    float2 f = mul2(at2(w, e), at2(h, e));
                    float2 rest;
                    if constexpr (GATE) f = mul2(f, sigmoid2(at2(gt, e), rest));
                    s2 = fma2(f, at2(gi, e), s2);
                    s3 = fma2(f, at2(ri, e), s3);
                }
                sum[1] += place.live ? s2.x + s2.y : 0.0f;
                sum[2] += place.live ? s3.x + s3.y : 0.0f;
            }
        }
        if (POST || has_dx) cta_sum(sum, turn);
        const float c1 = -q * q * inv_c * sum[0];              // dr = G + c1 r'
        float c2 = 0.0f;                                       // dh = p (..) + c2 h
        // p p p would be no binary32 number from a root mean square of 1.4e-13 down;
        // one p scales the sum, to the order of G, before the other two.
        if constexpr (POST) c2 = (-p * p) * (p * inv_c * (sum[1] + c1 * sum[2]));
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const Place<EXACT> place(i, pitch, vecs);
            const int64_t at = t * vecs + place.vec;
            float* gi = g[kKept ? i : 0];
            float* ri = r[kKept ? i : 0];
            float w[8];
            if constexpr (!kKept) {
                float d[8];
                stream(s + place.slot, gi, d, ri);
                w_pre.get(i, place.vec, w);
#pragma unroll
                for (int e = 0; e < 8; e += 2)
                    put2(gi, e, fma2(mul2(at2(d, e), two(q)), at2(w, e), at2(gi, e)));
            }
#pragma unroll
            for (int e = 0; e < 8; e += 2) put2(gi, e, fma2(at2(ri, e), two(c1), at2(gi, e)));
            if (place.live) store8<F32>(a.dr_out, at, gi);
            if (!has_h) continue;
            float h[8], gt[8], dh[8], dgate[8];
            values8<false>(s + place.slot, pitch, h);
            if constexpr (GATE) values8<false>(s + place.slot + at_gate, pitch, gt);
            w_post.get(i, place.vec, w);
#pragma unroll
            for (int e = 0; e < 8; e += 2) {
                float2 x = at2(gi, e), rest;
                float2 m = at2(h, e);
                if constexpr (POST) m = mul2(m, two(p));
                if constexpr (GATE) x = mul2(x, sigmoid2(at2(gt, e), rest));
                // acc_post leaves out the residual scale, which w holds
                put2(acc_post[i], e, fma2(x, m, at2(acc_post[i], e)));
                const float2 xw = mul2(x, at2(w, e));
                if constexpr (GATE) put2(dgate, e, mul2(mul2(xw, rest), m));
                put2(dh, e, POST ? fma2(xw, two(p), mul2(at2(h, e), two(c2))) : xw);
            }
            if (place.live) {
                store8<false>(a.dh, at, dh);
                if constexpr (GATE) store8<false>(a.dgate, at, dgate);
            }
        }
    }
    // partial rows [gridDim.x, 2, C]: dw_pre, dw_post
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int vec = tid + i * blockDim.x;
        if (vec >= vecs) continue;
        float4* part = reinterpret_cast<float4*>(a.workspace) +
                       static_cast<int64_t>(blockIdx.x) * 4 * vecs + vec * 2;
        if (a.dw_pre) {
            st_plain(part, make_float4(acc_pre[i][0], acc_pre[i][1], acc_pre[i][2], acc_pre[i][3]));
            st_plain(part + 1,
                     make_float4(acc_pre[i][4], acc_pre[i][5], acc_pre[i][6], acc_pre[i][7]));
        }
        if (a.dw_post) {
            part += 2 * vecs;
#pragma unroll
            for (int e = 0; e < 8; ++e) acc_post[i][e] *= a.res_scale;
            st_plain(part,
                     make_float4(acc_post[i][0], acc_post[i][1], acc_post[i][2], acc_post[i][3]));
            st_plain(part + 1,
                     make_float4(acc_post[i][4], acc_post[i][5], acc_post[i][6], acc_post[i][7]));
        }
    }
}

// dw[c] = the sum of `parts` partial rows, in 32 interleaved slices that are
// then added pairwise, always in the same order.  Block: 16 float4 columns x 32 slices.
constexpr int kSumCols = 16, kSumSlices = 32;
__global__ void __launch_bounds__(kSumCols* kSumSlices)
    sum_parts_kernel(const float* __restrict__ workspace, float* __restrict__ dw_pre,
                     float* __restrict__ dw_post, int64_t C, int parts) {
    __shared__ float4 slice[kSumSlices][kSumCols];
    grid_dependency_launch();
    const int col = threadIdx.x % kSumCols, part = threadIdx.x / kSumCols;
    const int64_t c4 = static_cast<int64_t>(blockIdx.x) * kSumCols + col;  // < 2 C / 4
    const bool post = c4 >= C / 4;
    float* out = post ? dw_post : dw_pre;
    grid_dependency_wait();
    float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
    if (out) {
#pragma unroll 8
        for (int i = part; i < parts; i += kSumSlices) {
            const float4 v = ld_ro(reinterpret_cast<const float4*>(workspace) + i * (C / 2) + c4);
            s.x += v.x;
            s.y += v.y;
            s.z += v.z;
            s.w += v.w;
        }
    }
    slice[part][col] = s;
#pragma unroll
    for (int n = kSumSlices / 2; n > 0; n /= 2) {
        __syncthreads();
        if (part >= n) continue;
        const float4 v = slice[part + n][col];
        s.x += v.x;
        s.y += v.y;
        s.z += v.z;
        s.w += v.w;
        slice[part][col] = s;
    }
    if (part == 0 && out)
        st_plain(reinterpret_cast<float4*>(out) + (c4 - (post ? C / 4 : 0)), s);
}

BackwardKind backward_kind(int64_t C, bool f32) {
    const int64_t vecs = C / 8;
    if (vecs <= kNarrow.threads) return kNarrow;
    if (!f32 && vecs <= kMiddle.threads && vecs % 32 == 0) return kMiddle;
    return vecs <= 2 * kWide.threads ? kWide : kWidest;
}
constexpr int kBackwardThreadsPerSm = 768;  // narrow rows, of about 80 registers

}  // namespace

// Partial rows a backward launch writes at most: one a CTA, as many CTAs an SM
// as its threads allow, no more than rows.  The caller's workspace is sized by
// this, so it must not change between that and the launch.
int64_t residual_norm_parts(int64_t T, int64_t C) {
    const int nv = backward_kind(C, true).nv;  // the kind with the fewer threads
    const int64_t per_sm = 1024 / shape_of(C, nv, kBackwardThreadsPerSm, 1, 1).threads;
    const int64_t most = device_sms() * (per_sm < 16 ? per_sm : 16);
    return T < most ? T : most;
}

cudaError_t launch_residual_norm_backward(const ResidualNormGrad& a, cudaStream_t stream) {
    const int slot = a.r_f32 ? 2 : 1;
    const int slots = (a.dr ? slot : 0) + (a.dx ? 1 + slot : 0) + (a.h ? 1 : 0) + (a.gate ? 1 : 0);
    const BackwardKind kind = backward_kind(a.C, a.r_f32);
    const Shape s = shape_of(a.C, kind.nv, kBackwardThreadsPerSm, slots, 1);
    int parts = 0;
    const auto launch = [&](auto* k) {
        parts = persistent_grid(reinterpret_cast<const void*>(k), s.threads, s.smem,
                                residual_norm_parts(a.T, a.C));
        if (const cudaError_t e = upload_checks(stream)) return e;
        return launch_pdl(k, parts, s.threads, s.smem, stream, true, a, s.fifo);
    };
    const cudaError_t e = with_options(a.r_f32, a.post, a.gate, [&](auto f32, auto post, auto gate) {
        const auto of = [&](auto nv, auto threads, auto mode) {
            return launch(
                &residual_norm_backward_kernel<nv(), threads(), f32(), post(), gate(), mode()>);
        };
        using std::integral_constant;
        constexpr integral_constant<int, 512> few;
        constexpr integral_constant<int, 896> many;
        if (kind.nv == 4)
            return of(integral_constant<int, 4>(), few, integral_constant<int, kAny>());
        const bool whole = a.dr && a.dx && a.h;
        if constexpr (!f32())
            if (kind.threads == many())
                return whole
                           ? of(integral_constant<int, 1>(), many, integral_constant<int, kExact>())
                           : of(integral_constant<int, 1>(), many, integral_constant<int, kAny>());
        return with_mode(whole, s.exact, [&](auto mode) {
            return kind.nv == 2 ? of(integral_constant<int, 2>(), few, mode)
                                : of(integral_constant<int, 1>(), few, mode);
        });
    });
    if (e != cudaSuccess || (!a.dw_pre && !a.dw_post)) return e;
    return launch_pdl(&sum_parts_kernel, static_cast<int>(a.C / (2 * kSumCols)),
                      kSumCols * kSumSlices, 0, stream, true,
                      static_cast<const float*>(a.workspace), a.dw_pre, a.dw_post, a.C, parts);
}

}  // namespace tkq
