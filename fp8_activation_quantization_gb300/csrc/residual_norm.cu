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
// One CTA per row, the row in registers between its reads and its writes, so
// each tensor is read and written once; both are bound by memory (bf16
// stream, with gate: 9 bytes a channel forward, 16 backward).  The stream r' is
// rounded to its type where it is stored; the norm that follows is taken of
// the binary32 value before that rounding.
#include <type_traits>

#include <cuda_runtime.h>

#include "tkq_device.cuh"
#include "tkq_internal.h"

namespace tkq {
namespace {

constexpr unsigned kAll = 0xffffffffu;
constexpr int kMaxThreads = 512;
constexpr int kNoCast = 2;  // in the place of an FP8 format: no codes wanted

// Sums of N values over the CTA, in the same order each time.  Two buffers in
// turn: a thread past the barrier of one sum has read the sum before.
template <int N>
__device__ __forceinline__ void cta_sum(float (&v)[N], float (*buf)[N][32], int& turn) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
#pragma unroll
    for (int i = 0; i < N; ++i)
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) v[i] += __shfl_xor_sync(kAll, v[i], o);
    if (warps == 1) return;
    if (lane == 0)
#pragma unroll
        for (int i = 0; i < N; ++i) buf[turn][i][warp] = v[i];
    __syncthreads();
#pragma unroll
    for (int i = 0; i < N; ++i) {
        float s = lane < warps ? buf[turn][i][lane] : 0.0f;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(kAll, s, o);
        v[i] = s;
    }
    turn ^= 1;
}

// Eight channels of a stream in bf16 or binary32.
template <bool F32>
struct Chunk {
    uint4 q[F32 ? 2 : 1];

    __device__ __forceinline__ void load(const void* base, int64_t vec) {
        const uint4* p = static_cast<const uint4*>(base) + vec * (F32 ? 2 : 1);
#pragma unroll
        for (int i = 0; i < (F32 ? 2 : 1); ++i) q[i] = ld_stream(p + i);
    }
    __device__ __forceinline__ void values(float* v) const {
        if constexpr (F32) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                v[4 * i] = __uint_as_float(q[i].x);
                v[4 * i + 1] = __uint_as_float(q[i].y);
                v[4 * i + 2] = __uint_as_float(q[i].z);
                v[4 * i + 3] = __uint_as_float(q[i].w);
            }
        } else {
            unpack8(q[0], v);
        }
    }
    static __device__ __forceinline__ void store(void* base, int64_t vec, const float* v) {
        uint4* p = static_cast<uint4*>(base) + vec * (F32 ? 2 : 1);
        if constexpr (F32) {
#pragma unroll
            for (int i = 0; i < 2; ++i)
                st_stream(p + i,
                          make_uint4(__float_as_uint(v[4 * i]), __float_as_uint(v[4 * i + 1]),
                                     __float_as_uint(v[4 * i + 2]), __float_as_uint(v[4 * i + 3])));
        } else {
            st_stream(p, pack8_bf16(v));
        }
    }
};

// Eight weights of a row vector, ones when there is none.
__device__ __forceinline__ void weights8(const float* w, int64_t vec, float* v) {
    float4 a = make_float4(1.f, 1.f, 1.f, 1.f), b = a;
    if (w) {
        a = ld_ro(reinterpret_cast<const float4*>(w) + vec * 2);
        b = ld_ro(reinterpret_cast<const float4*>(w) + vec * 2 + 1);
    }
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
}

__device__ __forceinline__ float sigmoid(float x) {
    return rcp_approx(1.0f + ex2_approx(x * -1.4426950408889634f));
}

// ---------------------------------------------------------------------------
// forward
// ---------------------------------------------------------------------------
template <int NV, bool F32, int FMT>
__global__ void __launch_bounds__(kMaxThreads)
    residual_norm_kernel(const ResidualNorm a, const SfLayout lay, int64_t rows_walk) {
    __shared__ float buf[2][1][32];
    grid_dependency_launch();
    int turn = 0;
    const int tid = threadIdx.x, vecs = static_cast<int>(a.C / 8);
    const float inv_c = 1.0f / static_cast<float>(a.C);
    grid_dependency_wait();
    for (int64_t t = blockIdx.x; t < rows_walk; t += gridDim.x) {
        if (t >= a.T) {  // the padding rows of the column-major scale layouts
            for (int j = tid; j < lay.groups; j += blockDim.x)
                store_scale(a.sf, lay, t, false, j, 0.0f);
            continue;
        }
        float v[NV][8];
        float sum[1] = {0.0f};
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int vec = tid + i * blockDim.x;
#pragma unroll
            for (int e = 0; e < 8; ++e) v[i][e] = 0.0f;
            if (vec < vecs && a.h) {
                Chunk<false> c;
                c.load(a.h, t * vecs + vec);
                c.values(v[i]);
#pragma unroll
                for (int e = 0; e < 8; ++e) sum[0] += v[i][e] * v[i][e];
            }
        }
        float p = 1.0f;
        if (a.post) {
            cta_sum<1>(sum, buf, turn);
            p = __frsqrt_rn(sum[0] * inv_c + a.eps);
            if (tid == 0 && a.rstd_post) st_plain(a.rstd_post + t, p);
        }
        sum[0] = 0.0f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int vec = tid + i * blockDim.x;
            if (vec >= vecs) continue;
            Chunk<F32> c;
            c.load(a.r, t * vecs + vec);
            float r[8];
            c.values(r);
            if (a.h) {
                float w[8];
                weights8(a.w_post, vec, w);
#pragma unroll
                for (int e = 0; e < 8; ++e) w[e] *= p * v[i][e];
                if (a.gate) {
                    Chunk<false> g;
                    g.load(a.gate, t * vecs + vec);
                    float s[8];
                    g.values(s);
#pragma unroll
                    for (int e = 0; e < 8; ++e) w[e] *= sigmoid(s[e]);
                }
#pragma unroll
                for (int e = 0; e < 8; ++e) r[e] = fmaf(a.res_scale, w[e], r[e]);
                Chunk<F32>::store(a.r_out, t * vecs + vec, r);
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                v[i][e] = r[e];
                sum[0] += r[e] * r[e];
            }
        }
        if (!a.pre) continue;
        cta_sum<1>(sum, buf, turn);
        const float q = __frsqrt_rn(sum[0] * inv_c + a.eps);
        if (tid == 0 && a.rstd_pre) st_plain(a.rstd_pre + t, q);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int vec = tid + i * blockDim.x;
            const bool live = vec < vecs;
            float w[8];
            if (live) weights8(a.w_pre, vec, w);
#pragma unroll
            for (int e = 0; e < 8; ++e) v[i][e] = live ? v[i][e] * q * w[e] : 0.0f;
            if (live && a.x_out)
                st_stream(static_cast<uint4*>(a.x_out) + t * vecs + vec, pack8_bf16(v[i]));
            if constexpr (FMT != kNoCast) {
                // a group is half a warp's vectors
                float m = absmax8(v[i]);
#pragma unroll
                for (int o = 1; o < 16; o <<= 1) m = fmaxf(m, __shfl_xor_sync(kAll, m, o));
                float sc, inv;
                group_scale<FMT>(m, sc, inv);
                if (lay.flags & (kSfRoundPow2 | kSfPacked)) pow2_scale(sc, inv);
                if (live) {
                    st_stream(static_cast<uint2*>(a.out) + t * vecs + vec,
                              quantize8<FMT>(v[i], sc, inv));
                    if ((tid & 15) == 0) store_scale(a.sf, lay, t, true, vec / 16, sc);
                }
            }
        }
    }
}

// ---------------------------------------------------------------------------
// backward
// ---------------------------------------------------------------------------
// One reduction a row: with f = w_post s, the sum that dh needs,
// sum e f m, is linear in the first mean and so follows from
//   S1 = sum dx w_pre n,  S2 = sum f m (dr' + q dx w_pre),  S3 = sum f m n:
//   sum f m dr = S2 - q (S1 / C) S3.
// The weight gradients are summed over a CTA's rows in registers and written
// as one partial row a CTA; sum_parts_kernel adds them up in order.
template <int NV, bool F32>
__global__ void __launch_bounds__(kMaxThreads)
    residual_norm_backward_kernel(const ResidualNormGrad a) {
    __shared__ float buf[2][3][32];
    grid_dependency_launch();
    int turn = 0;
    const int tid = threadIdx.x, vecs = static_cast<int>(a.C / 8);
    const float inv_c = 1.0f / static_cast<float>(a.C);
    float acc_pre[NV][8] = {}, acc_post[NV][8] = {};
    grid_dependency_wait();
    for (int64_t t = blockIdx.x; t < a.T; t += gridDim.x) {
        const float p = a.post ? ld_ro(a.rstd_post + t) : 1.0f;
        const float q = a.dx ? ld_ro(a.rstd_pre + t) : 0.0f;
        Chunk<false> dx[NV], h[NV], gate[NV];
        Chunk<F32> dr[NV], r[NV];
        float sum[3] = {0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int vec = tid + i * blockDim.x;
            dx[i] = {};
            h[i] = {};
            gate[i] = {};
            dr[i] = {};
            r[i] = {};
            if (vec >= vecs) continue;
            const int64_t at = t * vecs + vec;
            if (a.dx) {
                dx[i].load(a.dx, at);
                r[i].load(a.r, at);
            }
            if (a.dr) dr[i].load(a.dr, at);
            if (a.h) h[i].load(a.h, at);
            if (a.gate) gate[i].load(a.gate, at);
        }
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int vec = tid + i * blockDim.x;
            if (vec >= vecs) continue;
            float d[8], n[8], g[8], m[8], s[8], wq[8], wp[8];
            dx[i].values(d);
            r[i].values(n);
            dr[i].values(g);
            h[i].values(m);
            gate[i].values(s);
            weights8(a.w_pre, vec, wq);
            weights8(a.w_post, vec, wp);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float nn = n[e] * q;
                acc_pre[i][e] += d[e] * nn;
                const float dw = d[e] * wq[e];
                sum[0] += dw * nn;
                const float f = wp[e] * (a.gate ? sigmoid(s[e]) : 1.0f) * m[e] * p;
                sum[1] += f * (g[e] + q * dw);
                sum[2] += f * nn;
            }
        }
        if (a.dx || a.post) cta_sum<3>(sum, buf, turn);
        const float m1 = sum[0] * inv_c;
        const float m2 = a.post ? (sum[1] - q * m1 * sum[2]) * inv_c : 0.0f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int vec = tid + i * blockDim.x;
            if (vec >= vecs) continue;
            const int64_t at = t * vecs + vec;
            float d[8], n[8], g[8], m[8], s[8], w[8];
            dx[i].values(d);
            r[i].values(n);
            dr[i].values(g);
            weights8(a.w_pre, vec, w);
#pragma unroll
            for (int e = 0; e < 8; ++e) g[e] += q * (d[e] * w[e] - n[e] * q * m1);
            Chunk<F32>::store(a.dr_out, at, g);
            if (!a.h) continue;
            h[i].values(m);
            gate[i].values(s);
            weights8(a.w_post, vec, w);
            float dg[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float mm = m[e] * p, err = a.res_scale * g[e];
                const float sg = a.gate ? sigmoid(s[e]) : 1.0f;
                // 1 - sigmoid(x) = sigmoid(-x), without cancellation
                if (a.gate) dg[e] = err * mm * w[e] * sg * sigmoid(-s[e]);
                acc_post[i][e] += err * sg * mm;
                m[e] = p * (err * sg * w[e] - mm * (a.res_scale * m2));
            }
            Chunk<false>::store(a.dh, at, m);
            if (a.gate) Chunk<false>::store(a.dgate, at, dg);
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
            st_plain(part,
                     make_float4(acc_post[i][0], acc_post[i][1], acc_post[i][2], acc_post[i][3]));
            st_plain(part + 1,
                     make_float4(acc_post[i][4], acc_post[i][5], acc_post[i][6], acc_post[i][7]));
        }
    }
}

// dw[c] = the sum of `parts` partial rows, in slices of eight interleaved
// rows that are then added in order.  Block: 32 float4 columns x 8 slices.
__global__ void __launch_bounds__(256)
    sum_parts_kernel(const float* __restrict__ workspace, float* __restrict__ dw_pre,
                     float* __restrict__ dw_post, int64_t C, int parts) {
    __shared__ float4 slice[8][32];
    grid_dependency_launch();
    const int col = threadIdx.x & 31, part = threadIdx.x >> 5;
    const int64_t c4 = static_cast<int64_t>(blockIdx.x) * 32 + col;  // < 2 C / 4
    const bool post = c4 >= C / 4;
    float* out = post ? dw_post : dw_pre;
    grid_dependency_wait();
    float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
    if (out)
        for (int i = part; i < parts; i += 8) {
            const float4 v = ld_ro(reinterpret_cast<const float4*>(workspace) + i * (C / 2) + c4);
            s.x += v.x;
            s.y += v.y;
            s.z += v.z;
            s.w += v.w;
        }
    slice[part][col] = s;
    __syncthreads();
    if (part || !out) return;
    for (int i = 1; i < 8; ++i) {
        s.x += slice[i][col].x;
        s.y += slice[i][col].y;
        s.z += slice[i][col].z;
        s.w += slice[i][col].w;
    }
    st_plain(reinterpret_cast<float4*>(out) + (c4 - (post ? C / 4 : 0)), s);
}

// Vectors a thread holds and threads a CTA for rows of C channels.
struct Shape {
    int nv, threads;
};
Shape shape_of(int64_t C) {
    const int vecs = static_cast<int>(C / 8);
    const int nv = vecs <= kMaxThreads ? 1 : vecs <= 2 * kMaxThreads ? 2 : 4;
    return {nv, ((vecs + nv - 1) / nv + 31) / 32 * 32};
}

template <typename F>
cudaError_t with_nv(int nv, F&& f) {
    if (nv == 1) return f(std::integral_constant<int, 1>());
    if (nv == 2) return f(std::integral_constant<int, 2>());
    return f(std::integral_constant<int, 4>());
}
template <typename F>
cudaError_t with_bool(bool b, F&& f) {
    return b ? f(std::true_type()) : f(std::false_type());
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
    const Shape s = shape_of(a.C);
    return with_nv(s.nv, [&](auto nv) {
        return with_bool(a.r_f32, [&](auto f32) {
            auto go = [&](auto f) {
                auto* k = &residual_norm_kernel<decltype(nv)::value, decltype(f32)::value,
                                                decltype(f)::value>;
                const int grid =
                    persistent_grid(reinterpret_cast<const void*>(k), s.threads, 0, rows);
                if (const cudaError_t e = upload_checks(stream)) return e;
                return launch_pdl(k, grid, s.threads, 0, stream, true, a, lay, rows);
            };
            if (!a.out) return go(std::integral_constant<int, kNoCast>());
            if (fmt == kFmtE4M3) return go(std::integral_constant<int, kFmtE4M3>());
            return go(std::integral_constant<int, kFmtE5M2>());
        });
    });
}

// Partial rows a backward launch writes at most: the SMs times the CTAs of the
// smallest row that fit one, no more than rows.
int64_t residual_norm_parts(int64_t T, int64_t C) {
    const int64_t per_sm = 2048 / shape_of(C).threads;
    const int64_t most = num_sms() * (per_sm < 16 ? per_sm : 16);
    return T < most ? T : most;
}

cudaError_t launch_residual_norm_backward(const ResidualNormGrad& a, cudaStream_t stream) {
    const Shape s = shape_of(a.C);
    int parts = 0;
    const cudaError_t e = with_nv(s.nv, [&](auto nv) {
        return with_bool(a.r_f32, [&](auto f32) {
            auto* k =
                &residual_norm_backward_kernel<decltype(nv)::value, decltype(f32)::value>;
            parts = persistent_grid(reinterpret_cast<const void*>(k), s.threads, 0,
                                    residual_norm_parts(a.T, a.C));
            if (const cudaError_t e = upload_checks(stream)) return e;
            return launch_pdl(k, parts, s.threads, 0, stream, true, a);
        });
    });
    if (e != cudaSuccess || (!a.dw_pre && !a.dw_post)) return e;
    return launch_pdl(&sum_parts_kernel, static_cast<int>(a.C / 64), 256, 0, stream, true,
                      static_cast<const float*>(a.workspace), a.dw_pre, a.dw_post, a.C, parts);
}

}  // namespace tkq
