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
#include <type_traits>

#include <cuda_runtime.h>

#include "tkq_async.cuh"
#include "tkq_device.cuh"
#include "tkq_internal.h"

namespace tkq {
namespace {

constexpr unsigned kAll = 0xffffffffu;


// Sums of N values over the CTA, in the same order each time.  The lanes first
// split the values among them (half of a pair to each half of the warp), so
// that N values take log2(N) steps more than one, not N times as many.  Two
// buffers in turn: a thread past the barrier of one sum has read the sum before.
template <int N, int THREADS>
struct CtaSum {
    static constexpr int kMaxWarps = THREADS / 32;
    static constexpr int kPad = N == 1 ? 1 : N == 2 ? 2 : 4;  // values, lanes of one: 32 / kPad
    static constexpr int kLanes = 32 / kPad;
    float buf[2][kPad][kMaxWarps];

    __device__ __forceinline__ void operator()(float (&v)[N], int& turn) {
        const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
        float s;
        if constexpr (kPad == 1) {
            s = v[0];
        } else if constexpr (kPad == 2) {
            const bool hi = lane & 16;
            s = (hi ? v[1] : v[0]) + __shfl_xor_sync(kAll, hi ? v[0] : v[1], 16);
        } else {
            static_assert(N == 3);
            const bool hi = lane & 16, up = lane & 8;
            const float a = (hi ? v[2] : v[0]) + __shfl_xor_sync(kAll, hi ? v[0] : v[2], 16);
            const float b = (hi ? 0.0f : v[1]) + __shfl_xor_sync(kAll, hi ? v[1] : 0.0f, 16);
            s = (up ? b : a) + __shfl_xor_sync(kAll, up ? a : b, 8);
        }
#pragma unroll
        for (int o = kLanes / 2; o > 0; o >>= 1) s += __shfl_xor_sync(kAll, s, o);
        const int mine = lane / kLanes, j = lane % kLanes;
        if (warps > 1) {
            if (j == 0) buf[turn][mine][warp] = s;
            __syncthreads();
            s = 0.0f;
#pragma unroll
            for (int k = 0; k < kMaxWarps; k += kLanes)
                if (j + k < warps) s += buf[turn][mine][j + k];
#pragma unroll
            for (int o = kLanes / 2; o > 0; o >>= 1) s += __shfl_xor_sync(kAll, s, o);
            turn ^= 1;
        }
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] = kPad == 1 ? s : __shfl_sync(kAll, s, i * kLanes);
    }
};

// ---------------------------------------------------------------------------
// a thread's rows in flight
// ---------------------------------------------------------------------------
// Shared memory holds `depth` rows; of each row a thread copies, and later
// reads, only its own 16-byte pieces, so its wait for its own copies is all
// the ordering there is.  Piece `slot` of vector `vec` of a stage:
// (stage * slots + slot) * vecs + vec.
constexpr int kMaxDepth = 4;

struct Fifo {
    int depth, slots;  // stages, 16-byte pieces of a vector of one row
};

// Copies the vector at `at` (in vectors of eight) of a tensor to `dst`; a
// binary32 vector's second half goes `vecs` pieces further.
template <bool F32>
__device__ __forceinline__ void fetch(uint4* dst, int vecs, const void* base, int64_t at) {
    const uint4* p = static_cast<const uint4*>(base) + at * (F32 ? 2 : 1);
    cp_async16(dst, p);
    if constexpr (F32) cp_async16(dst + vecs, p + 1);
}
// Its eight values.
template <bool F32>
__device__ __forceinline__ void values8(const uint4* src, int vecs, float* v) {
    const uint4 a = *src;
    if constexpr (F32) {
        const uint4 b = src[vecs];
        v[0] = __uint_as_float(a.x); v[1] = __uint_as_float(a.y);
        v[2] = __uint_as_float(a.z); v[3] = __uint_as_float(a.w);
        v[4] = __uint_as_float(b.x); v[5] = __uint_as_float(b.y);
        v[6] = __uint_as_float(b.z); v[7] = __uint_as_float(b.w);
    } else {
        unpack8(a, v);
    }
}
template <bool F32>
__device__ __forceinline__ void store8(void* base, int64_t at, const float* v) {
    uint4* p = static_cast<uint4*>(base) + at * (F32 ? 2 : 1);
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

// Eight weights of a row vector times `scale`, ones in the place of an absent vector.
__device__ __forceinline__ void weights8(const float* w, int vec, float scale, float* v) {
    float4 a = make_float4(1.f, 1.f, 1.f, 1.f), b = a;
    if (w) {
        a = ld_ro(reinterpret_cast<const float4*>(w) + vec * 2);
        b = ld_ro(reinterpret_cast<const float4*>(w) + vec * 2 + 1);
    }
    v[0] = a.x * scale; v[1] = a.y * scale; v[2] = a.z * scale; v[3] = a.w * scale;
    v[4] = b.x * scale; v[5] = b.y * scale; v[6] = b.z * scale; v[7] = b.w * scale;
}

// A thread's weights: kept in registers for all its rows where they fit (KEPT),
// else read again for each row.
template <int NV, bool KEPT>
struct Weights {
    static constexpr bool kKept = KEPT;
    float kept[kKept ? NV : 1][8];
    const float* w;
    float scale;

    __device__ __forceinline__ void init(const float* weights, float s, int vecs) {
        w = weights;
        scale = s;
        if constexpr (kKept) {
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int vec = threadIdx.x + i * blockDim.x;
                if (vec < vecs) weights8(w, vec, scale, kept[i]);
            }
        }
    }
    __device__ __forceinline__ void get(int i, int vec, float* v) const {
        if constexpr (kKept) {
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = kept[i][e];
        } else {
            weights8(w, vec, scale, v);
        }
    }
};

// sigmoid(x) and 1 - sigmoid(x) = exp(-x) sigmoid(x), for two values.  Where
// exp(-x) overflows the first is 0 and the product NaN, which fminf makes 1.
__device__ __forceinline__ float2 sigmoid2(float2 x, float2& rest) {
    const float2 t = mul2(x, make_float2(-1.4426950408889634f, -1.4426950408889634f));
    const float2 e = make_float2(ex2_approx(t.x), ex2_approx(t.y));
    const float2 den = add2(make_float2(1.0f, 1.0f), e);
    const float2 s = make_float2(rcp_approx(den.x), rcp_approx(den.y));
    const float2 r = mul2(e, s);
    rest = make_float2(fminf(r.x, 1.0f), fminf(r.y, 1.0f));
    return s;
}
__device__ __forceinline__ float2 two(float a) { return make_float2(a, a); }
__device__ __forceinline__ float2 at2(const float* v, int e) { return make_float2(v[e], v[e + 1]); }
__device__ __forceinline__ void put2(float* v, int e, float2 a) {
    v[e] = a.x;
    v[e + 1] = a.y;
}

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
//   up to 8192            two vectors, 128 registers: 7168: 88 us, 95 us with one
//                         vector and 896 threads; 5120: 73 us, 76 us
//   up to 16384           two vectors, 64 registers, the weights read again for
//                         each row: 16384: 137 us, 148 us with four and 512 threads
template <int NV, bool KEPT>
constexpr int kForwardThreads = NV == 2 && KEPT ? 512 : 1024;

// ROWS consecutive rows are taken at a time, so that their reductions share the
// barriers and the shuffles, and one row's arithmetic covers the other's
// latencies.  WHOLE: there is a block and a pre-norm, and the row is exactly
// the CTA's vectors, so nothing of that is asked again for each vector.
template <int NV, bool KEPT, bool F32, bool POST, bool GATE, int ROWS, bool WHOLE>
__global__ void __launch_bounds__(kForwardThreads<NV, KEPT>)
    residual_norm_kernel(const ResidualNorm a, const SfLayout lay, int64_t rows_walk, int fmt,
                         Fifo q8) {
    extern __shared__ uint4 fifo[];
    __shared__ CtaSum<ROWS, kForwardThreads<NV, KEPT>> cta_sum;
    grid_dependency_launch();
    constexpr int kR = F32 ? 2 : 1;   // slots of r; then h, gate
    int turn = 0;
    const int tid = threadIdx.x, vecs = static_cast<int>(a.C / 8);
    const float inv_c = 1.0f / static_cast<float>(a.C);
    const int row_size = q8.slots * vecs;
    const bool has_h = WHOLE || a.h, pre = WHOLE || a.pre;
    const auto inside = [&](int vec) { return WHOLE || vec < vecs; };
    const auto fetch_rows = [&](int64_t t0, int stage) {
#pragma unroll
        for (int k = 0; k < ROWS; ++k) {
            if (t0 + k >= a.T) break;
            uint4* s = fifo + (stage * ROWS + k) * row_size;
            const int64_t row = (t0 + k) * vecs;
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int vec = tid + i * blockDim.x;
                if (!inside(vec)) continue;
                if (has_h) fetch<false>(s + kR * vecs + vec, vecs, a.h, row + vec);
                fetch<F32>(s + vec, vecs, a.r, row + vec);
                if constexpr (GATE) fetch<false>(s + (kR + 1) * vecs + vec, vecs, a.gate, row + vec);
            }
        }
        cp_async_commit();
    };
    const int64_t step = static_cast<int64_t>(gridDim.x) * ROWS;
    const int64_t start = static_cast<int64_t>(blockIdx.x) * ROWS;
    grid_dependency_wait();
    for (int d = 0; d < q8.depth - 1; ++d) fetch_rows(start + d * step, d);
    Weights<NV, KEPT> w_post, w_pre;
    w_post.init(a.w_post, a.res_scale, vecs);
    w_pre.init(a.w_pre, 1.0f, vecs);
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
                float2 c = two(0.0f);
#pragma unroll
                for (int i = 0; i < NV; ++i) {
                    const int vec = tid + i * blockDim.x;
                    if (!inside(vec)) continue;
                    values8<false>(s + k * row_size + kR * vecs + vec, vecs, v[k][i]);
#pragma unroll
                    for (int e = 0; e < 8; e += 2) c = fma2(at2(v[k][i], e), at2(v[k][i], e), c);
                }
                sum[k] = c.x + c.y;
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
            float2 c = two(0.0f);
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int vec = tid + i * blockDim.x;
                float* vi = v[k][i];
                if (!inside(vec)) {
#pragma unroll
                    for (int e = 0; e < 8; ++e) vi[e] = 0.0f;
                    continue;
                }
                const uint4* at = s + k * row_size + vec;
                float r[8];
                values8<F32>(at, vecs, r);
                if (has_h) {
                    float w[8], g[8];
                    if constexpr (!POST) values8<false>(at + kR * vecs, vecs, vi);
                    if constexpr (GATE) values8<false>(at + (kR + 1) * vecs, vecs, g);
                    w_post.get(i, vec, w);
#pragma unroll
                    for (int e = 0; e < 8; e += 2) {
                        float2 b = mul2(at2(w, e), at2(vi, e));
                        if constexpr (GATE) {
                            float2 rest;
                            b = mul2(b, sigmoid2(at2(g, e), rest));
                        }
                        put2(vi, e, POST ? fma2(b, two(p[k]), at2(r, e)) : add2(b, at2(r, e)));
                    }
                    if (ROWS == 1 || t + k < a.T) store8<F32>(a.r_out, (t + k) * vecs + vec, vi);
                } else {
#pragma unroll
                    for (int e = 0; e < 8; ++e) vi[e] = r[e];
                }
#pragma unroll
                for (int e = 0; e < 8; e += 2) c = fma2(at2(vi, e), at2(vi, e), c);
            }
            sum[k] = c.x + c.y;
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
                const int vec = tid + i * blockDim.x;
                float* vi = v[k][i];
                float w[8] = {};
                if (inside(vec)) w_pre.get(i, vec, w);
#pragma unroll
                for (int e = 0; e < 8; e += 2) put2(vi, e, mul2(mul2(at2(vi, e), two(q)), at2(w, e)));
                if (a.x_out && row && inside(vec))
                    st_stream(static_cast<uint4*>(a.x_out) + (t + k) * vecs + vec, pack8_bf16(vi));
            }
        }
        if (!a.out) continue;
        if (fmt == kFmtE4M3)
            cast_rows<kFmtE4M3>(a, lay, t, vecs, v);
        else
            cast_rows<kFmtE5M2>(a, lay, t, vecs, v);
    }
}

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
// WHOLE: dr', dx and h are given and the row is exactly the CTA's vectors.
// How a row is held, by its width (16 bytes a channel; measured at T C = 59 - 67
// million, bf16 stream, gate):
//   up to 4096 channels   one vector a thread, 512 threads of 128 registers:
//                         4096: 171 us, 278 us with the 72 registers below;
//                         2048: 165 us, 227 us
//   up to 7168            one vector, 896 threads of 72 registers: 7168: 162 us,
//                         174 us with two vectors and 448 threads of 128 registers
//   up to 8192            two vectors, 512 threads of 128 registers
//   up to 16384           four, the stream and the weights not kept
struct BackwardKind {
    int nv, threads;
};
constexpr BackwardKind kNarrow = {1, 512}, kMiddle = {1, 896}, kWide = {2, 512}, kWidest = {4, 512};
template <int NV, int THREADS, bool F32, bool POST, bool GATE, bool WHOLE>
__global__ void __launch_bounds__(THREADS)
    residual_norm_backward_kernel(const ResidualNormGrad a, Fifo q8) {
    extern __shared__ uint4 fifo[];
    __shared__ CtaSum<POST ? 3 : 1, THREADS> cta_sum;
    grid_dependency_launch();
    constexpr int kS = F32 ? 2 : 1;   // slots of a stream: h, gate, dr, dx, r
    constexpr bool kKept = NV <= 2;
    const bool has_dr = WHOLE || a.dr, has_dx = WHOLE || a.dx, has_h = WHOLE || a.h;
    int turn = 0;
    const int tid = threadIdx.x, vecs = static_cast<int>(a.C / 8);
    const int at_gate = vecs;
    const int at_dr = ((has_h ? 1 : 0) + (GATE ? 1 : 0)) * vecs;
    const int at_dx = at_dr + (has_dr ? kS : 0) * vecs;
    const int at_r = at_dx + vecs;
    const float inv_c = 1.0f / static_cast<float>(a.C);
    const int stage_size = q8.slots * vecs;
    const auto inside = [&](int vec) { return WHOLE || vec < vecs; };
    const auto fetch_row = [&](int64_t t, int stage) {
        if (t < a.T)
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int vec = tid + i * blockDim.x;
                if (!inside(vec)) continue;
                uint4* s = fifo + stage * stage_size + vec;
                const int64_t at = t * vecs + vec;
                if (has_dr) fetch<F32>(s + at_dr, vecs, a.dr, at);
                if (has_dx) {
                    fetch<false>(s + at_dx, vecs, a.dx, at);
                    fetch<F32>(s + at_r, vecs, a.r, at);
                }
                if (has_h) fetch<false>(s, vecs, a.h, at);
                if constexpr (GATE) fetch<false>(s + at_gate, vecs, a.gate, at);
            }
        cp_async_commit();
    };
    // dr', dx and r' of one vector, zeros for what is absent
    const auto stream = [&](const uint4* s, float* g, float* d, float* r) {
#pragma unroll
        for (int e = 0; e < 8; ++e) g[e] = d[e] = r[e] = 0.0f;
        if (has_dr) values8<F32>(s + at_dr, vecs, g);
        if (has_dx) {
            values8<false>(s + at_dx, vecs, d);
            values8<F32>(s + at_r, vecs, r);
        }
    };
    float acc_pre[NV][8] = {}, acc_post[NV][8] = {};
    grid_dependency_wait();
    for (int d = 0; d < q8.depth - 1; ++d)
        fetch_row(blockIdx.x + static_cast<int64_t>(d) * gridDim.x, d);
    Weights<NV, kKept> w_post, w_pre;
    w_post.init(a.w_post, a.res_scale, vecs);
    w_pre.init(a.w_pre, 1.0f, vecs);
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
            const int vec = tid + i * blockDim.x;
            if (!inside(vec)) continue;
            float* gi = g[kKept ? i : 0];
            float* ri = r[kKept ? i : 0];
            float d[8], w[8];
            stream(s + vec, gi, d, ri);
            float2 s1 = two(0.0f);
            if (has_dx) {
                w_pre.get(i, vec, w);
#pragma unroll
                for (int e = 0; e < 8; e += 2) {
                    const float2 dq = mul2(at2(d, e), two(q));
                    put2(acc_pre[i], e, fma2(dq, at2(ri, e), at2(acc_pre[i], e)));
                    const float2 dw = mul2(dq, at2(w, e));
                    s1 = fma2(dw, at2(ri, e), s1);
                    put2(gi, e, add2(dw, at2(gi, e)));
                }
            }
            sum[0] += s1.x + s1.y;
            if constexpr (POST) {
                float2 s2 = two(0.0f), s3 = s2;
                float h[8], gt[8];
                values8<false>(s + vec, vecs, h);
                if constexpr (GATE) values8<false>(s + vec + at_gate, vecs, gt);
                w_post.get(i, vec, w);
#pragma unroll
                for (int e = 0; e < 8; e += 2) {
                    float2 f = mul2(at2(w, e), at2(h, e));
                    float2 rest;
                    if constexpr (GATE) f = mul2(f, sigmoid2(at2(gt, e), rest));
                    s2 = fma2(f, at2(gi, e), s2);
                    s3 = fma2(f, at2(ri, e), s3);
                }
                sum[1] += s2.x + s2.y;
                sum[2] += s3.x + s3.y;
            }
        }
        if (POST || has_dx) cta_sum(sum, turn);
        const float c1 = -q * q * inv_c * sum[0];              // dr = G + c1 r'
        float c2 = 0.0f;                                       // dh = p (..) + c2 h
        if constexpr (POST) c2 = -p * p * p * inv_c * (sum[1] + c1 * sum[2]);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int vec = tid + i * blockDim.x;
            if (!inside(vec)) continue;
            const int64_t at = t * vecs + vec;
            float* gi = g[kKept ? i : 0];
            float* ri = r[kKept ? i : 0];
            float w[8];
            if constexpr (!kKept) {
                float d[8];
                stream(s + vec, gi, d, ri);
                w_pre.get(i, vec, w);
#pragma unroll
                for (int e = 0; e < 8; e += 2)
                    put2(gi, e, fma2(mul2(at2(d, e), two(q)), at2(w, e), at2(gi, e)));
            }
#pragma unroll
            for (int e = 0; e < 8; e += 2) put2(gi, e, fma2(at2(ri, e), two(c1), at2(gi, e)));
            store8<F32>(a.dr_out, at, gi);
            if (!has_h) continue;
            float h[8], gt[8], dh[8], dgate[8];
            values8<false>(s + vec, vecs, h);
            if constexpr (GATE) values8<false>(s + vec + at_gate, vecs, gt);
            w_post.get(i, vec, w);
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
            store8<false>(a.dh, at, dh);
            if constexpr (GATE) store8<false>(a.dgate, at, dgate);
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

// Vectors a thread holds, threads a CTA and stages in flight for rows of C
// channels of `slots` 16-byte pieces a vector, `rows` at a time.  The CTAs that an
// SM's registers hold (`threads_per_sm`) share 224 KB of shared memory for up to
// four stages each; rather than less than two stages there are fewer CTAs.
struct Shape {
    int threads;
    bool exact;  // the row is exactly the CTA's vectors
    size_t smem;
    Fifo fifo;
};
constexpr size_t kSmemPerSm = 224 * 1024;
Shape shape_of(int64_t C, int nv, int threads_per_sm, int slots, int rows) {
    Shape s;
    const int vecs = static_cast<int>(C / 8);
    s.threads = ((vecs + nv - 1) / nv + 31) / 32 * 32;
    s.exact = vecs == nv * s.threads;
    const size_t stage = static_cast<size_t>(slots) * vecs * 16 * rows;
    int ctas = threads_per_sm / s.threads;
    ctas = ctas < 1 ? 1 : ctas > 16 ? 16 : ctas;
    while (ctas > 1 && kSmemPerSm / (stage * ctas) < 2) --ctas;
    size_t depth = kSmemPerSm / (stage * ctas);
    depth = depth < 1 ? 1 : depth > kMaxDepth ? kMaxDepth : depth;
    s.fifo = {static_cast<int>(depth), slots};
    s.smem = depth * stage;
    return s;
}

template <typename F>
cudaError_t with_flag(bool b, F&& f) {
    return b ? f(std::true_type()) : f(std::false_type());
}
// The instance for the stream's type and whether there are a post-norm and a gate.
template <typename F>
cudaError_t with_options(bool f32, bool post, bool gate, F&& f) {
    return with_flag(f32, [&](auto f32_) {
        return with_flag(post, [&](auto post_) {
            return with_flag(gate, [&](auto gate_) { return f(f32_, post_, gate_); });
        });
    });
}

BackwardKind backward_kind(int64_t C) {
    const int64_t vecs = C / 8;
    return vecs <= kNarrow.threads     ? kNarrow
           : vecs <= kMiddle.threads   ? kMiddle
           : vecs <= 2 * kWide.threads ? kWide
                                       : kWidest;
}
constexpr int kBackwardThreadsPerSm = 768;  // narrow rows, of about 80 registers

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
            return launch(&residual_norm_kernel<2, false, f32(), post(), gate(), 1, false>, one, 1);
        return with_flag(nv == 2, [&](auto wide) {
            return with_flag(one.exact && a.h && a.pre, [&](auto whole) {
                constexpr int n = wide() ? 2 : 1;
                // two rows at a time once every SM has work for that and the next two fit
                if (a.T >= 4 * int64_t{num_sms()} && pair.fifo.depth >= 2)
                    return launch(
                        &residual_norm_kernel<n, true, f32(), post(), gate(), 2, whole()>, pair, 2);
                return launch(&residual_norm_kernel<n, true, f32(), post(), gate(), 1, whole()>, one,
                              1);
            });
        });
    });
}

// Partial rows a backward launch writes at most: one a CTA, as many CTAs an SM
// as its threads allow, no more than rows.
int64_t residual_norm_parts(int64_t T, int64_t C) {
    const int nv = backward_kind(C).nv;
    const int64_t per_sm = 1024 / shape_of(C, nv, kBackwardThreadsPerSm, 1, 1).threads;
    const int64_t most = num_sms() * (per_sm < 16 ? per_sm : 16);
    return T < most ? T : most;
}

cudaError_t launch_residual_norm_backward(const ResidualNormGrad& a, cudaStream_t stream) {
    const int slot = a.r_f32 ? 2 : 1;
    const int slots = (a.dr ? slot : 0) + (a.dx ? 1 + slot : 0) + (a.h ? 1 : 0) + (a.gate ? 1 : 0);
    const BackwardKind kind = backward_kind(a.C);
    const Shape s = shape_of(a.C, kind.nv, kBackwardThreadsPerSm, slots, 1);
    int parts = 0;
    const auto launch = [&](auto* k) {
        parts = persistent_grid(reinterpret_cast<const void*>(k), s.threads, s.smem,
                                residual_norm_parts(a.T, a.C));
        if (const cudaError_t e = upload_checks(stream)) return e;
        return launch_pdl(k, parts, s.threads, s.smem, stream, true, a, s.fifo);
    };
    const cudaError_t e = with_options(a.r_f32, a.post, a.gate, [&](auto f32, auto post, auto gate) {
        const auto of = [&](auto nv, auto threads, auto whole) {
            return launch(&residual_norm_backward_kernel<nv(), threads(), f32(), post(), gate(),
                                                         whole()>);
        };
        using std::integral_constant;
        constexpr integral_constant<int, 512> few;
        constexpr integral_constant<int, 896> many;
        if (kind.nv == 4) return of(integral_constant<int, 4>(), few, std::false_type());
        return with_flag(s.exact && a.dr && a.dx && a.h, [&](auto whole) {
            if (kind.nv == 2) return of(integral_constant<int, 2>(), few, whole);
            return kind.threads == few() ? of(integral_constant<int, 1>(), few, whole)
                                         : of(integral_constant<int, 1>(), many, whole);
        });
    });
    if (e != cudaSuccess || (!a.dw_pre && !a.dw_post)) return e;
    return launch_pdl(&sum_parts_kernel, static_cast<int>(a.C / (2 * kSumCols)),
                      kSumCols * kSumSlices, 0, stream, true,
                      static_cast<const float*>(a.workspace), a.dw_pre, a.dw_post, a.C, parts);
}

}  // namespace tkq
