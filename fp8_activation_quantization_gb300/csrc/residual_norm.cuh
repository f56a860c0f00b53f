// residual_norm.cuh -- what the two directions of the block norms share
// (residual_norm.cu, residual_norm_backward.cu): sums over a CTA, a thread's rows
// in flight, its weights, and the shape of a launch.
#pragma once

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
// the ordering there is.  A row that is not a whole number of warps leaves the
// CTA's last half warps without vectors of their own (C is a multiple of 128
// channels, 16 vectors): they take those of the half warps before them along, so
// that all threads run the same straight code, add nothing to sums and store
// nothing.  (Skipping them with a predicate around each vector took the backward of
// 8192 x 7168 from 162 to 182 us and that of 16384 x 4096 from 171 to 269 us.)
constexpr int kMaxDepth = 4;

struct Fifo {
    int depth, slots;  // stages, 16-byte pieces of a vector of one row
};

// A thread's i-th vector: its place in the CTA's slots, the row's vector, and
// whether that is its own.
template <bool EXACT>  // every vector is its thread's own
struct Place {
    int slot, vec;
    bool live;
    __device__ __forceinline__ Place(int i, int pitch, int vecs) {
        slot = threadIdx.x + i * blockDim.x;
        live = EXACT || slot < vecs;
        vec = live ? slot : slot - (pitch - vecs);
    }
};

// What an instance knows of its launch: nothing; that the operands of the usual
// call are there (WHOLE in the kernels); that, and that the row is exactly the
// CTA's vectors.
enum Mode { kAny, kWhole, kExact };

// Copies the vector at `at` (in vectors of eight) of a tensor to `dst`; a
// binary32 vector's second half goes `pitch` pieces further.
template <bool F32>
__device__ __forceinline__ void fetch(uint4* dst, int pitch, const void* base, int64_t at) {
    const uint4* p = static_cast<const uint4*>(base) + at * (F32 ? 2 : 1);
    cp_async16(dst, p);
    if constexpr (F32) cp_async16(dst + pitch, p + 1);
}
// Its eight values.
template <bool F32>
__device__ __forceinline__ void values8(const uint4* src, int pitch, float* v) {
    const uint4 a = *src;
    if constexpr (F32) {
        const uint4 b = src[pitch];
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

    template <bool EXACT>
    __device__ __forceinline__ void init(const float* weights, float s, int pitch, int vecs) {
        w = weights;
        scale = s;
        if constexpr (kKept) {
#pragma unroll
            for (int i = 0; i < NV; ++i) weights8(w, Place<EXACT>(i, pitch, vecs).vec, scale, kept[i]);
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
    const size_t stage = static_cast<size_t>(slots) * nv * s.threads * 16 * rows;
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
template <typename F>
cudaError_t with_mode(bool whole, bool exact, F&& f) {
    if (!whole) return f(std::integral_constant<int, kAny>());
    return exact ? f(std::integral_constant<int, kExact>()) : f(std::integral_constant<int, kWhole>());
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

}  // namespace
}  // namespace tkq
