// w4_product.cu -- products of few rows with 4-bit weights (tkq_w4_product): FP8 rows
// with 1x128 scales times E2M1 matrices with a scale per 1x32 (UE8M0) or 1x128 (fp32)
// group, of one matrix or of each row's expert; and the cast that makes such weights
// (tkq_w4_cast).
//
//   out[p, n] = sum_g xs[p, g] sum_{h in g} ws[e, n, h] sum_{k in h} x[p, k] w[e, n, k]
//
// g: groups of 128 channels, h: the weights' groups within them.  Every E2M1 and FP8
// value is a binary16 value, so the tensor core (m16n8k16, binary32 sums) adds exact
// products; a group's sum is then multiplied by its scales in binary32.
//
// Reading the weights bounds this: a few rows do 2 to 32 operations for each half byte.
// Weights take the place of the MMA's 16-row operand and up to eight rows of x that of
// the eight columns.  An expert's rows are cut into runs of 8 or 16, and the weights are
// read and widened once for each run: one matrix of 4096 x 4096 takes 8.5 us with one
// row, 12 with 16, 31 with 64 and 393 with 1024.  (The 5th-generation tensor core takes
// E2M1 operands beside FP8 ones, in bytes of shared memory that a tensor map of 4-bit
// elements can lay out, and would take many rows a run; that form has not been built.)
// A warp takes 32 or 64 rows of a matrix, 256 channels at a time, from a ring of its own
// in shared memory: one TMA box of rows of 128 bytes and a bulk copy for each row of x.
// (Copies of 16 bytes a lane took 134 us for 48 tokens, 8 of 64 matrices of 4096 x 2048,
// 70 of them without any arithmetic.)  A CTA takes an equal share of all row blocks, one
// after another; S of its warps share those of a block, each taking every S-th 256
// channels, where otherwise some of the warps would have none left at the end.  No warp
// waits for another but at the end of shared rows.
// Measured: those 48 tokens 79 us (3.6 TB/s), one token's 8 matrices of 4096 x 4096 21 us
// (3.3 TB/s), with fp32 scales 6 to 7 % less; 128 channels at a time, in twice as many stages,
// took 13 us more for the 48.  Nothing is full there (memory 46 %, the tensor pipe 22 %, issue
// slots 61 %): what is left is the latency of a warp's own steps, one after another; widening,
// 7 operations for 8 weights, is over a quarter of their instructions.
// FP8 MMAs (m16n8k32) would take codes of x as they are, but are slower here than binary16
// ones: 190 us where those took 145.
#include <cuda_runtime.h>

#include "tkq_async.cuh"
#include "tkq_device.cuh"
#include "tkq_internal.h"

namespace tkq {
namespace {

// What a warp takes: with up to eight rows of x (NT = 1 columns of eight) 32 rows of the
// matrix, 16 warps a CTA; with up to 16 (NT = 2) 64 rows, 8 warps.
template <int NT>
struct Shape {
    static constexpr int kWarps = NT == 1 ? 16 : 8, kThreads = kWarps * 32;
    static constexpr int kRows = NT == 1 ? 32 : 64, kTiles = kRows / 16;
    static constexpr int kPart = kTiles * 2;  // sums of a lane that shared rows exchange at a time
};
constexpr int kMaxExperts = 1024;
constexpr int kMaxPairs = 1024;
constexpr int kDepth = 2;        // stages of a warp's ring: what fits 227 KB
constexpr int kPitch = 288;      // bytes from row to row of x: four rows' equal pieces lie in different banks

// One stage of a warp's ring: two blocks of 128 channels of 32 or 64 rows of weights
// (128-byte swizzle, aligned to its 1024 bytes) and, apart from them, of 8 NT rows of x,
// and both scales.
template <int NT>
struct alignas(16) Side {
    uint8_t x[8 * NT * kPitch];
    uint32_t ws[2][Shape<NT>::kRows];
    float xs[2][8 * NT];
};

// What a CTA knows of the rows: the pairs of each expert in turn, cut into runs of at
// most 8 NT.
template <int NT>
struct Plan {
    uint64_t full[Shape<NT>::kWarps][kDepth];
    int sums[2][Shape<NT>::kWarps];
    int runs;
    int abort;
    uint16_t pair[kMaxPairs];
    uint16_t xrow[kMaxPairs];         // its row of x
    uint16_t run_first[kMaxPairs + 2];  // and the end of the last run
    uint16_t run_expert[kMaxPairs];
    union {
        struct {
            int count[kMaxExperts];
            uint16_t first[kMaxExperts];  // first of its pairs in `pair`, then the next one's place
        };
        float parts[Shape<NT>::kWarps][Shape<NT>::kPart][32];  // sums of shared rows, after the plan is made
    };
};

struct Args {
    const uint8_t* x;        // [M, K]
    const float* xs;         // [M, K/128]
    const uint32_t* ws;      // [E, N, K/128] words: four UE8M0 bytes or one fp32
    const int32_t* ids;      // [P] or null
    uint16_t* out;           // [P, N]
    int P, N, K, E, share;   // x's row of pair p is p / share
    int ctas;                // the device's own grid, which the order of sums follows
    unsigned int* status;
};

// Eight E2M1 weights of a word as four binary16 pairs, the low nibble first.
__device__ __forceinline__ void decode_e2m1(uint32_t v, uint32_t (&h)[4]) {
    asm("{\n\t.reg .b8 a, b, c, d;\n\t"
        "mov.b32 {a, b, c, d}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, a;\n\t"
        "cvt.rn.f16x2.e2m1x2 %1, b;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, c;\n\t"
        "cvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
        : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
        : "r"(v));
}

__device__ __forceinline__ void mma_16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                          uint32_t a3, uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// The scales 2^(b - 127) of a word's four UE8M0 bytes.
__device__ __forceinline__ void decode_ue8m0(uint32_t v, float (&s)[4]) {
    uint32_t lo, hi;
    asm("{\n\t.reg .b16 a, b;\n\t"
        "mov.b32 {a, b}, %2;\n\t"
        "cvt.rn.bf16x2.ue8m0x2 %0, a;\n\t"
        "cvt.rn.bf16x2.ue8m0x2 %1, b;\n\t}"
        : "=r"(lo), "=r"(hi)
        : "r"(v));
    s[0] = bf16_lo(lo);
    s[1] = bf16_hi(lo);
    s[2] = bf16_lo(hi);
    s[3] = bf16_hi(hi);
}

// A position in a warp's work: run of pairs, rows of its matrix, pair of blocks.
struct Cursor {
    int run, block_row, kb;
    int expert, first, rows;
};

// The pairs of each expert in rising order, cut into runs: every CTA makes the same ones.
// Pairs stay in the registers of the lanes that read them, 32 to a warp; the warps place
// theirs one after another.  (One warp doing all of it took 9 us for 384 pairs.)
template <int NT>
__device__ void make_plan(Plan<NT>& pl, const Args& a) {
    constexpr int kThreads = Shape<NT>::kThreads, kWarps = Shape<NT>::kWarps;
    constexpr int kPer = kMaxExperts / kThreads;  // experts of a thread, in turn
    constexpr int kMine = kMaxPairs / kThreads;   // pairs of a lane, kThreads apart
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int bits = 32 - __clz(a.E - 1);         // of an expert's number
    int expert[kMine];
#pragma unroll
    for (int i = 0; i < kMine; ++i) {
        const int p = i * kThreads + tid;
        const int e = p >= a.P ? -1 : a.ids ? ld_ro(a.ids + p) : 0;
        expert[i] = e >= 0 && e < a.E ? e : -1;
    }
    for (int e = tid; e < a.E; e += kThreads) pl.count[e] = 0;
    __syncthreads();
    unsigned same[kMine];
#pragma unroll
    for (int i = 0; i < kMine; ++i) {
        if (i * kThreads + warp * 32 >= a.P) break;
        same[i] = lanes_of_value(expert[i], bits, __ballot_sync(0xffffffffu, expert[i] >= 0));
        if (expert[i] >= 0 && lane == __ffs(same[i]) - 1) atomicAdd(&pl.count[expert[i]], __popc(same[i]));
    }
    __syncthreads();
    int n = 0, r = 0, cnt[kPer];
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        cnt[i] = tid * kPer + i < a.E ? pl.count[tid * kPer + i] : 0;
        n += cnt[i];
        r += (cnt[i] + 8 * NT - 1) / (8 * NT);
    }
    const int n_mine = n, r_mine = r;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int un = __shfl_up_sync(0xffffffffu, n, o), ur = __shfl_up_sync(0xffffffffu, r, o);
        if (lane >= o) {
            n += un;
            r += ur;
        }
    }
    if (lane == 31) {
        pl.sums[0][warp] = n;
        pl.sums[1][warp] = r;
    }
    __syncthreads();
    int before_n = lane < warp ? pl.sums[0][lane] : 0, before_r = lane < warp ? pl.sums[1][lane] : 0;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        before_n += __shfl_xor_sync(0xffffffffu, before_n, o);
        before_r += __shfl_xor_sync(0xffffffffu, before_r, o);
    }
    int at_n = before_n + n - n_mine, at_r = before_r + r - r_mine;
    if (tid == kThreads - 1) {
        pl.runs = at_r + r_mine;
        pl.run_first[at_r + r_mine] = static_cast<uint16_t>(at_n + n_mine);
    }
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        const int e = tid * kPer + i;
        if (e < a.E) pl.first[e] = static_cast<uint16_t>(at_n);
        for (int k = 0; k < cnt[i]; k += 8 * NT, ++at_r) {
            pl.run_first[at_r] = static_cast<uint16_t>(at_n + k);
            pl.run_expert[at_r] = static_cast<uint16_t>(e);
        }
        at_n += cnt[i];
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kMine; ++i)
        for (int w = 0; w < kWarps; ++w) {
            if (i * kThreads + w * 32 >= a.P) break;
            if (warp == w) {
                const bool live = expert[i] >= 0;
                const int at = live ? pl.first[expert[i]] : 0;
                __syncwarp();
                if (live) {
                    const int to = at + __popc(same[i] & ((1u << lane) - 1u)), p = i * kThreads + tid;
                    pl.pair[to] = static_cast<uint16_t>(p);
                    pl.xrow[to] = static_cast<uint16_t>(p / a.share);
                    if (lane == __ffs(same[i]) - 1)
                        pl.first[expert[i]] = static_cast<uint16_t>(at + __popc(same[i]));
                }
            }
            __syncthreads();
        }
}

// acc += the products of a stage's block b, 8 NV columns of them.
template <int NV, int NT, bool G32, int FMT>
__device__ __forceinline__ void multiply(const uint8_t* w, const Side<NT>& s,
                                         float (&acc)[Shape<NT>::kTiles][NT][4], int b, int lane) {
    constexpr int kTiles = Shape<NT>::kTiles;
    const int g = lane >> 2, t = lane & 3;
    float blk[kTiles][NV][4];
#pragma unroll
    for (int m = 0; m < kTiles; ++m)
#pragma unroll
        for (int n = 0; n < NV; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i) blk[m][n][i] = 0.0f;
    float ws[2 * kTiles][G32 ? 4 : 1];
#pragma unroll
    for (int q = 0; q < 2 * kTiles; ++q) {
        if constexpr (G32)
            decode_ue8m0(s.ws[b][q * 8 + g], ws[q]);
        else
            ws[q][0] = __uint_as_float(s.ws[b][q * 8 + g]);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        uint32_t xf[NV][4];
#pragma unroll
        for (int n = 0; n < NV; ++n) {
            const uint2 xv = *reinterpret_cast<const uint2*>(s.x + (n * 8 + g) * kPitch + b * 128 + i * 32 + t * 8);
            xf[n][0] = fp8x2_to_f16x2<FMT>(xv.x & 0xFFFFu);
            xf[n][1] = fp8x2_to_f16x2<FMT>(xv.x >> 16);
            xf[n][2] = fp8x2_to_f16x2<FMT>(xv.y & 0xFFFFu);
            xf[n][3] = fp8x2_to_f16x2<FMT>(xv.y >> 16);
        }
#pragma unroll
        for (int m2 = 0; m2 < kTiles / 2; ++m2) {
            uint32_t v[4];
            asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                         : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3])
                         : "r"(smem_u32(w + (m2 * 32 + lane) * 128 + (((4 * b + i) ^ (lane & 7)) << 4))));
            uint32_t h[4][4];
#pragma unroll
            for (int q = 0; q < 4; ++q) decode_e2m1(v[q], h[q]);
#pragma unroll
            for (int mm = 0; mm < 2; ++mm) {
                const int m = 2 * m2 + mm;
                const uint32_t(&lo)[4] = h[2 * mm], (&hi)[4] = h[2 * mm + 1];
                float s0 = 0.0f, s1 = 0.0f;
                if constexpr (G32) {
                    s0 = ws[2 * m][i];
                    s1 = ws[2 * m + 1][i];
                }
#pragma unroll
                for (int n = 0; n < NV; ++n) {
                    if constexpr (G32) {
                        float p[4] = {0.0f, 0.0f, 0.0f, 0.0f};
                        mma_16816(p, lo[0], hi[0], lo[1], hi[1], xf[n][0], xf[n][1]);
                        mma_16816(p, lo[2], hi[2], lo[3], hi[3], xf[n][2], xf[n][3]);
                        blk[m][n][0] = fmaf(p[0], s0, blk[m][n][0]);
                        blk[m][n][1] = fmaf(p[1], s0, blk[m][n][1]);
                        blk[m][n][2] = fmaf(p[2], s1, blk[m][n][2]);
                        blk[m][n][3] = fmaf(p[3], s1, blk[m][n][3]);
                    } else {
                        mma_16816(blk[m][n], lo[0], hi[0], lo[1], hi[1], xf[n][0], xf[n][1]);
                        mma_16816(blk[m][n], lo[2], hi[2], lo[3], hi[3], xf[n][2], xf[n][3]);
                    }
                }
            }
        }
    }
#pragma unroll
    for (int n = 0; n < NV; ++n) {
        const float2 xs = *reinterpret_cast<const float2*>(&s.xs[b][n * 8 + 2 * t]);
#pragma unroll
        for (int m = 0; m < kTiles; ++m) {
            const float s0 = G32 ? 1.0f : ws[2 * m][0];
            const float s1 = G32 ? 1.0f : ws[2 * m + 1][0];
            acc[m][n][0] = fmaf(blk[m][n][0], xs.x * s0, acc[m][n][0]);
            acc[m][n][1] = fmaf(blk[m][n][1], xs.y * s0, acc[m][n][1]);
            acc[m][n][2] = fmaf(blk[m][n][2], xs.x * s1, acc[m][n][2]);
            acc[m][n][3] = fmaf(blk[m][n][3], xs.y * s1, acc[m][n][3]);
        }
    }
}

template <int NT, bool G32, int FMT>
__global__ void __launch_bounds__(Shape<NT>::kThreads, 1)
    w4_kernel(const __grid_constant__ CUtensorMap map_w, const Args a) {
    extern __shared__ __align__(1024) uint8_t base[];
    using St = Side<NT>;
    constexpr int kWarps = Shape<NT>::kWarps, kRows = Shape<NT>::kRows, kTiles = Shape<NT>::kTiles;
    constexpr int kBytesW = kRows * 128, kPart = Shape<NT>::kPart;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    uint8_t* ring_w = base + warp * kDepth * kBytesW;
    St* ring = reinterpret_cast<St*>(base + kWarps * kDepth * kBytesW) + warp * kDepth;
    uint8_t* rest = base + kWarps * kDepth * (kBytesW + sizeof(St));
    Plan<NT>& pl = *reinterpret_cast<Plan<NT>*>(rest);
    uint64_t* full = pl.full[warp];
    const int g = lane >> 2, t = lane & 3;
    if (lane == 0)
        for (int i = 0; i < kDepth; ++i) mbar_init(&full[i], 1);
    if (threadIdx.x == 0) pl.abort = 0;
    fence_barrier_init();
    make_plan<NT>(pl, a);

    const int KB = a.K / 128, KP = (KB + 1) / 2, NB = a.N / kRows;
    // this CTA's share of the row blocks, and the warps that share one: the fewest with
    // which at least seven eighths of the warps' time is used, else the most
    const int items = pl.runs * NB;
    const int64_t grid = gridDim.x;
    const int begin = static_cast<int>(items * static_cast<int64_t>(blockIdx.x) / grid);
    const int end = static_cast<int>(items * (static_cast<int64_t>(blockIdx.x) + 1) / grid);
    const int most = (items + a.ctas - 1) / a.ctas;
    int S = 1;
    while (S < kWarps && 2 * S <= KP) {
        const int teams = kWarps / S;
        if (8 * most >= 7 * ((most + teams - 1) / teams * teams)) break;
        S *= 2;
    }
    const int team = warp / S, of_team = warp - team * S, teams = kWarps / S;

    const auto place = [&](Cursor& c, int item) {
        c.run = item / NB;
        c.block_row = item - c.run * NB;
        c.kb = of_team;
        if (item < end) {
            c.expert = pl.run_expert[c.run];
            c.first = pl.run_first[c.run];
            c.rows = pl.run_first[c.run + 1] - c.first;
        }
    };
    int load_item = begin + team, item = load_item;
    Cursor ld, at;
    ld.expert = ld.first = ld.rows = at.expert = at.first = at.rows = 0;
    // where this lane's next copies come from: its row of x and its scale, scales of the weights
    const uint8_t* from_x = a.x;
    const float* from_xs = a.xs;
    const uint32_t* from_ws = a.ws;
    const auto place_load = [&]() {
        place(ld, load_item);
        if (load_item >= end) return;
        if (lane < ld.rows) {
            const int64_t r = pl.xrow[ld.first + lane];
            from_x = a.x + r * a.K + ld.kb * 256;
            from_xs = a.xs + r * KB + 2 * ld.kb;
        }
        from_ws = a.ws + (static_cast<int64_t>(ld.expert) * a.N + ld.block_row * kRows + lane) * KB + 2 * ld.kb;
    };
    place_load();
    RingPos<kDepth> in, out;
    int on_way = 0;      // stages asked for and not yet waited for
    bool dead = false;   // a wait gave up: nothing is asked for or waited for any more

    // issues the copies of the next block of this warp's work, if there is one
    const auto load_next = [&]() {
        while (load_item < end && ld.kb >= KP) {
            load_item += teams;
            place_load();
        }
        if (load_item < end && !dead) {
            St& s = ring[in.stage];
            uint64_t* bar = &full[in.stage];
            const int row0 = ld.expert * a.N + ld.block_row * kRows;
            const bool both = 2 * ld.kb + 1 < KB;  // the last pair may be one block
            const uint32_t bytes = both ? 256 : 128;
            if (lane == 0) mbar_arrive_expect_tx(bar, kBytesW + ld.rows * bytes);
            __syncwarp();
            if (lane == 0) tma_load_2d(ring_w + in.stage * kBytesW, &map_w, ld.kb * 128, row0, bar);
            if (lane < ld.rows) {
                if (access_ok(from_x, bytes, false)) bulk_load(s.x + lane * kPitch, from_x, bytes, bar);
                cp_async4(&s.xs[0][lane], from_xs);
                if (both) cp_async4(&s.xs[1][lane], from_xs + 1);
                from_x += S * 256;
                from_xs += 2 * S;
            }
#pragma unroll
            for (int i = 0; i < kRows / 32; ++i) {
                const uint32_t* from = from_ws + static_cast<int64_t>(i * 32) * KB;
                cp_async4(&s.ws[0][i * 32 + lane], from);
                if (both) cp_async4(&s.ws[1][i * 32 + lane], from + 1);
            }
            from_ws += 2 * S;
            ld.kb += S;
            in.advance();
            ++on_way;
        }
        cp_async_commit();
    };
#pragma unroll
    for (int i = 0; i < kDepth - 1; ++i) load_next();

    for (; item < end; item += teams) {
        place(at, item);
        float acc[kTiles][NT][4];
#pragma unroll
        for (int m = 0; m < kTiles; ++m)
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int i = 0; i < 4; ++i) acc[m][n][i] = 0.0f;
        for (; at.kb < KP; at.kb += S) {
            load_next();
            if (!dead) {
                const bool ok = mbar_wait_bounded(&full[out.stage], out.phase, &pl.abort, a.status);
                dead = !__all_sync(0xffffffffu, ok);
                if (dead && lane == 0) *static_cast<volatile int*>(&pl.abort) = 1;
            }
            if (dead) continue;
            cp_async_wait(kDepth);
            __syncwarp();
            const St& s = ring[out.stage];
            const uint8_t* w = ring_w + out.stage * kBytesW;
            out.advance();
            --on_way;
            // columns without rows are left out, eight at a time
            const int blocks = 2 * at.kb + 1 < KB ? 2 : 1;
#pragma unroll 1
            for (int b = 0; b < blocks; ++b) {
                if (NT == 1 || at.rows <= 8)
                    multiply<1, NT, G32, FMT>(w, s, acc, b, lane);
                else
                    multiply<NT, NT, G32, FMT>(w, s, acc, b, lane);
            }
            // the stage is refilled by the next copies, made in the async proxy
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            __syncwarp();
        }
        // shared rows: the team's first warp adds the others' in their order
        if (S > 1)
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                if (n * 8 >= at.rows) break;
#pragma unroll
                for (int m = 0; m < kTiles; m += kPart / 4) {
                    named_bar_sync(1 + team, S * 32);
                    if (of_team)
#pragma unroll
                        for (int i = 0; i < kPart; ++i) pl.parts[warp][i][lane] = acc[m + i / 4][n][i & 3];
                    named_bar_sync(1 + team, S * 32);
                    if (of_team == 0)
                        for (int o = 1; o < S; ++o)
#pragma unroll
                            for (int i = 0; i < kPart; ++i) acc[m + i / 4][n][i & 3] += pl.parts[warp + o][i][lane];
                }
            }
        if (of_team || dead) continue;
        // this lane's results: rows 16 m + g (+ 8), columns 8 n + 2 t (+ 1)
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int j = n * 8 + 2 * t + i;
                if (j >= at.rows) continue;
                uint16_t* o = a.out + static_cast<int64_t>(pl.pair[at.first + j]) * a.N + at.block_row * kRows + g;
#pragma unroll
                for (int m = 0; m < 2 * kTiles; ++m)
                    st_plain(o + m * 8, static_cast<uint16_t>(pack_bf16x2(acc[m / 2][n][2 * (m & 1) + i], 0.0f)));
            }
    }
    // after a wait that gave up, copies still on their way land before the CTA leaves
    for (; on_way > 0; --on_way, out.advance())
        mbar_wait_bounded(&full[out.stage], out.phase, nullptr, a.status);
    // pairs of no expert get zeros
    if (a.ids)
        for (int p = blockIdx.x * kWarps + warp; p < a.P; p += gridDim.x * kWarps) {
            const int e = ld_ro(a.ids + p);
            if (e >= 0 && e < a.E) continue;
            uint4* o = reinterpret_cast<uint4*>(a.out + static_cast<int64_t>(p) * a.N);
            for (int v = lane; v < a.N / 8; v += 32) st_stream(o + v, make_uint4(0, 0, 0, 0));
        }
}

template <int NT, bool G32, int FMT>
cudaError_t launch(const CUtensorMap& map, Args a, int64_t items, cudaStream_t stream) {
    auto* k = &w4_kernel<NT, G32, FMT>;
    constexpr int kThreads = Shape<NT>::kThreads;
    constexpr size_t smem = Shape<NT>::kWarps * kDepth * (Shape<NT>::kRows * 128 + sizeof(Side<NT>)) +
                            sizeof(Plan<NT>);
    static_assert(smem <= 227 * 1024, "shared memory");
    const int grid = persistent_grid(reinterpret_cast<const void*>(k), kThreads, smem, items);
    a.ctas = static_cast<int>(items < device_sms() ? items : device_sms());
    if (const cudaError_t e = upload_checks(stream)) return e;
    k<<<grid, kThreads, smem, stream>>>(map, a);
    return cudaGetLastError();
}

template <int NT>
cudaError_t launch_form(const W4Product& p, const Args& a, int64_t experts, cudaStream_t stream) {
    constexpr int kRows = Shape<NT>::kRows;
    CUtensorMap map;
    if (!encode_u8_2d_swizzled(&map, p.w, p.K / 2, p.E * p.N, kRows)) return cudaErrorInvalidValue;
    const bool g32 = p.group == 32;
    const int fmt = p.fmt;
    const int64_t items = experts * (p.N / kRows);
    if (g32)
        return fmt == kFmtE4M3 ? launch<NT, true, kFmtE4M3>(map, a, items, stream)
                               : launch<NT, true, kFmtE5M2>(map, a, items, stream);
    return fmt == kFmtE4M3 ? launch<NT, false, kFmtE4M3>(map, a, items, stream)
                           : launch<NT, false, kFmtE5M2>(map, a, items, stream);
}

// ---------------------------------------------------------------------------
// weights to 4 bits
// ---------------------------------------------------------------------------
// A warp takes 128 values of a row, a lane four: the largest magnitude of 8 lanes (32
// values) or of all, the scale amax / 6 (UE8M0: the power of two not below it), and the
// codes of the quotient, to nearest, ties to even, by the hardware conversion.  E2M1 has no
// code for what is no number, so a group with a NaN (which fmaxf would drop) or an infinity
// says so in its scale, and every product with it is NaN.
__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

template <bool G32>
__global__ void __launch_bounds__(256) w4_cast_kernel(const uint2* __restrict__ w, uint16_t* __restrict__ codes,
                                                      void* __restrict__ sf, int64_t groups) {
    const int lane = threadIdx.x & 31;
    for (int64_t u = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5); u < groups;
         u += static_cast<int64_t>(gridDim.x) * 8) {
        const uint2 q = ld_ro(w + u * 32 + lane);
        const float v[4] = {bf16_lo(q.x), bf16_hi(q.x), bf16_lo(q.y), bf16_hi(q.y)};
        float m = max_nan(max_nan(fabsf(v[0]), fabsf(v[1])), max_nan(fabsf(v[2]), fabsf(v[3])));
#pragma unroll
        for (int o = 1; o < (G32 ? 8 : 32); o <<= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
        const bool finite = m <= 3.402823466e+38f;
        // the smallest scale is 2^-126, so that zeros and tiny groups have one
        float s = fmaxf(__fdiv_rn(m, 6.0f), 1.17549435e-38f);
        if constexpr (G32) {
            float inv;
            pow2_scale(s, inv);
            if ((lane & 7) == 0)
                st_plain(static_cast<uint8_t*>(sf) + u * 4 + (lane >> 3),
                         finite ? static_cast<uint8_t>(__float_as_uint(s) >> 23) : uint8_t{255});
        } else if (lane == 0) {
            st_plain(static_cast<float*>(sf) + u, finite ? s : __uint_as_float(0x7FFFFFFFu));
        }
        uint16_t c;
        asm("{\n\t.reg .b8 lo, hi;\n\t"
            "cvt.rn.satfinite.e2m1x2.f32 lo, %2, %1;\n\t"
            "cvt.rn.satfinite.e2m1x2.f32 hi, %4, %3;\n\t"
            "mov.b16 %0, {lo, hi};\n\t}"
            : "=h"(c)
            : "f"(__fdiv_rn(v[0], s)), "f"(__fdiv_rn(v[1], s)), "f"(__fdiv_rn(v[2], s)),
              "f"(__fdiv_rn(v[3], s)));
        st_plain(codes + u * 32 + lane, finite ? c : uint16_t{0});
    }
}

}  // namespace

cudaError_t launch_w4_product(const W4Product& p, cudaStream_t stream) {
    Args a = {};
    a.x = static_cast<const uint8_t*>(p.x);
    a.xs = p.x_sf;
    a.ws = static_cast<const uint32_t*>(p.w_sf);
    a.ids = p.ids;
    a.out = static_cast<uint16_t*>(p.out);
    a.P = static_cast<int>(p.T * p.k);
    a.N = static_cast<int>(p.N);
    a.K = static_cast<int>(p.K);
    a.E = p.E;
    a.share = p.each ? 1 : p.k;
    a.status = device_status_word();
    const int64_t experts = p.ids ? (a.P < p.E ? a.P : p.E) : 1;  // at most this many have rows
    // eight columns where an expert has at most eight rows on average (48 tokens, 8 of 64
    // matrices of 4096 x 2048: 101 us, with 16 columns 115, both with stages of 128 channels).
    // The host knows no more than the average: where routing is uneven the busiest experts'
    // matrices are read once for every eight of their rows (64 tokens, 8 of 64: 87 us, all of
    // them to the same 8: 66)
    return a.P <= 8 * experts ? launch_form<1>(p, a, experts, stream) : launch_form<2>(p, a, experts, stream);
}

cudaError_t launch_w4_cast(const void* w, void* codes, void* sf, int64_t N, int64_t K, int group,
                           cudaStream_t stream) {
    const int64_t groups = N * (K / 128);
    const auto k = group == 32 ? &w4_cast_kernel<true> : &w4_cast_kernel<false>;
    const int grid = persistent_grid(reinterpret_cast<const void*>(k), 256, 0, (groups + 7) / 8);
    if (const cudaError_t e = upload_checks(stream)) return e;
    k<<<grid, 256, 0, stream>>>(static_cast<const uint2*>(w), static_cast<uint16_t*>(codes), sf, groups);
    return cudaGetLastError();
}

}  // namespace tkq
