// expert_product.cu -- the experts' products of FP8 codes and scales on the tensor
// cores: rows in expert order times the weights of their experts
// (tkq_expert_product), and the weights' gradient, a sum over an expert's rows
// (tkq_expert_weight_grad).
//
//   out[r, n]   = sum_g sa[r, g] sw[e, n/128, g]  sum_{k in g} a[r, k] w[e, n, k]
//   dw[e, n, k] = sum_g sy[n, g] sx[k, g]         sum_{r in g} dyt[n, r] xt[k, r]
//
// g: groups of 128 along the contracted axis.  A scale belongs to a row and a group,
// so the products of one group are added up by the tensor core (four MMAs of 32), and
// the groups' sums in registers, each times its scales: binary32 throughout.
//
// A CTA works on tiles of 128 x 256 of the result.  One warp's lane copies boxes of
// 128 bytes x 128 and x 256 rows into a ring of kStages stages (TMA, 128-byte swizzle);
// one lane of another issues the MMAs into one of two TMEM accumulators of 256 columns;
// eight warps take an accumulator out (32 lanes x 128 columns a warp, a lane one row),
// multiply it by its scales and add it to their registers while the tensor core fills
// the other one.  Two warps bring the scales, four groups at a time, to a ring of their
// own: read by the eight warps themselves, a group before its use, they cost more than
// the products (2.0 ms against 1.1 with scales that are not read, 65536 rows, 32
// matrices of 4096 x 4096).
// Measured on that size: 0.91 ms, 2.4 PFLOP/s, at 2070 MHz, and 0.98 ms, 2.25 PFLOP/s, when it
// runs for seconds and the power limit holds the clock near 1850 MHz; the gradient of 8
// matrices 1.49 to 1.53 ms, 1.45 PFLOP/s.  Copies and MMAs alone take 0.66 and 0.77 ms.  No
// unit is full: a summing warp reads 16 columns of tensor memory, waits for them and does
// their arithmetic, one operation for each sum and in the gradient two, in turn.  Reads alone,
// which contend with the MMAs, make it 0.77 ms; the arithmetic comes on top, and in the gradient the
// stores, which the same warps make.  A few rows for each of many experts are bound by the
// weights: 384 rows of 60 matrices of 2816 x 2048 in 51 us, 6.8 TB/s.
// Every tile has 256 columns: the last one of a width that is an odd multiple of 128 reads,
// multiplies and drops 128 columns that are another matrix's or none (65536 rows, 32 matrices of
// N x 4096: N = 1408 takes 348 us and 1536 351, 384 takes 126 and 512 129, 128 takes 78 and 256 83).
#include <cuda_runtime.h>

#include "tkq_async.cuh"
#include "tkq_device.cuh"
#include "tkq_internal.h"
#include "tkq_tensor.cuh"

namespace tkq {
namespace {

constexpr int kBM = 128, kBN = 256, kBK = 128;  // kBK: the width of a tensor map's box
constexpr int kStages = 3;
constexpr int kEpilogueWarps = 8;
constexpr int kCols = kBN / (kEpilogueWarps / 4);  // columns of a warp
// Three warpgroups: the registers of the launch, 168 a thread, are split between the two
// that hold a tile's sums (128 a thread) and the one that copies and multiplies.  The
// splits measured, ms at 65536 rows and 4096 x 4096: rows' product 208 / 88: 0.96, 216 /
// 72: 1.14, 224 / 56: 1.04; gradient, whose sums take the columns' scales too, 208 / 88:
// 1.74, 216 / 72: 1.65, 224 / 56: 1.68.
constexpr int kThreads = (kEpilogueWarps + 4) * 32;
template <bool GRAD>
struct Split {
    static constexpr int kSum = GRAD ? 216 : 208, kOther = GRAD ? 72 : 88;
    static constexpr int kUnroll = GRAD ? 2 : 8;  // scales' copies issued at a time
    static_assert(2 * kSum + kOther <= 3 * 168, "shares of the launch's registers");
};
constexpr uint32_t kBytesA = kBM * kBK, kBytesB = kBN * kBK;
constexpr uint32_t kStageBytes = kBytesA + kBytesB;
constexpr uint32_t kTmemCols = 2 * kBN;
// Rows' product: a warp's 32 rows of 128 results, as two boxes of 64 columns, wait in
// shared memory for their TMA stores, which overlap the next tile (65536 rows and 4096 x
// 4096: 0.91 ms, stored directly 0.96, not stored 0.84).  They take the fourth stage's
// room: three stages are as fast as four, and without either the gradient's scales find
// more of the L1 (1.53 ms, with four stages 1.65).
constexpr uint32_t kBytesBox = 32 * 128, kBytesOut = 2 * kEpilogueWarps * kBytesBox;
constexpr int kMaxExperts = 1024;

struct Smem {
    uint64_t full[kStages], empty[kStages], acc_full[2], acc_empty[2], sc_full[3], sc_empty[3];
    uint32_t tmem;
    int abort;
    int start[kMaxExperts + 1];  // first row of each expert
    int tile[kMaxExperts + 1];   // rows' product: row tiles before each expert
};

// The scales of four groups: of a tile's rows, and of its columns (rows' product: of its
// two blocks of 128).  Groups are 8 banks apart, so that eight rows' four groups lie in
// different ones.
constexpr int kUnit = 4, kUnits = 3;
template <bool GRAD>
struct alignas(16) Scales {
    float a[kUnit][kBM + 8];
    float b[kUnit][GRAD ? kBN + 8 : 4];
};

struct Args {
    const float *a_sf, *b_sf;
    const int32_t* offsets;
    void* out;
    int R, N, K, E;
    uint32_t idesc;
    unsigned int* status;
};

// Arrives on `bar` when this thread's asynchronous copies so far have landed.
__device__ __forceinline__ void cp_async_arrive(uint64_t* bar) {
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}

// One tile of the walk: its expert, where its rows (of A) and columns (rows of B) start,
// and its groups.
struct Tile {
    int e, row, col, g0, groups;
};

// The walk over the tiles, the same for every role.  Rows' product: the tiles of one
// expert in turn, its row tiles fastest, so that the CTAs at work share its weights and
// rows in L2.  Gradient: expert by expert, the tiles of dw by rows of N.
template <bool GRAD>
struct Walk {
    int at, e, n_col, per_expert;
    __device__ __forceinline__ Walk(const Args& a) {
        at = blockIdx.x;
        e = 0;
        n_col = ((GRAD ? a.K : a.N) + kBN - 1) / kBN;
        per_expert = GRAD ? (a.N / kBM) * n_col : 0;
    }
    __device__ __forceinline__ bool get(const Args& a, const Smem& sm, Tile& t) {
        if constexpr (GRAD) {
            e = at / per_expert;
            if (e >= a.E) return false;
            const int local = at - e * per_expert;
            const int r = local / n_col;
            t.e = e;
            t.row = r * kBM;
            t.col = (local - r * n_col) * kBN;
            t.g0 = sm.start[e] / kBK;
            t.groups = sm.start[e + 1] / kBK - t.g0;
        } else {
            while (e < a.E && at >= sm.tile[e + 1] * n_col) ++e;
            if (e >= a.E) return false;
            const int rows = sm.tile[e + 1] - sm.tile[e];
            const int local = at - sm.tile[e] * n_col;
            const int c = local / rows;
            t.e = e;
            t.row = sm.start[e] + (local - c * rows) * kBM;
            t.col = c * kBN;
            t.g0 = 0;
            t.groups = a.K / kBK;
        }
        return true;
    }
    __device__ __forceinline__ void next() { at += gridDim.x; }
};

template <bool GRAD, bool F32>
__global__ void __launch_bounds__(kThreads, 1)
    product_kernel(const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_b,
                   const __grid_constant__ CUtensorMap map_out, const Args a) {
    extern __shared__ uint8_t raw[];
    uint8_t* ring = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t{1023});
    uint8_t* boxes = ring + kStages * kStageBytes;  // rows' product
    Scales<GRAD>* scales = reinterpret_cast<Scales<GRAD>*>(boxes + (GRAD ? 0 : kBytesOut));
    Smem& sm = *reinterpret_cast<Smem*>(scales + kUnits);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;

    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages; ++s) {
            mbar_init(&sm.full[s], 1);
            mbar_init(&sm.empty[s], 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(&sm.acc_full[b], 1);
            mbar_init(&sm.acc_empty[b], kEpilogueWarps);
        }
        for (int u = 0; u < kUnits; ++u) {
            mbar_init(&sm.sc_full[u], 64);
            mbar_init(&sm.sc_empty[u], kEpilogueWarps);
        }
        sm.abort = 0;
        fence_barrier_init();
    }
    __syncwarp();
    if (warp == 0) tmem_alloc(&sm.tmem, kTmemCols);
    // starts of the experts' rows, kept within the rows there are and in rising order
    if (warp == 1) {
        int from = 0, tiles = 0;
        for (int e0 = 0; e0 <= a.E; e0 += 32) {
            const int e = e0 + lane;
            int v = e <= a.E ? ld_ro(a.offsets + e) : 0;
            v = v < 0 ? 0 : v > a.R ? a.R : v;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int x = __shfl_up_sync(0xffffffffu, v, o);
                if (lane >= o) v = v > x ? v : x;
            }
            v = v > from ? v : from;
            if (e <= a.E) sm.start[e] = v;
            if constexpr (!GRAD) {
                int prev = __shfl_up_sync(0xffffffffu, v, 1);
                if (lane == 0) prev = e0 ? from : v;
                int n = e <= a.E ? (v - prev + kBM - 1) / kBM : 0;  // tiles of expert e - 1
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const int x = __shfl_up_sync(0xffffffffu, n, o);
                    if (lane >= o) n += x;
                }
                if (e <= a.E) sm.tile[e] = tiles + n;
                tiles += __shfl_sync(0xffffffffu, n, 31);
            }
            from = __shfl_sync(0xffffffffu, v, 31);
        }
    }
    tmem_fence_before();
    __syncthreads();
    tmem_fence_after();
    const uint32_t tmem = sm.tmem;
    Walk<GRAD> walk(a);
    Tile t;

    if (warp >= kEpilogueWarps) {
      asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(Split<GRAD>::kOther));
      if (warp == kEpilogueWarps) {
        // ------------------------------------------------------------ copies
        if (lane == 0) {
            RingPos<kStages> pos;
            uint32_t issued = 0;
            bool ok = true;
            for (; ok && walk.get(a, sm, t); walk.next()) {
                const int row_a = t.row, row_b = GRAD ? t.col : t.e * a.N + t.col;
                for (int g = 0; g < t.groups; ++g) {
                    if (!mbar_wait_bounded(&sm.empty[pos.stage], pos.phase ^ 1u, &sm.abort, a.status)) {
                        *static_cast<volatile int*>(&sm.abort) = 1;
                        ok = false;
                        break;
                    }
                    uint8_t* dst = ring + pos.stage * kStageBytes;
                    const int x = (t.g0 + g) * kBK;
                    mbar_arrive_expect_tx(&sm.full[pos.stage], kStageBytes);
                    tma_load_2d(dst, &map_a, x, row_a, &sm.full[pos.stage]);
                    tma_load_2d(dst + kBytesA, &map_b, x, row_b, &sm.full[pos.stage]);
                    pos.advance();
                    ++issued;
                }
            }
            // every copy this CTA issued has landed before it may leave
            const uint32_t first = issued > kStages ? issued - kStages : 0;
            for (uint32_t k = first; k < issued; ++k)
                mbar_wait_bounded(&sm.full[k % kStages], (k / kStages) & 1u, nullptr, a.status);
        }
      } else if (warp == kEpilogueWarps + 1) {
        // -------------------------------------------------------------- MMAs
        if (lane == 0) {
            RingPos<kStages> pos;
            RingPos<2> acc;
            bool ok = true;
            for (; ok && walk.get(a, sm, t); walk.next()) {
                for (int g = 0; g < t.groups; ++g) {
                    if (!mbar_wait_bounded(&sm.full[pos.stage], pos.phase, &sm.abort, a.status) ||
                        !mbar_wait_bounded(&sm.acc_empty[acc.stage], acc.phase ^ 1u, &sm.abort, a.status)) {
                        *static_cast<volatile int*>(&sm.abort) = 1;
                        ok = false;
                        break;
                    }
                    tmem_fence_after();
                    const uint32_t at = smem_u32(ring + pos.stage * kStageBytes);
                    const uint64_t da = smem_desc_k128(at), db = smem_desc_k128(at + kBytesA);
                    const uint32_t d = tmem + acc.stage * kBN;
#pragma unroll
                    for (int k = 0; k < kBK / 32; ++k)  // 32 bytes further in the swizzled row
                        mma_f8(d, da + 2 * k, db + 2 * k, a.idesc, k > 0);
                    mma_commit(&sm.empty[pos.stage]);
                    mma_commit(&sm.acc_full[acc.stage]);
                    pos.advance();
                    acc.advance();
                }
            }
            // the MMAs issued have ended before the accumulators are given back
            for (int b = 0; b < 2; ++b) {
                mbar_wait_bounded(&sm.acc_full[acc.stage], acc.phase ^ 1u, nullptr, a.status);
                acc.advance();
            }
        }
      } else {
        // ------------------------------------------------------------ scales
        const int groups_all = GRAD ? a.R / kBK : a.K / kBK;
        constexpr int kUnroll = Split<GRAD>::kUnroll;
        const int q = lane & 3, r8 = lane >> 2, half = warp & 1;  // a warp: 8 rows' four groups
        RingPos<kUnits> pos;
        bool ok = true;
        for (; ok && walk.get(a, sm, t); walk.next()) {
            const int rows_end = GRAD ? a.N : sm.start[t.e + 1];
            for (int g0 = 0; g0 < t.groups; g0 += kUnit) {
                ok = mbar_wait_bounded(&sm.sc_empty[pos.stage], pos.phase ^ 1u, &sm.abort, a.status);
                if (!__all_sync(0xffffffffu, ok)) {
                    if (lane == 0) *static_cast<volatile int*>(&sm.abort) = 1;
                    ok = false;
                    break;
                }
                Scales<GRAD>& sc = scales[pos.stage];
                if (g0 + q < t.groups) {
                    const int g = t.g0 + g0 + q;
                    // rows and columns beyond the edges: the last scale there is
#pragma unroll kUnroll
                    for (int i = 0; i < kBM / 16; ++i) {
                        const int r = (2 * i + half) * 8 + r8;
                        const int row = t.row + r < rows_end ? t.row + r : rows_end - 1;
                        cp_async4(&sc.a[q][r], a.a_sf + static_cast<int64_t>(row) * groups_all + g);
                    }
                    if constexpr (GRAD) {
#pragma unroll kUnroll
                        for (int i = 0; i < kBN / 16; ++i) {
                            const int r = (2 * i + half) * 8 + r8;
                            const int col = t.col + r < a.K ? t.col + r : a.K - 1;
                            cp_async4(&sc.b[q][r], a.b_sf + static_cast<int64_t>(col) * groups_all + g);
                        }
                    } else if (r8 == 0) {
                        const int c = t.col + half * 128 < a.N ? t.col / 128 + half : a.N / 128 - 1;
                        cp_async4(&sc.b[q][half],
                                  a.b_sf + (static_cast<int64_t>(t.e) * (a.N / 128) + c) * groups_all + g);
                    }
                }
                cp_async_arrive(&sm.sc_full[pos.stage]);
                pos.advance();
            }
        }
        asm volatile("cp.async.wait_all;" ::: "memory");
      }
    } else {
        // ---------------------------------------------------- scales and sums
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(Split<GRAD>::kSum));
        const int quarter = warp & 3, part = warp >> 2;  // TMEM lanes, columns
        const int row_in = quarter * 32 + lane;
        const uint32_t lane_base = tmem + (static_cast<uint32_t>(quarter * 32) << 16) + part * kCols;
        RingPos<2> acc;
        RingPos<kUnits> pos;
        bool ok = true;
        for (; ok && walk.get(a, sm, t); walk.next()) {
            // lanes part at the end of a tile (one stores a box, or those with a row store it); reads of
            // tensor memory are the whole warp's
            __syncwarp();
            uint64_t sum[kCols / 2];  // pairs of binary32
#pragma unroll
            for (int i = 0; i < kCols / 2; ++i) sum[i] = 0;
            for (int g = 0; g < t.groups; ++g) {
                const int q = g & (kUnit - 1);
                if (q == 0) ok = mbar_wait_lean(&sm.sc_full[pos.stage], pos.phase, &sm.abort, a.status);
                if (ok) ok = mbar_wait_lean(&sm.acc_full[acc.stage], acc.phase, &sm.abort, a.status);
                if (!__all_sync(0xffffffffu, ok)) {
                    if (lane == 0) *static_cast<volatile int*>(&sm.abort) = 1;
                    ok = false;
                    break;
                }
                const Scales<GRAD>& sc = scales[pos.stage];
                const float s = GRAD ? sc.a[q][row_in] : sc.a[q][row_in] * sc.b[q][part * kCols / 128];
                const uint64_t s2 = static_cast<uint64_t>(__float_as_uint(s)) << 32 | __float_as_uint(s);
                tmem_fence_after();
                const uint32_t from = lane_base + acc.stage * kBN;
#pragma unroll
                for (int c = 0; c < kCols / 16; ++c) {
                    uint64_t v[8];
                    tmem_read16(from + c * 16, v);
                    if (c == kCols / 16 - 1) {
                        tmem_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(&sm.acc_empty[acc.stage]);
                    }
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        uint64_t p = v[i];
                        if constexpr (GRAD)
                            p = mul_pair(p, *reinterpret_cast<const uint64_t*>(&sc.b[q][part * kCols + c * 16 + 2 * i]));
                        sum[c * 8 + i] = fma_pair(p, s2, sum[c * 8 + i]);
                    }
                }
                acc.advance();
                if (q == kUnit - 1 || g + 1 == t.groups) {
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&sm.sc_empty[pos.stage]);
                    pos.advance();
                }
            }
            const int row = t.row + row_in, col = t.col + part * kCols;
            const bool live = row < (GRAD ? a.N : sm.start[t.e + 1]);
            if (!ok || col >= (GRAD ? a.K : a.N)) continue;
            const int64_t at = GRAD ? (static_cast<int64_t>(t.e) * a.N + row) * a.K + col
                                    : static_cast<int64_t>(row) * a.N + col;
            const auto value = [&](int i) {
                return static_cast<uint32_t>(i & 1 ? sum[i / 2] >> 32 : sum[i / 2]);
            };
            const auto pair = [&](int i) {
                return pack_bf16x2(__uint_as_float(value(i)), __uint_as_float(value(i + 1)));
            };
            if constexpr (!GRAD) {
                // the expert has all of the warp's rows (and, checked build, the output all of them: a box
                // is refused as a whole, its rows then one by one)
                if (t.row + quarter * 32 + 32 <= sm.start[t.e + 1] &&
                    __all_sync(0xffffffffu, access_ok(static_cast<uint16_t*>(a.out) + at, kCols * 2, true))) {
                    uint8_t* box = boxes + warp * 2 * kBytesBox;
                    if (lane == 0) bulk_wait_read();  // the tile before
                    __syncwarp();
#pragma unroll
                    for (int c = 0; c < 16; ++c) {
                        const uint4 v = make_uint4(pair(8 * c), pair(8 * c + 2), pair(8 * c + 4), pair(8 * c + 6));
                        *reinterpret_cast<uint4*>(box + (c >> 3) * kBytesBox + lane * 128 +
                                                  (((c & 7) ^ (lane & 7)) << 4)) = v;
                    }
                    fence_async_smem();
                    __syncwarp();
                    if (lane == 0) {
                        tma_store_2d(&map_out, box, col, t.row + quarter * 32);
                        tma_store_2d(&map_out, box + kBytesBox, col + 64, t.row + quarter * 32);
                        bulk_commit();
                    }
                    continue;
                }
            }
            // a lane's row in whole sectors of 32 bytes
            if (!live) continue;
            constexpr int kPer = F32 ? 8 : 16;
#pragma unroll
            for (int i = 0; i < kCols; i += kPer) {
                uint32_t w[8];
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    w[j] = F32 ? value(i + j) : pair(i + 2 * j);
                st_sector(static_cast<uint8_t*>(a.out) + (at + i) * (F32 ? 4 : 2), w);
            }
        }
        if (lane == 0) bulk_wait();
    }
    __syncwarp();
    tmem_fence_before();
    __syncthreads();
    tmem_fence_after();
    if (warp == 0) tmem_free(tmem, kTmemCols);
}

template <bool GRAD, bool F32>
cudaError_t launch(const ExpertProduct& p, int64_t tiles, cudaStream_t stream) {
    CUtensorMap map_a, map_b, map_out = {};
    const bool made =
        GRAD ? encode_u8_2d_swizzled(&map_a, p.a, p.R, p.N, kBM) && encode_u8_2d_swizzled(&map_b, p.b, p.R, p.K, kBN)
             : encode_u8_2d_swizzled(&map_a, p.a, p.K, p.R, kBM) &&
                   encode_u8_2d_swizzled(&map_b, p.b, p.K, p.E * p.N, kBN);
    if (!made || (!GRAD && !encode_bf16_2d_swizzled(&map_out, p.out, p.N, p.R, 32)))
        return cudaErrorInvalidValue;
    Args a = {};
    a.a_sf = p.a_sf;
    a.b_sf = p.b_sf;
    a.offsets = p.offsets;
    a.out = p.out;
    a.R = static_cast<int>(p.R);
    a.N = static_cast<int>(p.N);
    a.K = static_cast<int>(p.K);
    a.E = p.E;
    a.idesc = mma_f8_desc(p.fmt_a, p.fmt_b, kBM, kBN);
    a.status = device_status_word();
    auto* k = &product_kernel<GRAD, F32>;
    const size_t smem = kStages * kStageBytes + (GRAD ? 0 : kBytesOut) + kUnits * sizeof(Scales<GRAD>) + sizeof(Smem) + 1024;
    const int grid = persistent_grid(reinterpret_cast<const void*>(k), kThreads, smem, tiles);
    if (const cudaError_t e = upload_checks(stream)) return e;
    k<<<grid, kThreads, smem, stream>>>(map_a, map_b, map_out, a);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_expert_product(const ExpertProduct& p, cudaStream_t stream) {
    // at most this many row tiles: every expert's last one may be partial
    const int64_t most = p.R / kBM + (p.E < p.R ? p.E : p.R);
    return launch<false, false>(p, most * ((p.N + kBN - 1) / kBN), stream);
}

cudaError_t launch_expert_weight_grad(const ExpertProduct& p, cudaStream_t stream) {
    if (p.R == 0)  // no rows: no gradient
        return cudaMemsetAsync(p.out, 0, p.E * p.N * p.K * (p.out_f32 ? 4 : 2), stream);
    const int64_t tiles = p.E * (p.N / kBM) * ((p.K + kBN - 1) / kBN);
    return p.out_f32 ? launch<true, true>(p, tiles, stream) : launch<true, false>(p, tiles, stream);
}

}  // namespace tkq
