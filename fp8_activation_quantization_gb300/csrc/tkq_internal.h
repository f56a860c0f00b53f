// tkq_internal.h -- launchers behind the C ABI (include/tkq.h).  Arguments are
// validated by the ABI layer before these are called.
#pragma once

#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>

namespace tkq {

// Tensor map of a row-major bf16 matrix [rows, cols] (row stride cols * 2
// bytes) for 2-D TMA boxes of box_rows x box_cols elements, no swizzle,
// out-of-range elements read as zero.  The driver entry point is looked up
// through the runtime once.  Returns false if the driver call is unavailable
// or rejects the arguments.
bool encode_bf16_2d(CUtensorMap* map, const void* base, int64_t cols, int64_t rows,
                    uint32_t box_cols, uint32_t box_rows);

// Number of SMs of the current device (cached per device; the environment
// variable TKQ_NUM_SMS overrides it for grid sizing experiments).
int num_sms();
// The same without the override: what a caller's buffer is sized by.
int device_sms();

// Address of the library's device status word on the current device (bit
// kDeviceTimeout: a bounded wait inside a kernel gave up).  Resolved once per
// device with cudaGetSymbolAddress.
unsigned int* device_status_word();

// Access checking of the checked build (-DTKQ_CHECKED; see tkq_device.cuh):
// the buffers of the current call, inputs and outputs, as address ranges.
constexpr uint32_t kDeviceOutOfBounds = 2u;  // status-word bit: an access was refused
constexpr int kCheckMax = 16;

struct CheckTable {
    unsigned long long lo[kCheckMax], hi[kCheckMax];  // [lo, hi) per buffer
    unsigned writable;                                // bit k: buffer k is an output
    int n;
    unsigned int* status;     // the library's device status word
    unsigned long long* bad;  // first refused address (bit 63: a store)
};

// The calling host thread's table for its current call (filled by the ABI
// layer, copied to the device by each launcher).  Checked build only.
CheckTable& host_check_table();

// Persistent grid: min(blocks needed, SMs x resident blocks per SM).
int persistent_grid(const void* kernel, int threads, size_t smem, int64_t blocks_needed);

// How many units of its walk each warp of a flat stream (token_cast.cu,
// swiglu_flat.cu), or each CTA of cast back, sends to L2 before it waits for
// the grid before it: a CTA of the next launch starts on an SM as soon as a
// CTA of the draining one exits there, so these prefetches fill the DRAM time
// the drain leaves idle.  Measured back to back on one GB300 (four CTAs per
// SM for the plain cast): one unit took the plain cast of [8192, 7168] from
// 29.44 to 29.15 us and the SwiGLU cast of [16384, 4096] from 27.07 to
// 26.38 us, two units less (29.26, 26.57 us); on an input of a few MB, where
// every warp has one or two units, prefetching them all took the plain cast of
// [1024, 4096] from 3.67 to 2.7-2.8 us.
inline int prologue_prefetch_units(int64_t input_bytes) {
    return input_bytes <= (int64_t{16} << 20) ? 4 : 1;
}

// Launch of one of the library's casts, with programmatic dependent launch
// allowed when `allow`: its grid may then be scheduled while the kernel before
// it on the stream is still draining, once every CTA of that kernel has
// started (the casts signal that at entry, grid_dependency_launch in
// tkq_device.cuh).  Each cast then waits (grid_dependency_wait) for the
// previous grid to complete, its memory visible, before any global load or
// store.  What overlaps is the launch, the CTAs' start-up and the L2
// prefetches the casts issue before that wait (prologue_prefetch_units and the
// rings' first boxes), which change no value any load returns.  After a kernel
// that does not signal, or after a copy, the launch is ordered as usual.
// Measured back to back, this takes 2.5-3.5 % off the ~30 us flat casts and,
// with the prefetches, 4.4 % off the transposed per-channel cast (56.5 to
// 54.0 us); it made the SwiGLU backward cast slower (152.0 against 154.5 us
// with the prefetches, 156.1 without), whose launcher passes allow = false.
// Returns the launch's error.
template <typename... Params, typename... Args>
inline cudaError_t launch_pdl(void (*kernel)(Params...), int grid, int block, size_t smem,
                              cudaStream_t stream, bool allow, Args... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(grid));
    cfg.blockDim = dim3(static_cast<unsigned>(block));
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = allow ? 1 : 0;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, static_cast<Params>(args)...);
    return e != cudaSuccess ? e : cudaGetLastError();
}

// sf_flags: TKQ_SF_* options of include/tkq.h (0 = row-major fp32 scales).
cudaError_t launch_per_token_cast(const void* x, void* out, void* sf, int64_t T, int64_t C,
                                  int fmt, unsigned sf_flags, cudaStream_t stream);

// The fp32 SwiGLU values y [T, H] the SwiGLU casts quantize (diagnostic).
cudaError_t launch_swiglu_values(const void* x, const float* w, float* y, int64_t T, int64_t H,
                                 cudaStream_t stream);

// The fp32 gradients [dg | du] ([T, 2H]) the SwiGLU backward cast quantizes
// (diagnostic).
cudaError_t launch_swiglu_backward_values(const void* x, const void* dy, const float* w, float* y,
                                          int64_t T, int64_t H, cudaStream_t stream);

// FP8 codes of n fp32 values, unscaled (diagnostic; n % 4 == 0).
cudaError_t launch_fp8_encode(const float* x, void* out, int64_t n, int fmt,
                              cudaStream_t stream);

// The per-token cast of a row-major fp32 [T, C] matrix.
cudaError_t launch_per_token_cast_f32(const float* x, void* out, void* sf, int64_t T, int64_t C,
                                      int fmt, unsigned sf_flags, cudaStream_t stream);

// clamp: null (no clamp) or the SwiGLU clamp bound c > 0; clamp_count (may be
// null) receives the number of clamped input values by atomic addition.
cudaError_t launch_swiglu_cast(const void* x, const float* w, void* out, void* sf, int64_t T,
                               int64_t H, int fmt, unsigned sf_flags, const float* clamp,
                               unsigned long long* clamp_count, cudaStream_t stream);

// The same operation as a flat stream (swiglu_flat.cu), bit-identical; the
// kernel for short launches.
cudaError_t launch_swiglu_cast_flat(const void* x, const float* w, void* out, void* sf, int64_t T,
                                    int64_t H, int fmt, unsigned sf_flags, const float* clamp,
                                    unsigned long long* clamp_count, cudaStream_t stream);

// Whether a SwiGLU forward cast of [T, 2H] runs as the flat stream: yes
// without a routing weight, and with one when its bf16 input is at most
// kSwigluFlatMaxBytes (measured: the flat stream is faster at every size
// without a weight, and with one up to 320 MiB of input; the two tie at
// 384 MiB and the ring is faster above).  The environment variable
// TKQ_SWIGLU_KERNEL ("flat" or "ring") overrides this for tests and
// measurements.
constexpr int64_t kSwigluFlatMaxBytes = int64_t{384} << 20;
bool swiglu_flat_chosen(int64_t T, int64_t H, bool weighted);

cudaError_t launch_swiglu_backward_cast(const void* x, const void* dy, const float* w, void* out,
                                        void* sf, int64_t T, int64_t H, int fmt,
                                        unsigned sf_flags, cudaStream_t stream);

// sf_flags: TKQ_SF_* layout of both the row scales [T, H/128] and the column
// scales [H, T/128] (0 = row-major fp32).
cudaError_t launch_swiglu_cast_t(const void* x, const float* w, void* out, float* sf,
                                 void* out_t, float* sf_t, int64_t T, int64_t H, int fmt,
                                 unsigned sf_flags, const float* clamp,
                                 unsigned long long* clamp_count, cudaStream_t stream);

// Per-channel cast (128-token groups; T % 128 == 0): codes [T, C] with sf
// [T/128, C], or codes [C, T] with sf [C, T/128] when transpose.
cudaError_t launch_per_channel_cast(const void* x, void* out, float* sf, int64_t T, int64_t C,
                                    int fmt, bool transpose, cudaStream_t stream);

// Per-block cast (128 x 128 blocks, ragged T): codes [T, C], sf [ceil(T/128), C/128].
cudaError_t launch_per_block_cast(const void* x, void* out, float* sf, int64_t T, int64_t C,
                                  int fmt, cudaStream_t stream);

// Cast back: out (fp32, or bf16 when out_bf16) = decode(code) * scale, with
// scales of gr x gc groups (1x128, 128x1 or 128x128).
cudaError_t launch_cast_back(const void* codes, const float* sf, void* out, int64_t T, int64_t C,
                             int gr, int gc, int fmt, bool out_bf16, cudaStream_t stream);

// Routing to experts (route.cu).  `ld`: row stride of the logits in elements.
struct RouteShape {
    int E, k;                      // experts, chosen per token
    int groups, topk_groups;       // groups of E / groups experts, of which topk_groups are searched
    int group_top;                 // 1 or 2 largest keys make a group's score
    bool sigmoid, renorm, bf16;
    float scale;
};
cudaError_t launch_route_topk(const void* logits, const float* bias, int32_t* ids, float* weights,
                              int32_t* counts, int64_t T, int64_t ld, const RouteShape& shape,
                              cudaStream_t stream);
cudaError_t launch_route_topk_backward(const void* logits, const int32_t* ids,
                                       const float* dweights, void* dlogits, int64_t T, int64_t ld,
                                       const RouteShape& shape, cudaStream_t stream);

// The SwiGLU cast with an 8-bit checkpoint of its input, and its backward from
// that checkpoint (swiglu_ckpt.cu).  out_kind: an FP8 format, or 2 for bf16
// gradients (dx_sf unused); y and dw may be null.
cudaError_t launch_swiglu_save(const void* x, const float* w, void* out, void* sf, void* ckpt,
                               float* ckpt_sf, int64_t T, int64_t H, int fmt, int ckpt_fmt,
                               unsigned sf_flags, cudaStream_t stream);
cudaError_t launch_swiglu_restore(const void* ckpt, const float* ckpt_sf, const void* dy,
                                  const float* w, void* dx, void* dx_sf, void* y, float* dw,
                                  int64_t T, int64_t H, int ckpt_fmt, int out_kind,
                                  unsigned sf_flags, cudaStream_t stream);

// The norms around a block (residual_norm.cu); optional pointers may be null.
struct ResidualNorm {
    const void *r, *h, *gate;       // [T, C]: residual stream, block output, gate logits
    const float *w_post, *w_pre;    // [C]
    void *r_out, *out, *sf, *x_out;
    float *rstd_post, *rstd_pre;    // [T]
    int64_t T, C;
    float res_scale, eps;
    bool post, pre, r_f32;
};
cudaError_t launch_residual_norm(const ResidualNorm& a, int fmt, unsigned sf_flags,
                                 cudaStream_t stream);

struct ResidualNormGrad {
    const void *dx, *dr, *r, *h, *gate;
    const float *w_post, *w_pre, *rstd_post, *rstd_pre;
    void *dr_out, *dh, *dgate;
    float *dw_post, *dw_pre;
    void* workspace;                // fp32 [residual_norm_parts, 2, C]
    int64_t T, C;
    float res_scale;
    bool post, r_f32;
};
int64_t residual_norm_parts(int64_t T, int64_t C);
cudaError_t launch_residual_norm_backward(const ResidualNormGrad& a, cudaStream_t stream);

// Tokens in the order of their experts and back (expert_rows.cu).  P = T * k pairs.
cudaError_t launch_expert_order(const int32_t* ids, int32_t* slots, int32_t* rows, int32_t* offsets,
                                int64_t P, int E, int align, int64_t R, cudaStream_t stream);

struct ExpertGather {
    const void* x;                     // [T, C] bf16 or codes
    const float* x_sf;                 // codes
    const int32_t *slots, *rows, *offsets;
    const float* weights;              // [T, k] or null
    void* out;
    float *out_sf, *row_weights;       // may be null
    int64_t T, C, R;
    int k, E, form, fmt;               // form: 0 bf16, 1 cast in fmt, 2 codes
};
cudaError_t launch_expert_gather(const ExpertGather& a, cudaStream_t stream);

cudaError_t launch_expert_reduce(const void* y, const int32_t* slots, const float* weights,
                                 const float* row_values, void* out, float* values, int64_t T, int64_t C,
                                 int k, int64_t R, bool out_f32, cudaStream_t stream);

struct ExpertReduceGrad {
    const void *dout, *y;
    const int32_t *slots, *rows, *offsets;
    const float* weights;
    void* dy;
    float *dy_sf, *dweights;
    int64_t T, C, R;
    int k, E, fmt;                     // fmt: an FP8 format, or 2 for bf16 rows
};
cudaError_t launch_expert_reduce_backward(const ExpertReduceGrad& a, cudaStream_t stream);

// The experts' products of FP8 codes and scales (expert_product.cu): the rows' product
// with the weights of their experts, and the weights' gradient.
struct ExpertProduct {
    const void* a;                     // rows' product: [R, K]; gradient: [N, R] (dy transposed)
    const float* a_sf;                 // [R, K/128];                [N, R/128]
    const void* b;                     // [E, N, K];                 [K, R] (x transposed)
    const float* b_sf;                 // [E, N/128, K/128];         [K, R/128]
    const int32_t* offsets;            // [E + 1]
    void* out;                         // bf16 [R, N];               [E, N, K]
    int64_t R, N, K;
    int E, fmt_a, fmt_b;
    bool out_f32;                      // gradient only
};
cudaError_t launch_expert_product(const ExpertProduct& p, cudaStream_t stream);
cudaError_t launch_expert_weight_grad(const ExpertProduct& p, cudaStream_t stream);

// Products of few rows with 4-bit weights (w4_product.cu).
struct W4Product {
    const void* x;                     // codes [M, K] (M = T, or T k with a row each)
    const float* x_sf;                 // [M, K/128]
    const void* w;                     // [E, N, K/2]
    const void* w_sf;                  // [E, N, K/32] UE8M0 or [E, N, K/128] fp32
    const int32_t* ids;                // [T, k] or null
    void* out;                         // bf16 [T k, N]
    int64_t T, N, K;
    int k, E, group, fmt;
    bool each;                         // a row of x for each pair
};
cudaError_t launch_w4_product(const W4Product& p, cudaStream_t stream);
cudaError_t launch_w4_cast(const void* w, void* codes, void* sf, int64_t N, int64_t K, int group,
                           cudaStream_t stream);

// Tensor map of a row-major matrix of bytes [rows, cols] for boxes of 128 bytes x box_rows
// in the 128-byte swizzle, out-of-range elements read as zero.
bool encode_u8_2d_swizzled(CUtensorMap* map, const void* base, int64_t cols, int64_t rows,
                           uint32_t box_rows);
// The same of a row-major bf16 matrix, boxes of 64 elements x box_rows.
bool encode_bf16_2d_swizzled(CUtensorMap* map, const void* base, int64_t cols, int64_t rows,
                             uint32_t box_rows);

}  // namespace tkq
