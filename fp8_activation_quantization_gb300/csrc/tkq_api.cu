// tkq_api.cu -- the C ABI of libtkq.so (declared in include/tkq.h): argument
// validation, status codes and dispatch to the kernel launchers.  Nothing here
// allocates device memory.
#include <atomic>
#include <cmath>
#include <cstdint>
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <functional>
#include <initializer_list>
#include <mutex>
#include <unordered_map>

#include <cuda_runtime.h>

#include "../../include/tkq.h"
#include "tkq_async.cuh"
#include "tkq_internal.h"

// The library's device status word (one per device): kernels OR status bits
// into it (tkq::kDeviceTimeout when a bounded wait gave up); the host reads and
// clears it with tkq_read_device_status.
__device__ unsigned int g_tkq_device_status;
// First address an access check refused (checked build; bit 63: a store).
__device__ unsigned long long g_tkq_bad_address;

namespace tkq {

namespace {
constexpr int kMaxDevices = 64;
std::atomic<int> g_sms[kMaxDevices];  // 0 = not yet queried
std::atomic<unsigned int*> g_status_ptr[kMaxDevices];
std::atomic<unsigned long long*> g_bad_ptr[kMaxDevices];

// One CTA waits on an mbarrier that nothing ever arrives on, so its bounded
// wait must give up after limit_ns and record a timeout in the status word.
__global__ void selftest_wait_kernel(unsigned int* status, uint64_t limit_ns) {
    __shared__ uint64_t bar;
    __shared__ int abort;
    if (threadIdx.x == 0) {
        mbar_init(&bar, 1);
        abort = 0;
        fence_barrier_init();
    }
    __syncthreads();
    if (threadIdx.x == 0) mbar_wait_bounded(&bar, 0, &abort, status, limit_ns);
}

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

struct Range {
    uintptr_t lo, hi;  // [lo, hi)
};
Range span(const void* p, int64_t bytes) {
    const uintptr_t a = reinterpret_cast<uintptr_t>(p);
    return {a, a + static_cast<uintptr_t>(bytes)};
}
bool overlap(Range a, Range b) { return a.lo < b.hi && b.lo < a.hi; }
}  // namespace

int device_sms() {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0) return 1;
    if (dev < kMaxDevices) {
        int v = g_sms[dev].load(std::memory_order_relaxed);
        if (v > 0) return v;
    }
    int v = 0;
    if (cudaDeviceGetAttribute(&v, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || v <= 0)
        v = 1;
    if (dev < kMaxDevices) g_sms[dev].store(v, std::memory_order_relaxed);
    return v;
}

int num_sms() {
    if (const char* env = std::getenv("TKQ_NUM_SMS")) {
        const int v = std::atoi(env);
        if (v > 0) return v;
    }
    return device_sms();
}

bool swiglu_flat_chosen(int64_t T, int64_t H, bool weighted) {
    if (const char* env = std::getenv("TKQ_SWIGLU_KERNEL")) {
        if (std::strcmp(env, "flat") == 0) return true;
        if (std::strcmp(env, "ring") == 0) return false;
    }
    return !weighted || T * 2 * H * 2 <= kSwigluFlatMaxBytes;
}

namespace {
using EncodeTiledFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                   const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                   const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                   CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_tiled() {
    static EncodeTiledFn fn = [] {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000,
                                             cudaEnableDefault, &q) != cudaSuccess ||
            q != cudaDriverEntryPointSuccess)
            p = nullptr;
        return reinterpret_cast<EncodeTiledFn>(p);
    }();
    return fn;
}
}  // namespace

namespace {
bool encode_2d(CUtensorMap* map, CUtensorMapDataType type, int64_t elem_bytes, const void* base,
               int64_t cols, int64_t rows, uint32_t box_cols, uint32_t box_rows,
               CUtensorMapSwizzle swizzle = CU_TENSOR_MAP_SWIZZLE_NONE) {
    EncodeTiledFn enc = encode_tiled();
    if (!enc) return false;
    const cuuint64_t dims[2] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows)};
    const cuuint64_t strides[1] = {static_cast<cuuint64_t>(cols * elem_bytes)};
    const cuuint32_t box[2] = {box_cols, box_rows};
    const cuuint32_t estr[2] = {1, 1};
    return enc(map, type, 2, const_cast<void*>(base), dims, strides, box, estr,
               CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle,
               CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}
}  // namespace

bool encode_bf16_2d(CUtensorMap* map, const void* base, int64_t cols, int64_t rows,
                    uint32_t box_cols, uint32_t box_rows) {
    return encode_2d(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, base, cols, rows, box_cols,
                     box_rows);
}

bool encode_u8_2d_swizzled(CUtensorMap* map, const void* base, int64_t cols, int64_t rows,
                           uint32_t box_rows) {
    return encode_2d(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, base, cols, rows, 128, box_rows,
                     CU_TENSOR_MAP_SWIZZLE_128B);
}

bool encode_bf16_2d_swizzled(CUtensorMap* map, const void* base, int64_t cols, int64_t rows,
                             uint32_t box_rows) {
    return encode_2d(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, base, cols, rows, 64, box_rows,
                     CU_TENSOR_MAP_SWIZZLE_128B);
}


unsigned int* device_status_word() {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0) return nullptr;
    if (dev < kMaxDevices) {
        unsigned int* p = g_status_ptr[dev].load(std::memory_order_acquire);
        if (p) return p;
    }
    void* p = nullptr;
    if (cudaGetSymbolAddress(&p, g_tkq_device_status) != cudaSuccess) return nullptr;
    if (dev < kMaxDevices)
        g_status_ptr[dev].store(static_cast<unsigned int*>(p), std::memory_order_release);
    return static_cast<unsigned int*>(p);
}

CheckTable& host_check_table() {
    thread_local CheckTable table{};
    return table;
}

namespace {
unsigned long long* bad_address_word() {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0) return nullptr;
    if (dev < kMaxDevices) {
        unsigned long long* p = g_bad_ptr[dev].load(std::memory_order_acquire);
        if (p) return p;
    }
    void* p = nullptr;
    if (cudaGetSymbolAddress(&p, g_tkq_bad_address) != cudaSuccess) return nullptr;
    if (dev < kMaxDevices)
        g_bad_ptr[dev].store(static_cast<unsigned long long*>(p), std::memory_order_release);
    return static_cast<unsigned long long*>(p);
}

#ifdef TKQ_CHECKED
// Adds one buffer to the call's table.
void register_one(Range r, bool output) {
    CheckTable& t = host_check_table();
    if (output) {
        uint64_t withhold = 0;
        if (const char* env = std::getenv("TKQ_CHECK_WITHHOLD"))
            withhold = std::strtoull(env, nullptr, 10);
        r.hi = r.hi - r.lo > withhold ? r.hi - withhold : r.lo;
    }
    if (r.hi <= r.lo || t.n >= kCheckMax) return;
    t.lo[t.n] = r.lo;
    t.hi[t.n] = r.hi;
    if (output) t.writable |= 1u << t.n;
    ++t.n;
}
#endif

// The buffers of the call about to launch, for the checked build's access
// checks (a no-op otherwise): inputs may be read, outputs read and written.
// Empty ranges (an absent optional buffer) are skipped.  The environment
// variable TKQ_CHECK_WITHHOLD=n (checked build only) leaves the last n bytes of
// every output out of the table, so that the kernels' stores there are refused
// and reported: the test of the checks themselves, with no access outside any
// allocation.
void register_call(std::initializer_list<Range> inputs, std::initializer_list<Range> outputs) {
#ifdef TKQ_CHECKED
    CheckTable& t = host_check_table();
    t = CheckTable{};
    for (const Range& r : inputs) register_one(r, false);
    for (const Range& r : outputs) register_one(r, true);
    t.status = device_status_word();
    t.bad = bad_address_word();
#else
    (void)inputs;
    (void)outputs;
#endif
}

// Per (kernel, device, threads, smem): resident blocks per SM.  The first
// launch on a device raises the kernel's dynamic shared-memory limit and asks
// the occupancy calculator; later launches reuse the answer, which keeps both
// calls off the per-launch host path.
struct OccKey {
    const void* kernel;
    int dev, threads;
    size_t smem;
    bool operator==(const OccKey& o) const {
        return kernel == o.kernel && dev == o.dev && threads == o.threads && smem == o.smem;
    }
};
struct OccKeyHash {
    size_t operator()(const OccKey& k) const {
        return std::hash<const void*>()(k.kernel) ^ (static_cast<size_t>(k.dev) << 1) ^
               (static_cast<size_t>(k.threads) << 8) ^ (k.smem << 20);
    }
};
std::mutex g_occ_mutex;
std::unordered_map<OccKey, int, OccKeyHash> g_occ;
std::unordered_map<OccKey, size_t, OccKeyHash> g_smem_limit;  // by kernel and device
}  // namespace

int persistent_grid(const void* kernel, int threads, size_t smem, int64_t blocks_needed) {
    int dev = 0;
    cudaGetDevice(&dev);
    const OccKey key{kernel, dev, threads, smem};
    int per_sm = 0;
    {
        std::lock_guard<std::mutex> lock(g_occ_mutex);
        auto it = g_occ.find(key);
        if (it != g_occ.end()) per_sm = it->second;
    }
    if (per_sm == 0) {
        // 48 KB need no permission, a kernel's static shared memory (33 KB at most) among them
        if (smem > 14 * 1024) {
            // the limit only goes up: a kernel may be launched with several sizes
            std::lock_guard<std::mutex> lock(g_occ_mutex);
            size_t& limit = g_smem_limit[OccKey{kernel, dev, 0, 0}];
            if (smem > limit) {
                cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                     static_cast<int>(smem));
                limit = smem;
            }
        }
        if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kernel, threads, smem) !=
                cudaSuccess ||
            per_sm <= 0)
            per_sm = 1;
        std::lock_guard<std::mutex> lock(g_occ_mutex);
        g_occ[key] = per_sm;
    }
    const int64_t cap = static_cast<int64_t>(num_sms()) * per_sm;
    const int64_t g = blocks_needed < cap ? blocks_needed : cap;
    return static_cast<int>(g > 0 ? g : 1);
}

}  // namespace tkq

namespace {

tkq_status check_common(int64_t T, int64_t C, int group, int fmt) {
    if (T < 0 || C <= 0) return TKQ_ERR_SHAPE;
    if (group != 128) return TKQ_ERR_GROUP;
    if (C % group) return TKQ_ERR_SHAPE;
    if (fmt != TKQ_FMT_E4M3 && fmt != TKQ_FMT_E5M2) return TKQ_ERR_FMT;
    // TMA row coordinates are 32-bit; C beyond 2^30 is far beyond one GPU
    if (T > INT32_MAX || C > (int64_t{1} << 30)) return TKQ_ERR_SHAPE;
    return TKQ_OK;
}

// One buffer of a call: its address, bytes and alignment.  Absent buffers
// (NULL) take no part.
struct Buffer {
    const void* p;
    int64_t bytes;
    uintptr_t align;
};

// Alignment of all buffers, and overlap of every output with every other
// buffer; then the call's table for the checked build.
template <size_t NI, size_t NO>
tkq_status check_buffers(const Buffer (&in)[NI], const Buffer (&out)[NO]) {
    for (const Buffer& b : in)
        if (b.p && !tkq::aligned(b.p, b.align)) return TKQ_ERR_ALIGN;
    for (const Buffer& b : out)
        if (b.p && !tkq::aligned(b.p, b.align)) return TKQ_ERR_ALIGN;
    const auto range = [](const Buffer& b) {
        return b.p ? tkq::span(b.p, b.bytes) : tkq::Range{0, 0};
    };
    for (size_t i = 0; i < NO; ++i) {
        for (const Buffer& b : in)
            if (tkq::overlap(range(out[i]), range(b))) return TKQ_ERR_ALIAS;
        for (size_t k = i + 1; k < NO; ++k)
            if (tkq::overlap(range(out[i]), range(out[k]))) return TKQ_ERR_ALIAS;
    }
#ifdef TKQ_CHECKED
    tkq::register_call({}, {});
    for (const Buffer& b : in) tkq::register_one(range(b), false);
    for (const Buffer& b : out) tkq::register_one(range(b), true);
#endif
    return TKQ_OK;
}

tkq_status launch_status(cudaError_t e) { return e == cudaSuccess ? TKQ_OK : TKQ_ERR_CUDA; }

constexpr unsigned kSfAllFlags =
    TKQ_SF_ROUND_POW2 | TKQ_SF_UE8M0_PACKED | TKQ_SF_COL_MAJOR | TKQ_Q_RECIPROCAL;

}  // namespace

extern "C" {

int64_t tkq_sf_bytes(int64_t T, int64_t groups_per_row, unsigned sf_flags) {
    if (T < 0 || groups_per_row < 0 || (sf_flags & ~kSfAllFlags)) return -1;
    const int64_t T4 = (T + 3) / 4 * 4;
    const int64_t W = (groups_per_row + 3) / 4;
    const bool cm = sf_flags & TKQ_SF_COL_MAJOR;
    if (sf_flags & TKQ_SF_UE8M0_PACKED) return (cm ? W * T4 : T * W) * 4;
    return (cm ? groups_per_row * T4 : T * groups_per_row) * 4;
}

namespace {
// Checks shared by the row casts: scale flags, scale-buffer alignment.
tkq_status check_sf(const void* sf, unsigned sf_flags) {
    if (sf_flags & ~kSfAllFlags) return TKQ_ERR_FLAGS;
    const uintptr_t a = (sf_flags & TKQ_SF_COL_MAJOR) ? 16 : 4;
    return tkq::aligned(sf, a) ? TKQ_OK : TKQ_ERR_ALIGN;
}
}  // namespace

tkq_status tkq_per_token_cast_ex(const void* x, void* out, void* sf, int64_t T, int64_t C,
                                 int group, int fmt, unsigned sf_flags, tkq_stream_t stream) {
    tkq_status st = check_common(T, C, group, fmt);
    if (st != TKQ_OK) return st;
    if (sf_flags & ~kSfAllFlags) return TKQ_ERR_FLAGS;
    if (T == 0) return TKQ_OK;
    if (!x || !out || !sf) return TKQ_ERR_NULL;
    if (!tkq::aligned(x, 16) || !tkq::aligned(out, 16)) return TKQ_ERR_ALIGN;
    if ((st = check_sf(sf, sf_flags)) != TKQ_OK) return st;
    const auto rx = tkq::span(x, T * C * 2), ro = tkq::span(out, T * C),
               rs = tkq::span(sf, tkq_sf_bytes(T, C / group, sf_flags));
    if (tkq::overlap(rx, ro) || tkq::overlap(rx, rs) || tkq::overlap(ro, rs)) return TKQ_ERR_ALIAS;
    tkq::register_call({rx}, {ro, rs});
    return launch_status(tkq::launch_per_token_cast(x, out, sf, T, C, fmt, sf_flags,
                                                    static_cast<cudaStream_t>(stream)));
}

tkq_status tkq_per_token_cast_f32(const float* x, void* out, void* sf, int64_t T, int64_t C,
                                  int group, int fmt, unsigned sf_flags, tkq_stream_t stream) {
    tkq_status st = check_common(T, C, group, fmt);
    if (st != TKQ_OK) return st;
    if (sf_flags & ~kSfAllFlags) return TKQ_ERR_FLAGS;
    if (T == 0) return TKQ_OK;
    if (!x || !out || !sf) return TKQ_ERR_NULL;
    if (!tkq::aligned(x, 16) || !tkq::aligned(out, 16)) return TKQ_ERR_ALIGN;
    if ((st = check_sf(sf, sf_flags)) != TKQ_OK) return st;
    const auto rx = tkq::span(x, T * C * 4), ro = tkq::span(out, T * C),
               rs = tkq::span(sf, tkq_sf_bytes(T, C / group, sf_flags));
    if (tkq::overlap(rx, ro) || tkq::overlap(rx, rs) || tkq::overlap(ro, rs)) return TKQ_ERR_ALIAS;
    tkq::register_call({rx}, {ro, rs});
    return launch_status(tkq::launch_per_token_cast_f32(x, out, sf, T, C, fmt, sf_flags,
                                                        static_cast<cudaStream_t>(stream)));
}

tkq_status tkq_per_token_cast(const void* x, void* out, float* sf, int64_t T, int64_t C,
                              int group, int fmt, tkq_stream_t stream) {
    return tkq_per_token_cast_ex(x, out, sf, T, C, group, fmt, 0u, stream);
}

namespace {
// The SwiGLU clamp arguments: a finite bound > 0 and, if given, an 8-byte
// aligned counter that overlaps none of the call's other buffers.
tkq_status check_clamp(float clamp, const uint64_t* count, const tkq::Range* others, int n) {
    if (!(clamp > 0.0f && clamp < INFINITY)) return TKQ_ERR_VALUE;
    if (!count) return TKQ_OK;
    if (!tkq::aligned(count, 8)) return TKQ_ERR_ALIGN;
    const auto rc = tkq::span(count, 8);
    for (int i = 0; i < n; ++i)
        if (tkq::overlap(rc, others[i])) return TKQ_ERR_ALIAS;
    return TKQ_OK;
}

tkq_status swiglu_cast_impl(const void* x, const float* w, void* out, void* sf, int64_t T,
                            int64_t H, int group, int fmt, unsigned sf_flags, const float* clamp,
                            uint64_t* clamp_count, tkq_stream_t stream) {
    tkq_status st = check_common(T, H, group, fmt);
    if (st != TKQ_OK) return st;
    if (sf_flags & ~kSfAllFlags) return TKQ_ERR_FLAGS;
    if (clamp && !(*clamp > 0.0f && *clamp < INFINITY)) return TKQ_ERR_VALUE;
    if (T == 0) return TKQ_OK;
    if (!x || !out || !sf) return TKQ_ERR_NULL;
    if (!tkq::aligned(x, 16) || !tkq::aligned(out, 16) || (w && !tkq::aligned(w, 4)))
        return TKQ_ERR_ALIGN;
    if ((st = check_sf(sf, sf_flags)) != TKQ_OK) return st;
    const auto rx = tkq::span(x, T * H * 4), ro = tkq::span(out, T * H),
               rs = tkq::span(sf, tkq_sf_bytes(T, H / group, sf_flags));
    if (tkq::overlap(rx, ro) || tkq::overlap(rx, rs) || tkq::overlap(ro, rs)) return TKQ_ERR_ALIAS;
    const auto rw = w ? tkq::span(w, T * 4) : tkq::Range{0, 0};
    if (tkq::overlap(rw, ro) || tkq::overlap(rw, rs)) return TKQ_ERR_ALIAS;
    if (clamp) {
        const tkq::Range others[4] = {rx, ro, rs, rw};
        if ((st = check_clamp(*clamp, clamp_count, others, 4)) != TKQ_OK) return st;
    }
    const auto rc = clamp && clamp_count ? tkq::span(clamp_count, 8) : tkq::Range{0, 0};
    tkq::register_call({rx, rw}, {ro, rs, rc});
    return launch_status(tkq::launch_swiglu_cast(
        x, w, out, sf, T, H, fmt, sf_flags, clamp,
        reinterpret_cast<unsigned long long*>(clamp_count), static_cast<cudaStream_t>(stream)));
}
}  // namespace

tkq_status tkq_swiglu_cast_ex(const void* x, const float* w, void* out, void* sf, int64_t T,
                              int64_t H, int group, int fmt, unsigned sf_flags,
                              tkq_stream_t stream) {
    return swiglu_cast_impl(x, w, out, sf, T, H, group, fmt, sf_flags, nullptr, nullptr, stream);
}

tkq_status tkq_swiglu_cast(const void* x, const float* w, void* out, float* sf, int64_t T,
                           int64_t H, int group, int fmt, tkq_stream_t stream) {
    return swiglu_cast_impl(x, w, out, sf, T, H, group, fmt, 0u, nullptr, nullptr, stream);
}

tkq_status tkq_swiglu_cast_clamp(const void* x, const float* w, void* out, void* sf, int64_t T,
                                 int64_t H, int group, int fmt, unsigned sf_flags,
                                 float clamp_value, uint64_t* clamp_count, tkq_stream_t stream) {
    return swiglu_cast_impl(x, w, out, sf, T, H, group, fmt, sf_flags, &clamp_value,
                            clamp_count, stream);
}

tkq_status tkq_swiglu_backward_cast_ex(const void* x, const void* dy, const float* w, void* out,
                                       void* sf, int64_t T, int64_t H, int group, int fmt,
                                       unsigned sf_flags, tkq_stream_t stream) {
    tkq_status st = check_common(T, H, group, fmt);
    if (st != TKQ_OK) return st;
    if (sf_flags & ~kSfAllFlags) return TKQ_ERR_FLAGS;
    if (T == 0) return TKQ_OK;
    if (!x || !dy || !out || !sf) return TKQ_ERR_NULL;
    if (!tkq::aligned(x, 16) || !tkq::aligned(dy, 16) || !tkq::aligned(out, 16) ||
        (w && !tkq::aligned(w, 4)))
        return TKQ_ERR_ALIGN;
    if ((st = check_sf(sf, sf_flags)) != TKQ_OK) return st;
    const auto ro = tkq::span(out, T * 2 * H),
               rs = tkq::span(sf, tkq_sf_bytes(T, 2 * H / group, sf_flags));
    const tkq::Range inputs[3] = {tkq::span(x, T * H * 4), tkq::span(dy, T * H * 2),
                                  w ? tkq::span(w, T * 4) : tkq::Range{0, 0}};
    if (tkq::overlap(ro, rs)) return TKQ_ERR_ALIAS;
    for (const auto& in : inputs)
        if (tkq::overlap(in, ro) || tkq::overlap(in, rs)) return TKQ_ERR_ALIAS;
    tkq::register_call({inputs[0], inputs[1], inputs[2]}, {ro, rs});
    return launch_status(tkq::launch_swiglu_backward_cast(x, dy, w, out, sf, T, H, fmt, sf_flags,
                                                          static_cast<cudaStream_t>(stream)));
}

tkq_status tkq_swiglu_backward_cast(const void* x, const void* dy, const float* w, void* out,
                                    float* sf, int64_t T, int64_t H, int group, int fmt,
                                    tkq_stream_t stream) {
    return tkq_swiglu_backward_cast_ex(x, dy, w, out, sf, T, H, group, fmt, 0u, stream);
}

namespace {
tkq_status swiglu_cast_t_impl(const void* x, const float* w, void* out, void* sf, void* out_t,
                              void* sf_t, int64_t T, int64_t H, int group, int fmt,
                              unsigned sf_flags, const float* clamp, uint64_t* clamp_count,
                              tkq_stream_t stream) {
    tkq_status st = check_common(T, H, group, fmt);
    if (st != TKQ_OK) return st;
    if (T % group) return TKQ_ERR_SHAPE;
    if (sf_flags & ~kSfAllFlags) return TKQ_ERR_FLAGS;
    if (clamp && !(*clamp > 0.0f && *clamp < INFINITY)) return TKQ_ERR_VALUE;
    if (T == 0) return TKQ_OK;
    // TMA box coordinates are 32-bit
    if (H > (int64_t{1} << 30) || T > INT32_MAX) return TKQ_ERR_SHAPE;
    if (!x || !out || !sf || !out_t || !sf_t) return TKQ_ERR_NULL;
    if (!tkq::aligned(x, 16) || !tkq::aligned(out, 16) || !tkq::aligned(out_t, 16) ||
        (w && !tkq::aligned(w, 4)))
        return TKQ_ERR_ALIGN;
    if ((st = check_sf(sf, sf_flags)) != TKQ_OK || (st = check_sf(sf_t, sf_flags)) != TKQ_OK)
        return st;
    const tkq::Range r[5] = {tkq::span(x, T * H * 4), tkq::span(out, T * H),
                             tkq::span(sf, tkq_sf_bytes(T, H / group, sf_flags)),
                             tkq::span(out_t, T * H),
                             tkq::span(sf_t, tkq_sf_bytes(H, T / group, sf_flags))};
    for (int i = 0; i < 5; ++i)
        for (int k = i + 1; k < 5; ++k)
            if (tkq::overlap(r[i], r[k])) return TKQ_ERR_ALIAS;
    const auto rw = w ? tkq::span(w, T * 4) : tkq::Range{0, 0};
    for (int i = 1; i < 5; ++i)
        if (tkq::overlap(rw, r[i])) return TKQ_ERR_ALIAS;
    if (clamp) {
        const tkq::Range others[6] = {r[0], r[1], r[2], r[3], r[4], rw};
        if ((st = check_clamp(*clamp, clamp_count, others, 6)) != TKQ_OK) return st;
    }
    const auto rc = clamp && clamp_count ? tkq::span(clamp_count, 8) : tkq::Range{0, 0};
    tkq::register_call({r[0], rw}, {r[1], r[2], r[3], r[4], rc});
    return launch_status(tkq::launch_swiglu_cast_t(
        x, w, out, static_cast<float*>(sf), out_t, static_cast<float*>(sf_t), T, H, fmt, sf_flags,
        clamp, reinterpret_cast<unsigned long long*>(clamp_count),
        static_cast<cudaStream_t>(stream)));
}
}  // namespace

tkq_status tkq_swiglu_cast_t(const void* x, const float* w, void* out, float* sf, void* out_t,
                             float* sf_t, int64_t T, int64_t H, int group, int fmt,
                             tkq_stream_t stream) {
    return swiglu_cast_t_impl(x, w, out, sf, out_t, sf_t, T, H, group, fmt, 0u, nullptr,
                              nullptr, stream);
}

tkq_status tkq_swiglu_cast_t_ex(const void* x, const float* w, void* out, void* sf, void* out_t,
                                void* sf_t, int64_t T, int64_t H, int group, int fmt,
                                unsigned sf_flags, tkq_stream_t stream) {
    return swiglu_cast_t_impl(x, w, out, sf, out_t, sf_t, T, H, group, fmt, sf_flags, nullptr,
                              nullptr, stream);
}

tkq_status tkq_swiglu_cast_t_clamp(const void* x, const float* w, void* out, void* sf,
                                   void* out_t, void* sf_t, int64_t T, int64_t H, int group,
                                   int fmt, unsigned sf_flags, float clamp_value,
                                   uint64_t* clamp_count, tkq_stream_t stream) {
    return swiglu_cast_t_impl(x, w, out, sf, out_t, sf_t, T, H, group, fmt, sf_flags,
                              &clamp_value, clamp_count, stream);
}

tkq_status tkq_per_channel_cast(const void* x, void* out, float* sf, int64_t T, int64_t C,
                                int group, int fmt, int transpose, tkq_stream_t stream) {
    tkq_status st = check_common(T, C, group, fmt);
    if (st != TKQ_OK) return st;
    if (T % group) return TKQ_ERR_SHAPE;
    if (T == 0) return TKQ_OK;
    if (!x || !out || !sf) return TKQ_ERR_NULL;
    if (!tkq::aligned(x, 16) || !tkq::aligned(out, 16) || !tkq::aligned(sf, 4))
        return TKQ_ERR_ALIGN;
    const auto rx = tkq::span(x, T * C * 2), ro = tkq::span(out, T * C),
               rs = tkq::span(sf, (T / group) * C * 4);
    if (tkq::overlap(rx, ro) || tkq::overlap(rx, rs) || tkq::overlap(ro, rs)) return TKQ_ERR_ALIAS;
    tkq::register_call({rx}, {ro, rs});
    return launch_status(tkq::launch_per_channel_cast(x, out, sf, T, C, fmt, transpose != 0,
                                                      static_cast<cudaStream_t>(stream)));
}

tkq_status tkq_per_block_cast(const void* x, void* out, float* sf, int64_t T, int64_t C,
                              int block, int fmt, tkq_stream_t stream) {
    tkq_status st = check_common(T, C, block, fmt);
    if (st != TKQ_OK) return st;
    if (T == 0) return TKQ_OK;
    if (!x || !out || !sf) return TKQ_ERR_NULL;
    if (!tkq::aligned(x, 16) || !tkq::aligned(out, 16) || !tkq::aligned(sf, 4))
        return TKQ_ERR_ALIGN;
    const auto rx = tkq::span(x, T * C * 2), ro = tkq::span(out, T * C),
               rs = tkq::span(sf, (T + block - 1) / block * (C / block) * 4);
    if (tkq::overlap(rx, ro) || tkq::overlap(rx, rs) || tkq::overlap(ro, rs)) return TKQ_ERR_ALIAS;
    tkq::register_call({rx}, {ro, rs});
    return launch_status(
        tkq::launch_per_block_cast(x, out, sf, T, C, fmt, static_cast<cudaStream_t>(stream)));
}

tkq_status tkq_cast_back(const void* codes, const float* sf, void* out, int64_t T, int64_t C,
                         int group_rows, int group_cols, int fmt, int out_dtype,
                         tkq_stream_t stream) {
    if (T < 0 || C <= 0 || C % 128 || T > INT32_MAX || C > (int64_t{1} << 30))
        return TKQ_ERR_SHAPE;
    const bool per_token = group_rows == 1 && group_cols == 128;
    const bool per_channel = group_rows == 128 && group_cols == 1;
    const bool per_block = group_rows == 128 && group_cols == 128;
    if (!per_token && !per_channel && !per_block) return TKQ_ERR_GROUP;
    if (fmt != TKQ_FMT_E4M3 && fmt != TKQ_FMT_E5M2) return TKQ_ERR_FMT;
    if (out_dtype != TKQ_OUT_F32 && out_dtype != TKQ_OUT_BF16) return TKQ_ERR_FMT;
    if (T == 0) return TKQ_OK;
    if (!codes || !sf || !out) return TKQ_ERR_NULL;
    if (!tkq::aligned(codes, 16) || !tkq::aligned(out, 16) ||
        !tkq::aligned(sf, group_cols == 1 ? 16 : 4))
        return TKQ_ERR_ALIGN;
    const int64_t out_bytes = T * C * (out_dtype == TKQ_OUT_F32 ? 4 : 2);
    const int64_t sf_bytes = (T + group_rows - 1) / group_rows * (C / group_cols) * 4;
    const auto ro = tkq::span(out, out_bytes), rq = tkq::span(codes, T * C),
               rs = tkq::span(sf, sf_bytes);
    if (tkq::overlap(ro, rq) || tkq::overlap(ro, rs)) return TKQ_ERR_ALIAS;
    tkq::register_call({rq, rs}, {ro});
    return launch_status(tkq::launch_cast_back(codes, sf, out, T, C, group_rows, group_cols, fmt,
                                               out_dtype == TKQ_OUT_BF16,
                                               static_cast<cudaStream_t>(stream)));
}

namespace {
tkq_status check_route(int64_t T, int64_t E, int64_t ld, int dtype, int k, unsigned flags,
                       float scale) {
    if (T < 0 || T > INT32_MAX || E <= 0 || E > 1024 || ld < E || ld > (int64_t{1} << 28) ||
        k <= 0 || k > 32 || k > E)
        return TKQ_ERR_SHAPE;
    if (dtype != TKQ_OUT_F32 && dtype != TKQ_OUT_BF16) return TKQ_ERR_FMT;
    if (flags & ~(TKQ_ROUTE_SIGMOID | TKQ_ROUTE_RENORM)) return TKQ_ERR_FLAGS;
    if (!std::isfinite(scale)) return TKQ_ERR_VALUE;
    return TKQ_OK;
}

tkq::RouteShape route_shape(int64_t E, int dtype, int k, unsigned flags, float scale) {
    tkq::RouteShape s = {};
    s.E = static_cast<int>(E);
    s.k = k;
    s.groups = s.topk_groups = s.group_top = 1;
    s.sigmoid = flags & TKQ_ROUTE_SIGMOID;
    s.renorm = flags & TKQ_ROUTE_RENORM;
    s.bf16 = dtype == TKQ_OUT_BF16;
    s.scale = scale;
    return s;
}

// Bytes of T rows of E elements with a row stride of ld elements.
int64_t strided_bytes(int64_t T, int64_t E, int64_t ld, int64_t item) {
    return ((T - 1) * ld + E) * item;
}
}  // namespace

tkq_status tkq_route_topk(const void* logits, const float* bias, int32_t* ids, float* weights,
                          int32_t* counts, int64_t T, int64_t E, int64_t ld, int dtype, int k,
                          int n_groups, int topk_groups, int group_top, unsigned route_flags,
                          float scale, tkq_stream_t stream) {
    tkq_status st = check_route(T, E, ld, dtype, k, route_flags, scale);
    if (st != TKQ_OK) return st;
    if (n_groups <= 0 || n_groups > 32 || E % n_groups || topk_groups <= 0 ||
        topk_groups > n_groups)
        return TKQ_ERR_SHAPE;
    if (group_top != 1 && group_top != 2) return TKQ_ERR_VALUE;
    if (T == 0) return TKQ_OK;
    if (!logits || !ids || !weights) return TKQ_ERR_NULL;
    const int64_t item = dtype == TKQ_OUT_BF16 ? 2 : 4;
    const Buffer in[] = {{logits, strided_bytes(T, E, ld, item), static_cast<uintptr_t>(item)},
                         {bias, E * 4, 4}};
    const Buffer out[] = {{ids, T * k * 4, 4}, {weights, T * k * 4, 4}, {counts, E * 4, 4}};
    if ((st = check_buffers(in, out)) != TKQ_OK) return st;
    tkq::RouteShape s = route_shape(E, dtype, k, route_flags, scale);
    s.groups = n_groups;
    s.topk_groups = topk_groups;
    s.group_top = group_top;
    return launch_status(tkq::launch_route_topk(logits, bias, ids, weights, counts, T, ld, s,
                                                static_cast<cudaStream_t>(stream)));
}

tkq_status tkq_route_topk_backward(const void* logits, const int32_t* ids, const float* dweights,
                                   void* dlogits, int64_t T, int64_t E, int64_t ld, int dtype,
                                   int k, unsigned route_flags, float scale, tkq_stream_t stream) {
    tkq_status st = check_route(T, E, ld, dtype, k, route_flags, scale);
    if (st != TKQ_OK) return st;
    if (T == 0) return TKQ_OK;
    if (!logits || !ids || !dweights || !dlogits) return TKQ_ERR_NULL;
    const int64_t item = dtype == TKQ_OUT_BF16 ? 2 : 4;
    const uintptr_t al = static_cast<uintptr_t>(item);
    const Buffer in[] = {{logits, strided_bytes(T, E, ld, item), al},
                         {ids, T * k * 4, 4},
                         {dweights, T * k * 4, 4}};
    const Buffer out[] = {{dlogits, T * E * item, al}};
    if ((st = check_buffers(in, out)) != TKQ_OK) return st;
    return launch_status(tkq::launch_route_topk_backward(
        logits, ids, dweights, dlogits, T, ld, route_shape(E, dtype, k, route_flags, scale),
        static_cast<cudaStream_t>(stream)));
}

tkq_status tkq_swiglu_cast_checkpoint(const void* x, const float* w, void* out, void* sf,
                                      void* ckpt, float* ckpt_sf, int64_t T, int64_t H, int group,
                                      int fmt, int ckpt_fmt, unsigned sf_flags,
                                      tkq_stream_t stream) {
    tkq_status st = check_common(T, H, group, fmt);
    if (st != TKQ_OK || (st = check_common(T, H, group, ckpt_fmt)) != TKQ_OK) return st;
    if (sf_flags & ~kSfAllFlags) return TKQ_ERR_FLAGS;
    if (T == 0) return TKQ_OK;
    if (!x || !out || !sf || !ckpt || !ckpt_sf) return TKQ_ERR_NULL;
    const Buffer ins[] = {{x, T * H * 4, 16}, {w, T * 4, 4}};
    const Buffer outs[] = {
        {out, T * H, 16},
        {sf, tkq_sf_bytes(T, H / group, sf_flags), (sf_flags & TKQ_SF_COL_MAJOR) ? 16u : 4u},
        {ckpt, T * 2 * H, 16},
        {ckpt_sf, T * 2 * (H / group) * 4, 4}};
    if ((st = check_buffers(ins, outs)) != TKQ_OK) return st;
    return launch_status(tkq::launch_swiglu_save(x, w, out, sf, ckpt, ckpt_sf, T, H, fmt, ckpt_fmt,
                                                 sf_flags, static_cast<cudaStream_t>(stream)));
}

namespace {
// fmt: an FP8 format, or 2 for bf16 gradients (no dx_sf).
tkq_status swiglu_restore_impl(const void* ckpt, const float* ckpt_sf, const void* dy,
                               const float* w, void* dx, void* dx_sf, void* y, float* dw,
                               int64_t T, int64_t H, int group, int ckpt_fmt, int fmt,
                               unsigned sf_flags, tkq_stream_t stream) {
    const bool cast = fmt != 2;
    tkq_status st = check_common(T, H, group, ckpt_fmt);
    if (st != TKQ_OK) return st;
    if (sf_flags & ~kSfAllFlags) return TKQ_ERR_FLAGS;
    if (T == 0) return TKQ_OK;
    if (!ckpt || !ckpt_sf || !dy || !dx || (cast && !dx_sf)) return TKQ_ERR_NULL;
    const Buffer ins[] = {{ckpt, T * 2 * H, 16},
                          {ckpt_sf, T * 2 * (H / group) * 4, 4},
                          {dy, T * H * 2, 16},
                          {w, T * 4, 4}};
    const Buffer outs[] = {{dx, T * 2 * H * (cast ? 1 : 2), 16},
                           {cast ? dx_sf : nullptr, tkq_sf_bytes(T, 2 * (H / group), sf_flags),
                            (sf_flags & TKQ_SF_COL_MAJOR) ? 16u : 4u},
                           {y, T * H * 2, 16},
                           {dw, T * 4, 4}};
    if ((st = check_buffers(ins, outs)) != TKQ_OK) return st;
    return launch_status(tkq::launch_swiglu_restore(ckpt, ckpt_sf, dy, w, dx, dx_sf, y, dw, T, H,
                                                    ckpt_fmt, fmt, sf_flags,
                                                    static_cast<cudaStream_t>(stream)));
}
}  // namespace

tkq_status tkq_swiglu_checkpoint_backward(const void* ckpt, const float* ckpt_sf, const void* dy,
                                          const float* w, void* dx, void* y, float* dw, int64_t T,
                                          int64_t H, int group, int ckpt_fmt, tkq_stream_t stream) {
    return swiglu_restore_impl(ckpt, ckpt_sf, dy, w, dx, nullptr, y, dw, T, H, group, ckpt_fmt, 2,
                               0u, stream);
}

tkq_status tkq_swiglu_checkpoint_backward_cast(const void* ckpt, const float* ckpt_sf,
                                               const void* dy, const float* w, void* dx,
                                               void* dx_sf, void* y, float* dw, int64_t T,
                                               int64_t H, int group, int ckpt_fmt, int fmt,
                                               unsigned sf_flags, tkq_stream_t stream) {
    if (const tkq_status st = check_common(T, H, group, fmt)) return st;
    return swiglu_restore_impl(ckpt, ckpt_sf, dy, w, dx, dx_sf, y, dw, T, H, group, ckpt_fmt, fmt,
                               sf_flags, stream);
}

namespace {
constexpr unsigned kNormAllFlags = TKQ_NORM_POST | TKQ_NORM_PRE | TKQ_NORM_RES_F32;
constexpr int64_t kNormMaxChannels = 16384;

tkq_status check_norm(int64_t T, int64_t C, unsigned norm_flags, float res_scale) {
    if (T < 0 || T > INT32_MAX || C <= 0 || C > kNormMaxChannels || C % 128) return TKQ_ERR_SHAPE;
    if (norm_flags & ~kNormAllFlags) return TKQ_ERR_FLAGS;
    if (!std::isfinite(res_scale)) return TKQ_ERR_VALUE;
    return TKQ_OK;
}
}  // namespace

tkq_status tkq_residual_norm_cast(const void* r, const void* h, const float* w_post,
                                  const void* gate, const float* w_pre, void* r_out, void* out,
                                  void* sf, void* x_out, float* rstd_post, float* rstd_pre,
                                  int64_t T, int64_t C, int group, int fmt, unsigned sf_flags,
                                  unsigned norm_flags, float res_scale, float eps,
                                  tkq_stream_t stream) {
    tkq_status st = check_norm(T, C, norm_flags, res_scale);
    if (st != TKQ_OK || (st = check_common(T, C, group, fmt)) != TKQ_OK) return st;
    if (!(eps >= 0.0f && std::isfinite(eps))) return TKQ_ERR_VALUE;
    const bool post = norm_flags & TKQ_NORM_POST, pre = norm_flags & TKQ_NORM_PRE;
    if (sf_flags & ~kSfAllFlags) return TKQ_ERR_FLAGS;
    if (T == 0) return TKQ_OK;
    if ((!h && (post || w_post || gate || r_out)) || (!post && rstd_post) ||
        (!pre && (w_pre || out || x_out || rstd_pre)) || (!h && !pre))
        return TKQ_ERR_FLAGS;
    if (!r || (h && !r_out) || (pre && !out && !x_out) || !out != !sf) return TKQ_ERR_NULL;
    const int64_t n = T * C, rb = norm_flags & TKQ_NORM_RES_F32 ? 4 : 2;
    const Buffer ins[] = {{r, n * rb, 16},
                          {h, n * 2, 16},
                          {w_post, C * 4, 16},
                          {gate, n * 2, 16},
                          {w_pre, C * 4, 16}};
    const Buffer outs[] = {
        {r_out, n * rb, 16},
        {out, n, 16},
        {sf, tkq_sf_bytes(T, C / group, sf_flags), (sf_flags & TKQ_SF_COL_MAJOR) ? 16u : 4u},
        {x_out, n * 2, 16},
        {rstd_post, T * 4, 4},
        {rstd_pre, T * 4, 4}};
    if ((st = check_buffers(ins, outs)) != TKQ_OK) return st;
    const tkq::ResidualNorm a = {r,  h,   gate,  w_post,    w_pre,    r_out, out, sf,
                                 x_out, rstd_post, rstd_pre, T, C, res_scale, eps, post,
                                 pre, rb == 4};
    return launch_status(
        tkq::launch_residual_norm(a, fmt, sf_flags, static_cast<cudaStream_t>(stream)));
}

int64_t tkq_residual_norm_workspace(int64_t T, int64_t C) {
    if (check_norm(T, C, 0u, 0.0f) != TKQ_OK) return -1;
    return tkq::residual_norm_parts(T, C) * 2 * C * 4;
}

tkq_status tkq_residual_norm_backward(const void* dr, const void* dx, const void* r, const void* h,
                                      const float* w_post, const void* gate, const float* w_pre,
                                      const float* rstd_post, const float* rstd_pre, void* dr_out,
                                      void* dh, void* dgate, float* dw_post, float* dw_pre,
                                      void* workspace, int64_t T, int64_t C, unsigned norm_flags,
                                      float res_scale, tkq_stream_t stream) {
    tkq_status st = check_norm(T, C, norm_flags, res_scale);
    if (st != TKQ_OK) return st;
    const bool post = norm_flags & TKQ_NORM_POST, pre = norm_flags & TKQ_NORM_PRE;
    if (T == 0) return TKQ_OK;
    if ((!h && (post || w_post || gate || dh || dgate || dw_post)) || (!gate && dgate) ||
        (!pre && (dx || w_pre || dw_pre)))
        return TKQ_ERR_FLAGS;
    if (!dr_out || (!dr && !dx) || (h && !dh) || (gate && !dgate) || (post && !rstd_post) ||
        (pre && (!dx || !r || !rstd_pre)) || ((dw_post || dw_pre) && !workspace))
        return TKQ_ERR_NULL;
    const int64_t n = T * C, rb = norm_flags & TKQ_NORM_RES_F32 ? 4 : 2;
    const Buffer ins[] = {{dr, n * rb, 16},
                          {dx, n * 2, 16},
                          {pre ? r : nullptr, n * rb, 16},
                          {h, n * 2, 16},
                          {w_post, C * 4, 16},
                          {gate, n * 2, 16},
                          {w_pre, C * 4, 16},
                          {post ? rstd_post : nullptr, T * 4, 4},
                          {pre ? rstd_pre : nullptr, T * 4, 4}};
    const Buffer outs[] = {{dr_out, n * rb, 16}, {dh, n * 2, 16},
                           {dgate, n * 2, 16},   {dw_post, C * 4, 16},
                           {dw_pre, C * 4, 16},  {dw_post || dw_pre ? workspace : nullptr,
                                                  tkq_residual_norm_workspace(T, C), 16}};
    if ((st = check_buffers(ins, outs)) != TKQ_OK) return st;
    const tkq::ResidualNormGrad a = {dx,     dr, r,     h,       gate,   w_post,    w_pre,
                                     rstd_post, rstd_pre, dr_out, dh, dgate, dw_post, dw_pre,
                                     workspace, T, C, res_scale, post, rb == 4};
    return launch_status(
        tkq::launch_residual_norm_backward(a, static_cast<cudaStream_t>(stream)));
}

namespace {
// The pairs and rows of tokens in expert order.
tkq_status check_pairs(int64_t T, int k, int64_t E, int64_t R) {
    if (T < 0 || k <= 0 || k > 32 || T > (int64_t{1} << 30) / k || E <= 0 || E > 1024 || R < 0 ||
        R > INT32_MAX)
        return TKQ_ERR_SHAPE;
    return TKQ_OK;
}

tkq_status check_row_channels(int64_t C, int group) {
    if (group != 128) return TKQ_ERR_GROUP;
    return C <= 0 || C % 128 || C > (int64_t{1} << 20) ? TKQ_ERR_SHAPE : TKQ_OK;
}

bool fp8_fmt(int fmt) { return fmt == TKQ_FMT_E4M3 || fmt == TKQ_FMT_E5M2; }
}  // namespace

int64_t tkq_expert_rows(int64_t T, int k, int64_t E, int align) {
    if (check_pairs(T, k, E, 0) != TKQ_OK || align <= 0 || align > 1024) return -1;
    const int64_t P = T * k;
    return (P + (E < P ? E : P) * (align - 1)) / align * align;
}

tkq_status tkq_expert_order(const int32_t* ids, int32_t* slots, int32_t* rows, int32_t* offsets,
                            int64_t T, int k, int64_t E, int align, int64_t R,
                            tkq_stream_t stream) {
    tkq_status st = check_pairs(T, k, E, R);
    if (st != TKQ_OK) return st;
    const int64_t need = tkq_expert_rows(T, k, E, align);
    if (need < 0 || R < need) return TKQ_ERR_SHAPE;
    if ((T && (!ids || !slots)) || (R && !rows) || !offsets) return TKQ_ERR_NULL;
    const Buffer in[] = {{ids, T * k * 4, 4}};
    const Buffer out[] = {{slots, T * k * 4, 4}, {rows, R * 4, 4}, {offsets, (E + 1) * 4, 4}};
    if ((st = check_buffers(in, out)) != TKQ_OK) return st;
    return launch_status(tkq::launch_expert_order(ids, slots, rows, offsets, T * k,
                                                  static_cast<int>(E), align, R,
                                                  static_cast<cudaStream_t>(stream)));
}

tkq_status tkq_expert_gather(const void* x, const float* x_sf, const int32_t* slots,
                             const int32_t* rows, const int32_t* offsets, const float* weights,
                             void* out, float* out_sf, float* row_weights, int64_t T, int64_t C,
                             int group, int k, int64_t E, int64_t R, int form, int fmt,
                             tkq_stream_t stream) {
    tkq_status st = check_pairs(T, k, E, R);
    if (st != TKQ_OK || (st = check_row_channels(C, group)) != TKQ_OK) return st;
    if (form != TKQ_ROWS_BF16 && form != TKQ_ROWS_CAST && form != TKQ_ROWS_CODES)
        return TKQ_ERR_FLAGS;
    if (!fp8_fmt(fmt)) return TKQ_ERR_FMT;
    if (T == 0 || R == 0) return TKQ_OK;
    const bool codes_in = form == TKQ_ROWS_CODES, codes_out = form != TKQ_ROWS_BF16;
    if (!x || !slots || !rows || !offsets || !out || codes_in != !!x_sf || codes_out != !!out_sf ||
        !weights != !row_weights)
        return TKQ_ERR_NULL;
    const int64_t G = C / 128;
    const Buffer in[] = {{x, T * C * (codes_in ? 1 : 2), 16}, {x_sf, T * G * 4, 4},
                         {slots, T * k * 4, 4},               {rows, R * 4, 4},
                         {offsets, (E + 1) * 4, 4},           {weights, T * k * 4, 4}};
    // bf16 rows are stored in whole sectors of 32 bytes
    const Buffer outs[] = {{out, R * C * (codes_out ? 1 : 2), codes_out ? 16u : 32u},
                           {out_sf, R * G * 4, 4},
                           {row_weights, R * 4, 4}};
    if ((st = check_buffers(in, outs)) != TKQ_OK) return st;
    const tkq::ExpertGather a = {x, x_sf, slots, rows, offsets, weights, out, out_sf, row_weights,
                                 T, C, R, k, static_cast<int>(E), form, fmt};
    return launch_status(tkq::launch_expert_gather(a, static_cast<cudaStream_t>(stream)));
}

tkq_status tkq_expert_reduce(const void* y, const int32_t* slots, const float* weights,
                             const float* row_values, void* out, float* values, int64_t T,
                             int64_t C, int group, int k, int64_t R, int out_dtype,
                             tkq_stream_t stream) {
    tkq_status st = check_pairs(T, k, 1, R);
    if (st != TKQ_OK || (st = check_row_channels(C, group)) != TKQ_OK) return st;
    if (out_dtype != TKQ_OUT_F32 && out_dtype != TKQ_OUT_BF16) return TKQ_ERR_FMT;
    if (T == 0) return TKQ_OK;
    if ((R && !y) || !slots || !out || (R && !row_values != !values)) return TKQ_ERR_NULL;
    const bool f32 = out_dtype == TKQ_OUT_F32;
    const Buffer in[] = {{y, R * C * 2, 16},
                         {slots, T * k * 4, 4},
                         {weights, T * k * 4, 4},
                         {row_values, R * 4, 4}};
    const Buffer outs[] = {{out, T * C * (f32 ? 4 : 2), 16}, {values, T * k * 4, 4}};
    if ((st = check_buffers(in, outs)) != TKQ_OK) return st;
    return launch_status(tkq::launch_expert_reduce(y, slots, weights, row_values, out, values, T, C,
                                                   k, R, f32, static_cast<cudaStream_t>(stream)));
}

tkq_status tkq_expert_reduce_backward(const void* dout, const void* y, const int32_t* slots,
                                      const int32_t* rows, const int32_t* offsets,
                                      const float* weights, void* dy, float* dy_sf,
                                      float* dweights, int64_t T, int64_t C, int group, int k,
                                      int64_t E, int64_t R, int form, int fmt,
                                      tkq_stream_t stream) {
    tkq_status st = check_pairs(T, k, E, R);
    if (st != TKQ_OK || (st = check_row_channels(C, group)) != TKQ_OK) return st;
    if (form != TKQ_ROWS_BF16 && form != TKQ_ROWS_CAST) return TKQ_ERR_FLAGS;
    if (!fp8_fmt(fmt)) return TKQ_ERR_FMT;
    if (T == 0) return TKQ_OK;
    const bool cast = form == TKQ_ROWS_CAST;
    if (!dout || !slots || !offsets || !weights || !dweights ||
        (R && (!y || !rows || !dy || cast != !!dy_sf)))
        return TKQ_ERR_NULL;
    const int64_t G = C / 128;
    const Buffer in[] = {{dout, T * C * 2, 16}, {y, R * C * 2, 16},        {slots, T * k * 4, 4},
                         {rows, R * 4, 4},      {offsets, (E + 1) * 4, 4}, {weights, T * k * 4, 4}};
    const Buffer outs[] = {{dy, R * C * (cast ? 1 : 2), 16},
                           {cast ? dy_sf : nullptr, R * G * 4, 4},
                           {dweights, T * k * 4, 4}};
    if ((st = check_buffers(in, outs)) != TKQ_OK) return st;
    const tkq::ExpertReduceGrad a = {dout, y, slots, rows, offsets, weights, dy, dy_sf, dweights,
                                     T, C, R, k, static_cast<int>(E), cast ? fmt : 2};
    return launch_status(tkq::launch_expert_reduce_backward(a, static_cast<cudaStream_t>(stream)));
}

namespace {
// Sizes of the experts' products; E * N * K stays far from 2^63.
tkq_status check_product(int64_t R, int64_t E, int64_t N, int64_t K, int group) {
    if (group != 128) return TKQ_ERR_GROUP;
    const int64_t most = int64_t{1} << 20;
    if (R < 0 || R > INT32_MAX - 1024 || E <= 0 || E > 1024 || N <= 0 || N > most || N % 128 || K <= 0 ||
        K > most || K % 128 || E * N > INT32_MAX - 1024 ||
        E * (N / 128) * ((K + 255) / 256) > INT32_MAX / 2 ||
        (R / 128 + E) * ((N + 255) / 256) > INT32_MAX / 2)
        return TKQ_ERR_SHAPE;
    return TKQ_OK;
}
}  // namespace

tkq_status tkq_expert_product(const void* a, const float* a_sf, const void* w, const float* w_sf,
                              const int32_t* offsets, void* out, int64_t R, int64_t E, int64_t N,
                              int64_t K, int group, int fmt_a, int fmt_w, tkq_stream_t stream) {
    tkq_status st = check_product(R, E, N, K, group);
    if (st != TKQ_OK) return st;
    if (!fp8_fmt(fmt_a) || !fp8_fmt(fmt_w)) return TKQ_ERR_FMT;
    if (R == 0) return TKQ_OK;
    if (!a || !a_sf || !w || !w_sf || !offsets || !out) return TKQ_ERR_NULL;
    const Buffer in[] = {{a, R * K, 16},
                         {a_sf, R * (K / 128) * 4, 4},
                         {w, E * N * K, 16},
                         {w_sf, E * (N / 128) * (K / 128) * 4, 4},
                         {offsets, (E + 1) * 4, 4}};
    const Buffer outs[] = {{out, R * N * 2, 32}};
    if ((st = check_buffers(in, outs)) != TKQ_OK) return st;
    const tkq::ExpertProduct p = {a, a_sf, w, w_sf, offsets, out, R, N, K, static_cast<int>(E),
                                  fmt_a, fmt_w, false};
    return launch_status(tkq::launch_expert_product(p, static_cast<cudaStream_t>(stream)));
}

tkq_status tkq_expert_weight_grad(const void* dy_t, const float* dy_sf, const void* x_t,
                                  const float* x_sf, const int32_t* offsets, void* dw, int64_t R,
                                  int64_t E, int64_t N, int64_t K, int group, int fmt_dy,
                                  int fmt_x, int out_dtype, tkq_stream_t stream) {
    tkq_status st = check_product(R, E, N, K, group);
    if (st != TKQ_OK) return st;
    if (R % 128) return TKQ_ERR_SHAPE;
    if (!fp8_fmt(fmt_dy) || !fp8_fmt(fmt_x) ||
        (out_dtype != TKQ_OUT_F32 && out_dtype != TKQ_OUT_BF16))
        return TKQ_ERR_FMT;
    if ((R && (!dy_t || !dy_sf || !x_t || !x_sf)) || !offsets || !dw) return TKQ_ERR_NULL;
    const bool f32 = out_dtype == TKQ_OUT_F32;
    const Buffer in[] = {{dy_t, N * R, 16},
                         {dy_sf, N * (R / 128) * 4, 4},
                         {x_t, K * R, 16},
                         {x_sf, K * (R / 128) * 4, 4},
                         {offsets, (E + 1) * 4, 4}};
    const Buffer outs[] = {{dw, E * N * K * (f32 ? 4 : 2), 32}};
    if ((st = check_buffers(in, outs)) != TKQ_OK) return st;
    const tkq::ExpertProduct p = {dy_t, dy_sf, x_t, x_sf, offsets, dw, R, N, K, static_cast<int>(E),
                                  fmt_dy, fmt_x, f32};
    return launch_status(tkq::launch_expert_weight_grad(p, static_cast<cudaStream_t>(stream)));
}

tkq_status tkq_w4_product(const void* x, const float* x_sf, const void* w, const void* w_sf,
                          const int32_t* ids, void* out, int64_t T, int k, int64_t rows, int64_t E,
                          int64_t N, int64_t K, int group, int w_group, int fmt,
                          tkq_stream_t stream) {
    tkq_status st = check_product(0, E, N, K, group);
    if (st != TKQ_OK || (st = check_pairs(T, k, E, 0)) != TKQ_OK) return st;
    if (w_group != 32 && w_group != 128) return TKQ_ERR_GROUP;
    if (T * k > 1024 || (rows != T && rows != T * k) || (!ids && (k != 1 || E != 1)))
        return TKQ_ERR_SHAPE;
    if (!fp8_fmt(fmt)) return TKQ_ERR_FMT;
    if (T == 0) return TKQ_OK;
    if (!x || !x_sf || !w || !w_sf || !out) return TKQ_ERR_NULL;
    const Buffer in[] = {{x, rows * K, 16},
                         {x_sf, rows * (K / 128) * 4, 4},
                         {w, E * N * (K / 2), 16},
                         {w_sf, E * N * (K / 128) * 4, 4},  // four bytes or one fp32 a block
                         {ids, T * k * 4, 4}};
    const Buffer outs[] = {{out, T * k * N * 2, 16}};
    if ((st = check_buffers(in, outs)) != TKQ_OK) return st;
    const tkq::W4Product p = {x, x_sf, w, w_sf, ids, out, T, N, K, k, static_cast<int>(E), w_group,
                              fmt, rows != T};
    return launch_status(tkq::launch_w4_product(p, static_cast<cudaStream_t>(stream)));
}

tkq_status tkq_w4_cast(const void* w, void* codes, void* sf, int64_t N, int64_t K, int w_group,
                       tkq_stream_t stream) {
    if (N < 0 || N > INT32_MAX || K <= 0 || K % 128 || K > (int64_t{1} << 20)) return TKQ_ERR_SHAPE;
    if (w_group != 32 && w_group != 128) return TKQ_ERR_GROUP;
    if (N == 0) return TKQ_OK;
    if (!w || !codes || !sf) return TKQ_ERR_NULL;
    const Buffer in[] = {{w, N * K * 2, 16}};
    const Buffer outs[] = {{codes, N * (K / 2), 4}, {sf, N * (K / 128) * 4, 4}};
    if (const tkq_status st = check_buffers(in, outs)) return st;
    return launch_status(
        tkq::launch_w4_cast(w, codes, sf, N, K, w_group, static_cast<cudaStream_t>(stream)));
}

tkq_status tkq_swiglu_values(const void* x, const float* w, float* y, int64_t T, int64_t H,
                             tkq_stream_t stream) {
    tkq_status st = check_common(T, H, 128, TKQ_FMT_E4M3);
    if (st != TKQ_OK) return st;
    if (T == 0) return TKQ_OK;
    if (!x || !y) return TKQ_ERR_NULL;
    if (!tkq::aligned(x, 16) || !tkq::aligned(y, 16) || (w && !tkq::aligned(w, 4)))
        return TKQ_ERR_ALIGN;
    const auto rx = tkq::span(x, T * H * 4), ry = tkq::span(y, T * H * 4);
    const auto rw = w ? tkq::span(w, T * 4) : tkq::Range{0, 0};
    if (tkq::overlap(rx, ry) || tkq::overlap(rw, ry)) return TKQ_ERR_ALIAS;
    tkq::register_call({rx, rw}, {ry});
    return launch_status(
        tkq::launch_swiglu_values(x, w, y, T, H, static_cast<cudaStream_t>(stream)));
}

tkq_status tkq_swiglu_backward_values(const void* x, const void* dy, const float* w, float* y,
                                      int64_t T, int64_t H, tkq_stream_t stream) {
    tkq_status st = check_common(T, H, 128, TKQ_FMT_E4M3);
    if (st != TKQ_OK) return st;
    if (T == 0) return TKQ_OK;
    if (!x || !dy || !y) return TKQ_ERR_NULL;
    if (!tkq::aligned(x, 16) || !tkq::aligned(dy, 16) || !tkq::aligned(y, 16) ||
        (w && !tkq::aligned(w, 4)))
        return TKQ_ERR_ALIGN;
    const auto rx = tkq::span(x, T * H * 4), rd = tkq::span(dy, T * H * 2),
               ry = tkq::span(y, T * H * 8);
    const auto rw = w ? tkq::span(w, T * 4) : tkq::Range{0, 0};
    if (tkq::overlap(rx, ry) || tkq::overlap(rd, ry) || tkq::overlap(rw, ry)) return TKQ_ERR_ALIAS;
    tkq::register_call({rx, rd, rw}, {ry});
    return launch_status(tkq::launch_swiglu_backward_values(x, dy, w, y, T, H,
                                                            static_cast<cudaStream_t>(stream)));
}

tkq_status tkq_fp8_encode(const float* x, void* out, int64_t n, int fmt, tkq_stream_t stream) {
    if (n < 0 || n % 4) return TKQ_ERR_SHAPE;
    if (fmt != TKQ_FMT_E4M3 && fmt != TKQ_FMT_E5M2) return TKQ_ERR_FMT;
    if (n == 0) return TKQ_OK;
    if (!x || !out) return TKQ_ERR_NULL;
    if (!tkq::aligned(x, 16) || !tkq::aligned(out, 4)) return TKQ_ERR_ALIGN;
    const auto rx = tkq::span(x, n * 4), ro = tkq::span(out, n);
    if (tkq::overlap(rx, ro)) return TKQ_ERR_ALIAS;
    tkq::register_call({rx}, {ro});
    return launch_status(
        tkq::launch_fp8_encode(x, out, n, fmt, static_cast<cudaStream_t>(stream)));
}

tkq_status tkq_read_device_status(uint32_t* flags, int clear) {
    if (!flags) return TKQ_ERR_NULL;
    if (cudaDeviceSynchronize() != cudaSuccess) return TKQ_ERR_CUDA;
    unsigned int v = 0;
    if (cudaMemcpyFromSymbol(&v, g_tkq_device_status, sizeof v) != cudaSuccess)
        return TKQ_ERR_CUDA;
    if (clear) {
        const unsigned int zero = 0;
        if (cudaMemcpyToSymbol(g_tkq_device_status, &zero, sizeof zero) != cudaSuccess)
            return TKQ_ERR_CUDA;
    }
    *flags = v;
    return (v & TKQ_DEVICE_TIMEOUT) ? TKQ_ERR_TIMEOUT : TKQ_OK;
}

tkq_status tkq_selftest_wait_timeout(int64_t limit_ns, tkq_stream_t stream) {
    if (limit_ns <= 0 || limit_ns > int64_t{2000000000}) return TKQ_ERR_SHAPE;
    unsigned int* status = tkq::device_status_word();
    if (!status) return TKQ_ERR_CUDA;
    tkq::selftest_wait_kernel<<<1, 32, 0, static_cast<cudaStream_t>(stream)>>>(
        status, static_cast<uint64_t>(limit_ns));
    return launch_status(cudaGetLastError());
}

const char* tkq_status_string(int status) {
    switch (status) {
        case TKQ_OK: return "TKQ_OK";
        case TKQ_ERR_NULL: return "TKQ_ERR_NULL: a required pointer is NULL";
        case TKQ_ERR_SHAPE: return "TKQ_ERR_SHAPE: invalid or unsupported extents";
        case TKQ_ERR_GROUP: return "TKQ_ERR_GROUP: group must be 128";
        case TKQ_ERR_FMT: return "TKQ_ERR_FMT: unknown FP8 format";
        case TKQ_ERR_ALIGN: return "TKQ_ERR_ALIGN: misaligned pointer";
        case TKQ_ERR_CUDA: return "TKQ_ERR_CUDA: kernel launch failed";
        case TKQ_ERR_TIMEOUT:
            return "TKQ_ERR_TIMEOUT: a bounded wait inside a kernel gave up (outputs incomplete)";
        case TKQ_ERR_ALIAS: return "TKQ_ERR_ALIAS: buffers overlap";
        case TKQ_ERR_FLAGS: return "TKQ_ERR_FLAGS: unknown option flags";
        case TKQ_ERR_VALUE: return "TKQ_ERR_VALUE: invalid scalar argument";
        default: return "TKQ_ERR_UNKNOWN";
    }
}

int tkq_version(void) { return 300; }

int tkq_checked_build(void) {
#ifdef TKQ_CHECKED
    return 1;
#else
    return 0;
#endif
}

tkq_status tkq_read_check_address(uint64_t* addr, int clear) {
    if (!addr) return TKQ_ERR_NULL;
    if (cudaDeviceSynchronize() != cudaSuccess) return TKQ_ERR_CUDA;
    unsigned long long v = 0;
    if (cudaMemcpyFromSymbol(&v, g_tkq_bad_address, sizeof v) != cudaSuccess) return TKQ_ERR_CUDA;
    if (clear) {
        const unsigned long long zero = 0;
        if (cudaMemcpyToSymbol(g_tkq_bad_address, &zero, sizeof zero) != cudaSuccess)
            return TKQ_ERR_CUDA;
    }
    *addr = v;
    return TKQ_OK;
}

}  // extern "C"
