// C ABI of libcq: argument validation and dispatch to the kernel launchers.
// Every check runs before any launch, so an error return means that nothing
// was launched and nothing was written. See include/cq.h, include/cq_kv.h and include/cq_tree.h
// for the contract.
#include <algorithm>
#include <cstdint>
#include <atomic>
#include <map>
#include <mutex>
#include <utility>

#include <cuda_runtime.h>

#include "cq.h"
#include "cq_internal.h"
#include "kv.cuh"
#include "tree.cuh"

namespace {

// Status word of kernels that take no workspace (cq_gemv / cq_gemm copy waits).
__device__ int g_cq_status;

constexpr int MAX_DEVICES = 64;
std::mutex g_dev_mutex;
bool g_dev_ready[MAX_DEVICES];
cq::DeviceInfo g_dev[MAX_DEVICES];

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
// Quantized activation rows: Q8_K rows are 292 bytes per 256 elements, so a
// token's row is only 4-byte aligned; the kernels read activations in 32-bit words.
bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

bool is_weight_fmt(int f) {
    return f == CQ_Q4_0 || f == CQ_Q4_1 || f == CQ_Q8_0 || f == CQ_Q4_K || f == CQ_Q5_K || f == CQ_Q6_K;
}
// Q6_K rows of 210-byte superblocks meet the bulk copies' 16-byte rule only
// eight superblocks at a time: K a multiple of 2048.
bool fmt_shape_ok(int f, int64_t K) { return f != CQ_Q6_K || K % 2048 == 0; }
bool is_act_fmt(int f) { return f == CQ_Q8_0 || f == CQ_Q8_1 || f == CQ_Q8_K; }

// Largest K accepted by the single-pass kernels (activation rows staged in
// 96 KB of shared memory: 96 KB / 304 B per 256 elements).
constexpr int64_t K_MAX = 65536;

cq_status check_shape(int64_t M, int64_t N, int64_t K) {
    if (M < 0 || N < 0 || K < 0) return CQ_ERR_INVALID_ARG;
    if (K == 0 || K % 256 != 0 || K > K_MAX) return CQ_ERR_SHAPE;
    if (N > (int64_t(1) << 31)) return CQ_ERR_SHAPE;
    return CQ_OK;
}

}  // namespace

namespace cq {
std::atomic<int> g_weights_const{0};
bool weights_const() { return g_weights_const.load(std::memory_order_relaxed) != 0; }

std::mutex g_attr_mutex;
std::map<std::pair<int, const void*>, int> g_attr_raised;

cudaError_t raise_smem_limit(const void* kernel, int bytes) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    std::lock_guard<std::mutex> lock(g_attr_mutex);
    int& have = g_attr_raised[{dev, kernel}];
    if (have >= bytes) return cudaSuccess;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess) have = bytes;
    return e;
}

// Library-owned stream-ordered scratch: one memory pool per device, created on
// first use, keeping up to 512 MB between calls so that steady-state
// allocations map no new memory.
std::mutex g_pool_mutex;
bool g_pool_ready[MAX_DEVICES];
cudaMemPool_t g_pool[MAX_DEVICES];

void* scratch_alloc(size_t bytes, cudaStream_t s) {
    int dev = 0;
    if (bytes == 0 || cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= MAX_DEVICES) return nullptr;
    // No allocation while the stream is being captured into a graph: the
    // caller then takes its allocation-free path.
    cudaStreamCaptureStatus cap = cudaStreamCaptureStatusNone;
    if (cudaStreamIsCapturing(s, &cap) != cudaSuccess) {
        (void)cudaGetLastError();
        return nullptr;
    }
    if (cap != cudaStreamCaptureStatusNone) return nullptr;
    cudaMemPool_t pool;
    {
        std::lock_guard<std::mutex> lock(g_pool_mutex);
        if (!g_pool_ready[dev]) {
            cudaMemPoolProps props{};
            props.allocType = cudaMemAllocationTypePinned;
            props.location.type = cudaMemLocationTypeDevice;
            props.location.id = dev;
            if (cudaMemPoolCreate(&g_pool[dev], &props) != cudaSuccess) {
                (void)cudaGetLastError();
                return nullptr;
            }
            uint64_t keep = uint64_t(512) << 20;
            (void)cudaMemPoolSetAttribute(g_pool[dev], cudaMemPoolAttrReleaseThreshold, &keep);
            g_pool_ready[dev] = true;
        }
        pool = g_pool[dev];
    }
    void* p = nullptr;
    if (cudaMallocFromPoolAsync(&p, bytes, pool, s) != cudaSuccess) {
        (void)cudaGetLastError();
        return nullptr;
    }
    if ((reinterpret_cast<uintptr_t>(p) & 255u) != 0) {   // the GEMM workspaces want 256-byte alignment
        (void)cudaFreeAsync(p, s);
        return nullptr;
    }
    return p;
}

cudaError_t scratch_free(void* p, cudaStream_t s) { return p != nullptr ? cudaFreeAsync(p, s) : cudaSuccess; }

cudaError_t device_info(DeviceInfo* out) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= MAX_DEVICES) return cudaErrorInvalidDevice;
    std::lock_guard<std::mutex> lock(g_dev_mutex);
    if (!g_dev_ready[dev]) {
        DeviceInfo d{};
        e = cudaDeviceGetAttribute(&d.sm_count, cudaDevAttrMultiProcessorCount, dev);
        if (e != cudaSuccess) return e;
        e = cudaDeviceGetAttribute(&d.smem_optin, cudaDevAttrMaxSharedMemoryPerBlockOptin, dev);
        if (e != cudaSuccess) return e;
        e = cudaGetSymbolAddress(reinterpret_cast<void**>(&d.status), g_cq_status);
        if (e != cudaSuccess) return e;
        g_dev[dev] = d;
        g_dev_ready[dev] = true;
    }
    *out = g_dev[dev];
    return cudaSuccess;
}
}  // namespace cq

extern "C" {

const char* cq_status_string(cq_status s) {
    switch (s) {
    case CQ_OK: return "ok";
    case CQ_ERR_INVALID_ARG: return "invalid argument";
    case CQ_ERR_UNSUPPORTED_FORMAT: return "unsupported format";
    case CQ_ERR_SHAPE: return "unsupported shape";
    case CQ_ERR_ALIGNMENT: return "pointer not 16-byte aligned";
    case CQ_ERR_WORKSPACE: return "workspace missing or too small";
    case CQ_ERR_CUDA: return "CUDA error";
    case CQ_ERR_DEVICE_STATUS: return "device reported bad input";
    case CQ_ERR_TIMEOUT: return "device wait timed out";
    }
    return "unknown status";
}

cq_status cq_quantize_act(cq_format act_fmt, int64_t M, int64_t K, const float* x, void* xq, void* stream) {
    if (!is_act_fmt(act_fmt)) return CQ_ERR_UNSUPPORTED_FORMAT;
    cq_status st = check_shape(M, 1, K);
    if (st != CQ_OK) return st;
    if (M == 0) return CQ_OK;
    if (x == nullptr || xq == nullptr) return CQ_ERR_INVALID_ARG;
    if (!aligned16(x) || !aligned16(xq)) return CQ_ERR_ALIGNMENT;
    cudaError_t e = cq::launch_quantize(act_fmt, M, K, x, xq, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? CQ_OK : CQ_ERR_CUDA;
}

cq_status cq_gemv(cq_format w_fmt, int64_t M, int64_t N, int64_t K, const void* W, const void* xq, float* y,
                  void* stream) {
    if (!is_weight_fmt(w_fmt)) return CQ_ERR_UNSUPPORTED_FORMAT;
    cq_status st = check_shape(M, N, K);
    if (st != CQ_OK) return st;
    if (M > 16 || !fmt_shape_ok(w_fmt, K)) return CQ_ERR_SHAPE;
    if (M == 0 || N == 0) return CQ_OK;
    if (W == nullptr || xq == nullptr || y == nullptr) return CQ_ERR_INVALID_ARG;
    if (!aligned16(W) || !aligned4(xq) || !aligned16(y)) return CQ_ERR_ALIGNMENT;
    cq::DeviceInfo dev;
    if (cq::device_info(&dev) != cudaSuccess) return CQ_ERR_CUDA;
    cudaError_t e = cq::launch_gemv(dev, w_fmt, static_cast<int>(M), N, K, W, xq, y, nullptr,
                                    static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? CQ_OK : CQ_ERR_CUDA;
}

size_t cq_repack_size(cq_format w_fmt, int64_t N, int64_t K) {
    if (N < 0 || K > K_MAX) return 0;
    return static_cast<size_t>(cq::repack_size(w_fmt, N, K));
}

cq_status cq_repack(cq_format w_fmt, int64_t N, int64_t K, const void* W, void* Wp, void* stream) {
    if (w_fmt != CQ_Q4_0 && w_fmt != CQ_Q4_1 && w_fmt != CQ_Q8_0) return CQ_ERR_UNSUPPORTED_FORMAT;
    cq_status st = check_shape(1, N, K);
    if (st != CQ_OK) return st;
    if (N == 0) return CQ_OK;
    if (W == nullptr || Wp == nullptr) return CQ_ERR_INVALID_ARG;
    if (!aligned16(W) || !aligned16(Wp)) return CQ_ERR_ALIGNMENT;
    cudaError_t e = cq::launch_repack(w_fmt, N, K, W, Wp, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? CQ_OK : CQ_ERR_CUDA;
}

cq_status cq_gemv_packed(cq_format w_fmt, int64_t M, int64_t N, int64_t K, const void* Wp, const void* xq, float* y,
                         void* stream) {
    if (w_fmt != CQ_Q4_0 && w_fmt != CQ_Q4_1 && w_fmt != CQ_Q8_0) return CQ_ERR_UNSUPPORTED_FORMAT;
    cq_status st = check_shape(M, N, K);
    if (st != CQ_OK) return st;
    if (M > 16) return CQ_ERR_SHAPE;
    if (M == 0 || N == 0) return CQ_OK;
    if (Wp == nullptr || xq == nullptr || y == nullptr) return CQ_ERR_INVALID_ARG;
    if (!aligned16(Wp) || !aligned4(xq) || !aligned16(y)) return CQ_ERR_ALIGNMENT;
    cq::DeviceInfo dev;
    if (cq::device_info(&dev) != cudaSuccess) return CQ_ERR_CUDA;
    const int need = cq::gemv_packed_smem(w_fmt, static_cast<int>(M), K);
    if (need > (dev.smem_optin < 227 * 1024 ? dev.smem_optin : 227 * 1024)) return CQ_ERR_SHAPE;
    cudaError_t e = cq::launch_gemv_packed(dev, w_fmt, static_cast<int>(M), N, K, Wp, xq, y,
                                           static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? CQ_OK : CQ_ERR_CUDA;
}

cq_status cq_set_option(cq_option opt, int64_t value) {
    if (opt != CQ_OPT_WEIGHTS_CONST || (value != 0 && value != 1)) return CQ_ERR_INVALID_ARG;
    cq::g_weights_const.store(static_cast<int>(value), std::memory_order_relaxed);
    return CQ_OK;
}

cq_status cq_gemv_x(cq_format w_fmt, int64_t M, int64_t N, int64_t K, const void* W, const float* x, void* xq,
                    float* y, void* stream) {
    if (!is_weight_fmt(w_fmt)) return CQ_ERR_UNSUPPORTED_FORMAT;
    cq_status st = check_shape(M, N, K);
    if (st != CQ_OK) return st;
    if (M > 16 || !fmt_shape_ok(w_fmt, K)) return CQ_ERR_SHAPE;
    if (M == 0) return CQ_OK;
    if (x == nullptr || xq == nullptr || (N > 0 && (W == nullptr || y == nullptr))) return CQ_ERR_INVALID_ARG;
    if (!aligned16(x) || !aligned16(xq) || (N > 0 && (!aligned16(W) || !aligned16(y)))) return CQ_ERR_ALIGNMENT;
    cq::DeviceInfo dev;
    if (cq::device_info(&dev) != cudaSuccess) return CQ_ERR_CUDA;
    cudaError_t e = cq::launch_gemv(dev, w_fmt, static_cast<int>(M), N, K, W, xq, y, x,
                                    static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? CQ_OK : CQ_ERR_CUDA;
}

cq_status cq_gemv_swiglu(cq_format w_fmt, int64_t M, int64_t F, int64_t K, const void* W_gate, const void* W_up,
                         const void* xq, float* h, void* stream) {
    if (!is_weight_fmt(w_fmt)) return CQ_ERR_UNSUPPORTED_FORMAT;
    cq_status st = check_shape(M, F, K);
    if (st != CQ_OK) return st;
    if (M < 1 || M > 16 || F < 1 || !fmt_shape_ok(w_fmt, K)) return CQ_ERR_SHAPE;
    const int64_t ce = w_fmt == CQ_Q4_K || w_fmt == CQ_Q5_K || w_fmt == CQ_Q6_K ? 256 : 128;
    if (2 * (K / ce) > 512) return CQ_ERR_SHAPE;
    if (W_gate == nullptr || W_up == nullptr || xq == nullptr || h == nullptr) return CQ_ERR_INVALID_ARG;
    if (!aligned16(W_gate) || !aligned16(W_up) || !aligned4(xq) || !aligned16(h)) return CQ_ERR_ALIGNMENT;
    cq::DeviceInfo dev;
    if (cq::device_info(&dev) != cudaSuccess) return CQ_ERR_CUDA;
    cudaError_t e = cq::launch_gemv_swiglu(dev, w_fmt, static_cast<int>(M), F, K, W_gate, W_up, xq, h,
                                           static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? CQ_OK : CQ_ERR_CUDA;
}

cq_status cq_selftest_wait_timeout(int64_t limit_ns, int32_t* out_code, void* stream) {
    if (out_code == nullptr || limit_ns < 1000 || limit_ns > 1000000000) return CQ_ERR_INVALID_ARG;
    cq::DeviceInfo dev;
    if (cq::device_info(&dev) != cudaSuccess) return CQ_ERR_CUDA;
    if (cq::launch_wait_timeout_probe(static_cast<uint64_t>(limit_ns), dev.status,
                                      static_cast<cudaStream_t>(stream)) != cudaSuccess)
        return CQ_ERR_CUDA;
    return cq_read_global_status(out_code, 1);
}

cq_status cq_read_global_status(int32_t* out_code, int clear) {
    if (out_code == nullptr) return CQ_ERR_INVALID_ARG;
    if (cudaDeviceSynchronize() != cudaSuccess) return CQ_ERR_CUDA;
    int v = 0;
    if (cudaMemcpyFromSymbol(&v, g_cq_status, sizeof v) != cudaSuccess) return CQ_ERR_CUDA;
    if (clear) {
        const int z = 0;
        if (cudaMemcpyToSymbol(g_cq_status, &z, sizeof z) != cudaSuccess) return CQ_ERR_CUDA;
    }
    *out_code = v;
    if (v & CQ_DEV_WAIT_TIMEOUT) return CQ_ERR_TIMEOUT;
    return v ? CQ_ERR_DEVICE_STATUS : CQ_OK;
}

}  // extern "C"

namespace {

// cq_gemm formats: Q4_K and the 32-element formats (their activation rows are
// read by TMA, so xq must be 16-byte aligned), all on tcgen05 kernels that
// take an optional workspace (cq_gemm_ws).
bool is_gemm_fmt(int f) { return f == CQ_Q4_K || f == CQ_Q4_0 || f == CQ_Q4_1 || f == CQ_Q8_0; }

// with_ws: the caller's workspace (cq_gemm_ws). Otherwise scratch = true takes
// the workspace from the library's pool when it can (cq_gemm), and false never
// allocates (cq_gemm_noalloc).
cq_status gemm_common(cq_format w_fmt, int64_t M, int64_t N, int64_t K, const void* W, const void* xq, float* y,
                      void* workspace, size_t workspace_bytes, bool with_ws, void* stream, bool scratch = false) {
    if (!is_gemm_fmt(w_fmt)) return CQ_ERR_UNSUPPORTED_FORMAT;
    cq_status st = check_shape(M, N, K);
    if (st != CQ_OK) return st;
    if (M > (int64_t(1) << 31) - 1) return CQ_ERR_SHAPE;
    if (M == 0 || N == 0) return CQ_OK;
    if (W == nullptr || xq == nullptr || y == nullptr) return CQ_ERR_INVALID_ARG;
    const size_t need = with_ws ? cq::gemm_workspace_size(w_fmt, M, K) : 0;
    if (need > 0 && (workspace == nullptr || workspace_bytes < need)) return CQ_ERR_WORKSPACE;
    const bool xq_ok = w_fmt == CQ_Q4_K ? aligned4(xq) : aligned16(xq);
    if (!aligned16(W) || !xq_ok || !aligned16(y)) return CQ_ERR_ALIGNMENT;
    if (need > 0 && (reinterpret_cast<uintptr_t>(workspace) & 255u) != 0) return CQ_ERR_ALIGNMENT;
    cq::DeviceInfo dev;
    if (cq::device_info(&dev) != cudaSuccess) return CQ_ERR_CUDA;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    void* ws = need > 0 ? workspace : nullptr;
    void* own = !with_ws && scratch ? cq::scratch_alloc(cq::gemm_workspace_size(w_fmt, M, K), s) : nullptr;
    if (own != nullptr) ws = own;
    const cudaError_t e = w_fmt == CQ_Q4_K ? cq::launch_gemm(dev, w_fmt, M, N, K, W, xq, y, ws, s)
                                           : cq::launch_gemm_tc32(dev, w_fmt, M, N, K, W, xq, y, ws, s);
    const cudaError_t f = cq::scratch_free(own, s);
    return e == cudaSuccess && f == cudaSuccess ? CQ_OK : CQ_ERR_CUDA;
}

}  // namespace

extern "C" {

cq_status cq_gemm(cq_format w_fmt, int64_t M, int64_t N, int64_t K, const void* W, const void* xq, float* y,
                  void* stream) {
    return gemm_common(w_fmt, M, N, K, W, xq, y, nullptr, 0, false, stream, true);
}

cq_status cq_gemm_noalloc(cq_format w_fmt, int64_t M, int64_t N, int64_t K, const void* W, const void* xq, float* y,
                          void* stream) {
    return gemm_common(w_fmt, M, N, K, W, xq, y, nullptr, 0, false, stream, false);
}

size_t cq_gemm_workspace_size(cq_format w_fmt, int64_t M, int64_t N, int64_t K) {
    if (!is_gemm_fmt(w_fmt) || check_shape(M, N, K) != CQ_OK) return 0;
    return cq::gemm_workspace_size(w_fmt, M, K);
}

cq_status cq_gemm_ws(cq_format w_fmt, int64_t M, int64_t N, int64_t K, const void* W, const void* xq, float* y,
                     void* workspace, size_t workspace_bytes, void* stream) {
    return gemm_common(w_fmt, M, N, K, W, xq, y, workspace, workspace_bytes, true, stream);
}

}  // extern "C"

extern "C" {

static cq_status moe_check_shape(int64_t T, int64_t K, int64_t F, int64_t E, int64_t topk) {
    if (T < 0 || K < 0 || F < 0 || E < 0 || topk < 0) return CQ_ERR_INVALID_ARG;
    if (K == 0 || K % 256 != 0 || K > 4096) return CQ_ERR_SHAPE;
    if (F == 0 || F % 256 != 0 || F > 8192) return CQ_ERR_SHAPE;
    if (E < 1 || E > 256 || topk < 1 || topk > E) return CQ_ERR_SHAPE;
    if (T * topk > (int64_t(1) << 20)) return CQ_ERR_SHAPE;
    return CQ_OK;
}

size_t cq_moe_workspace_size(int64_t T, int64_t K, int64_t F, int64_t E, int64_t topk) {
    if (moe_check_shape(T, K, F, E, topk) != CQ_OK) return 0;
    return cq::moe_layout(T, K, F, E, topk).total;
}

cq_status cq_moe_workspace_offsets(int64_t T, int64_t K, int64_t F, int64_t E, int64_t topk, size_t* status_off,
                                   size_t* h_off, size_t* hq_off) {
    cq_status st = moe_check_shape(T, K, F, E, topk);
    if (st != CQ_OK) return st;
    if (status_off == nullptr || h_off == nullptr || hq_off == nullptr) return CQ_ERR_INVALID_ARG;
    const cq::MoeLayout L = cq::moe_layout(T, K, F, E, topk);
    *status_off = L.status;
    *h_off = L.h;
    *hq_off = L.hq;
    return CQ_OK;
}

cq_status cq_moe_gemv(cq_format w_fmt, int64_t T, int64_t K, int64_t F, int64_t E, int64_t topk, const void* W_gate,
                      const void* W_up, const void* W_down, const int32_t* expert_ids, const float* route_w,
                      const void* xq, float* y, void* workspace, size_t workspace_bytes, void* stream) {
    if (w_fmt != CQ_Q4_0) return CQ_ERR_UNSUPPORTED_FORMAT;
    cq_status st = moe_check_shape(T, K, F, E, topk);
    if (st != CQ_OK) return st;
    if (T == 0) return CQ_OK;
    if (!W_gate || !W_up || !W_down || !expert_ids || !route_w || !xq || !y) return CQ_ERR_INVALID_ARG;
    if (workspace == nullptr || workspace_bytes < cq::moe_layout(T, K, F, E, topk).total) return CQ_ERR_WORKSPACE;
    if ((reinterpret_cast<uintptr_t>(workspace) & 255u) != 0) return CQ_ERR_ALIGNMENT;
    for (const void* q : {W_gate, W_up, W_down, static_cast<const void*>(expert_ids),
                          static_cast<const void*>(route_w), xq, static_cast<const void*>(y)})
        if (!aligned16(q)) return CQ_ERR_ALIGNMENT;
    cq::DeviceInfo dev;
    if (cq::device_info(&dev) != cudaSuccess) return CQ_ERR_CUDA;
    cudaError_t e = cq::launch_moe(dev, static_cast<int>(T), static_cast<int>(K), static_cast<int>(F),
                                   static_cast<int>(E), static_cast<int>(topk), W_gate, W_up, W_down, expert_ids,
                                   route_w, xq, y, workspace, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? CQ_OK : CQ_ERR_CUDA;
}

cq_status cq_read_device_status(const void* workspace, int32_t* out_code, void* stream) {
    if (out_code == nullptr) return CQ_ERR_INVALID_ARG;
    if (workspace != nullptr) return cq_moe_read_status(workspace, out_code, stream);
    if (cudaStreamSynchronize(static_cast<cudaStream_t>(stream)) != cudaSuccess) return CQ_ERR_CUDA;
    int v = 0;
    if (cudaMemcpyFromSymbol(&v, g_cq_status, sizeof v) != cudaSuccess) return CQ_ERR_CUDA;
    const int z = 0;
    if (v != 0 && cudaMemcpyToSymbol(g_cq_status, &z, sizeof z) != cudaSuccess) return CQ_ERR_CUDA;
    *out_code = v;
    if (v & CQ_DEV_WAIT_TIMEOUT) return CQ_ERR_TIMEOUT;
    return v ? CQ_ERR_DEVICE_STATUS : CQ_OK;
}

cq_status cq_moe_read_status(const void* workspace, int32_t* out_code, void* stream) {
    if (workspace == nullptr || out_code == nullptr) return CQ_ERR_INVALID_ARG;
    if (cudaStreamSynchronize(static_cast<cudaStream_t>(stream)) != cudaSuccess) return CQ_ERR_CUDA;
    int v = 0;
    if (cudaMemcpy(&v, workspace, sizeof v, cudaMemcpyDeviceToHost) != cudaSuccess) return CQ_ERR_CUDA;
    *out_code = v;
    if (v & CQ_DEV_WAIT_TIMEOUT) return CQ_ERR_TIMEOUT;
    return v ? CQ_ERR_DEVICE_STATUS : CQ_OK;
}

}  // extern "C"

namespace {

bool aligned_to(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
int dtype_bytes(int dt) { return dt == CQ_F32 ? 4 : dt == CQ_F16 || dt == CQ_BF16 ? 2 : 0; }
int page_shift(int64_t page_size) {
    return page_size == 16 ? 4 : page_size == 32 ? 5 : page_size == 64 ? 6 : page_size == 128 ? 7 : -1;
}
constexpr int64_t INT_LIMIT = (int64_t(1) << 31) - 1;

// The cache's description: sizes first (none of them is dereferenced), then its pointers.
cq_status check_cache(const cq_kv_cache* c, cq::KvView* out) {
    if (c == nullptr || c->num_pages < 0) return CQ_ERR_INVALID_ARG;
    const int shift = page_shift(c->page_size);
    if (shift < 0 || (c->head_dim != 64 && c->head_dim != 128) || c->kv_heads < 1 || c->kv_heads > 1024 ||
        c->num_pages > INT_LIMIT || c->reserved != 0)
        return CQ_ERR_SHAPE;
    if (c->page_stride < int64_t(c->kv_heads) * c->page_size * c->head_dim || c->scale_stride < c->kv_heads)
        return CQ_ERR_SHAPE;
    if (c->k == nullptr || c->v == nullptr || c->k_scale == nullptr || c->v_scale == nullptr) return CQ_ERR_INVALID_ARG;
    if (!aligned16(c->k) || !aligned16(c->v) || (c->page_stride & 15) != 0 || !aligned4(c->k_scale) ||
        !aligned4(c->v_scale))
        return CQ_ERR_ALIGNMENT;
    *out = cq::KvView{static_cast<int8_t*>(c->k), static_cast<int8_t*>(c->v), c->k_scale, c->v_scale, c->num_pages,
                      c->page_stride, c->scale_stride, c->page_size, shift, c->kv_heads, c->head_dim};
    return CQ_OK;
}

// Rows of `width` values: stride (elements) and base fit 16-byte accesses.
cq_status check_rows(const void* p, int64_t stride, int64_t width, int bytes) {
    if (p == nullptr) return CQ_ERR_INVALID_ARG;
    if (stride < width || stride > (int64_t(1) << 40)) return CQ_ERR_SHAPE;
    return aligned16(p) && (stride * bytes & 15) == 0 ? CQ_OK : CQ_ERR_ALIGNMENT;
}

cq_status status_of(cudaError_t e) { return e == cudaSuccess ? CQ_OK : CQ_ERR_CUDA; }

// cq_attn_paged, and with masks cq_attn_tree.
cq_status attend(const cq_kv_cache* cache, cq_dtype dtype, int64_t R, int64_t T, int64_t q_heads, int64_t max_new,
                 const void* q, int64_t q_stride, const int32_t* block_table, int64_t max_blocks, const int32_t* kv_len,
                 const int32_t* q_start, const uint64_t* tree, bool needs_tree, float scale, int causal, int64_t window,
                 void* out, int64_t out_stride, float* lse, void* workspace, size_t workspace_bytes, void* stream) {
    const int bytes = dtype_bytes(dtype);
    if (bytes == 0) return CQ_ERR_UNSUPPORTED_FORMAT;
    if (R < 0 || T < 0 || q_heads < 0 || max_new < 0 || max_blocks < 0 || window < 0 || (causal != 0 && causal != 1))
        return CQ_ERR_INVALID_ARG;
    cq::KvView c;
    cq_status st = check_cache(cache, &c);
    if (st != CQ_OK) return st;
    if (q_heads < 1 || q_heads > 1024 || q_heads % c.heads != 0 || R > 16384 || T > INT_LIMIT ||
        max_blocks > (INT_LIMIT >> c.page_shift) || T * (q_heads / c.heads) > (int64_t(1) << 30))
        return CQ_ERR_SHAPE;
    if (R == 0 || T == 0) return CQ_OK;
    const int64_t width = q_heads * c.dim;
    if ((st = check_rows(q, q_stride, width, bytes)) != CQ_OK) return st;
    if ((st = check_rows(out, out_stride, width, bytes)) != CQ_OK) return st;
    if (kv_len == nullptr || q_start == nullptr || (max_blocks > 0 && block_table == nullptr) || (needs_tree && tree == nullptr))
        return CQ_ERR_INVALID_ARG;
    const size_t need = cq::attn_workspace_size(c.dim);
    if (workspace == nullptr || workspace_bytes < need) return CQ_ERR_WORKSPACE;
    if (!aligned4(kv_len) || !aligned4(q_start) || !aligned4(block_table) || !aligned4(lse) || !aligned_to(tree, 8) ||
        !aligned_to(workspace, 256))
        return CQ_ERR_ALIGNMENT;
    cq::DeviceInfo dev;
    if (cq::device_info(&dev) != cudaSuccess) return CQ_ERR_CUDA;
    cq::AttnArgs a{};
    a.q = q; a.out = out; a.lse = lse;
    a.table = block_table; a.kv_len = kv_len; a.q_start = q_start;
    a.tree = tree;
    a.status = dev.status; a.ws = workspace;
    a.q_stride = q_stride; a.out_stride = out_stride;
    a.max_blocks = max_blocks;
    a.window = std::min(window, int64_t(1) << 32);   // wider than any length and position: sums with positions stay in range
    a.max_new = std::min(max_new, T);
    a.scale = scale;
    a.R = static_cast<int>(R); a.T = static_cast<int>(T); a.heads = static_cast<int>(q_heads); a.causal = causal;
    return status_of(cq::launch_attn(dev, c, dtype, a, static_cast<cudaStream_t>(stream)));
}

}  // namespace

extern "C" {

cq_status cq_kv_plan(int64_t R, int64_t page_size, int64_t max_blocks, int64_t num_pages, const int32_t* past_len,
                     const int32_t* new_len, const int32_t* free_pages, int64_t n_free, int32_t* block_table,
                     int64_t T, int32_t* kv_len, int32_t* q_start, int64_t* slots, int32_t* positions, int32_t* used,
                     void* stream) {
    if (R < 0 || max_blocks < 0 || num_pages < 0 || n_free < 0 || T < 0) return CQ_ERR_INVALID_ARG;
    const int shift = page_shift(page_size);
    if (shift < 0 || R > 16384 || T > INT_LIMIT || n_free > INT_LIMIT || num_pages > INT_LIMIT ||
        max_blocks > (INT_LIMIT >> shift))
        return CQ_ERR_SHAPE;
    if (q_start == nullptr || used == nullptr || (T > 0 && (slots == nullptr || positions == nullptr)) ||
        (R > 0 && (past_len == nullptr || new_len == nullptr || kv_len == nullptr)) ||
        (R > 0 && max_blocks > 0 && block_table == nullptr) || (n_free > 0 && free_pages == nullptr))
        return CQ_ERR_INVALID_ARG;
    const void* words[] = {past_len, new_len, free_pages, block_table, kv_len, q_start, positions, used};
    for (const void* p : words)
        if (!aligned4(p)) return CQ_ERR_ALIGNMENT;
    if (!aligned_to(slots, 8)) return CQ_ERR_ALIGNMENT;
    cq::DeviceInfo dev;
    if (cq::device_info(&dev) != cudaSuccess) return CQ_ERR_CUDA;
    return status_of(cq::launch_kv_plan(dev, static_cast<int>(R), shift, max_blocks, num_pages, past_len, new_len,
                                        free_pages, static_cast<int>(n_free), block_table, static_cast<int>(T), kv_len,
                                        q_start, slots, positions, used, static_cast<cudaStream_t>(stream)));
}

cq_status cq_kv_append(const cq_kv_cache* cache, cq_dtype dtype, int64_t T, const void* k, int64_t k_stride,
                       const void* v, int64_t v_stride, const int64_t* slots, void* stream) {
    const int bytes = dtype_bytes(dtype);
    if (bytes == 0) return CQ_ERR_UNSUPPORTED_FORMAT;
    if (T < 0) return CQ_ERR_INVALID_ARG;
    cq::KvView c;
    cq_status st = check_cache(cache, &c);
    if (st != CQ_OK) return st;
    if (T > INT_LIMIT) return CQ_ERR_SHAPE;
    if (T == 0) return CQ_OK;
    const int64_t width = int64_t(c.heads) * c.dim;
    if ((st = check_rows(k, k_stride, width, bytes)) != CQ_OK) return st;
    if ((st = check_rows(v, v_stride, width, bytes)) != CQ_OK) return st;
    if (slots == nullptr) return CQ_ERR_INVALID_ARG;
    if (!aligned_to(slots, 8)) return CQ_ERR_ALIGNMENT;
    cq::DeviceInfo dev;
    if (cq::device_info(&dev) != cudaSuccess) return CQ_ERR_CUDA;
    return status_of(cq::launch_kv_append(dev, c, dtype, T, k, k_stride, v, v_stride, slots,
                                          static_cast<cudaStream_t>(stream)));
}

cq_status cq_kv_read(const cq_kv_cache* cache, cq_dtype dtype, int64_t T, const int64_t* slots, void* k_out,
                     void* v_out, void* stream) {
    if (dtype_bytes(dtype) == 0) return CQ_ERR_UNSUPPORTED_FORMAT;
    if (T < 0) return CQ_ERR_INVALID_ARG;
    cq::KvView c;
    const cq_status st = check_cache(cache, &c);
    if (st != CQ_OK) return st;
    if (T > INT_LIMIT) return CQ_ERR_SHAPE;
    if (T == 0 || (k_out == nullptr && v_out == nullptr)) return CQ_OK;
    if (slots == nullptr) return CQ_ERR_INVALID_ARG;
    if (!aligned_to(slots, 8) || !aligned16(k_out) || !aligned16(v_out)) return CQ_ERR_ALIGNMENT;
    cq::DeviceInfo dev;
    if (cq::device_info(&dev) != cudaSuccess) return CQ_ERR_CUDA;
    return status_of(cq::launch_kv_read(dev, c, dtype, T, slots, k_out, v_out, static_cast<cudaStream_t>(stream)));
}

size_t cq_attn_workspace_size(int64_t q_heads, int64_t kv_heads, int64_t head_dim) {
    if (kv_heads < 1 || q_heads < 1 || q_heads > 1024 || q_heads % kv_heads != 0 || (head_dim != 64 && head_dim != 128))
        return 0;
    return cq::attn_workspace_size(head_dim);
}

cq_status cq_attn_paged(const cq_kv_cache* cache, cq_dtype dtype, int64_t R, int64_t T, int64_t q_heads,
                        int64_t max_new, int64_t max_kv, const void* q, int64_t q_stride, const int32_t* block_table,
                        int64_t max_blocks, const int32_t* kv_len, const int32_t* q_start, float scale, int causal,
                        int64_t window, void* out, int64_t out_stride, float* lse, void* workspace,
                        size_t workspace_bytes, void* stream) {
    if (dtype_bytes(dtype) == 0) return CQ_ERR_UNSUPPORTED_FORMAT;
    if (max_kv < 0) return CQ_ERR_INVALID_ARG;
    return attend(cache, dtype, R, T, q_heads, max_new, q, q_stride, block_table, max_blocks, kv_len, q_start, nullptr, false,
                  scale, causal, window, out, out_stride, lse, workspace, workspace_bytes, stream);
}

cq_status cq_attn_tree(const cq_kv_cache* cache, cq_dtype dtype, int64_t R, int64_t T, int64_t q_heads,
                       int64_t max_new, const void* q, int64_t q_stride, const int32_t* block_table,
                       int64_t max_blocks, const int32_t* kv_len, const int32_t* q_start, const uint64_t* mask,
                       float scale, void* out, int64_t out_stride, float* lse, void* workspace, size_t workspace_bytes,
                       void* stream) {
    return attend(cache, dtype, R, T, q_heads, max_new, q, q_stride, block_table, max_blocks, kv_len, q_start, mask, true,
                  scale, 1, 0, out, out_stride, lse, workspace, workspace_bytes, stream);
}

cq_status cq_qk_rope(cq_dtype in, cq_dtype out, int64_t T, int64_t q_heads, int64_t kv_heads, int64_t head_dim,
                     int64_t rot_dim, int adjacent, const void* q, int64_t q_stride, const void* k, int64_t k_stride,
                     const int32_t* positions, const double* freqs, const float* q_norm, const float* k_norm, float eps,
                     void* q_out, int64_t q_out_stride, void* k_out, int64_t k_out_stride, void* stream) {
    const int bi = dtype_bytes(in), bo = dtype_bytes(out);
    if (bi == 0 || bo == 0 || (in != out && in != CQ_F32)) return CQ_ERR_UNSUPPORTED_FORMAT;
    if (T < 0 || q_heads < 0 || kv_heads < 0 || head_dim < 0 || rot_dim < 0 || (adjacent != 0 && adjacent != 1) || !(eps >= 0.0f))
        return CQ_ERR_INVALID_ARG;
    if ((head_dim != 64 && head_dim != 128) || rot_dim > head_dim || rot_dim % 8 != 0 || q_heads > 1024 || kv_heads > 1024 ||
        T > INT_LIMIT)
        return CQ_ERR_SHAPE;
    if (T == 0 || q_heads + kv_heads == 0) return CQ_OK;
    if (positions == nullptr || (rot_dim > 0 && freqs == nullptr)) return CQ_ERR_INVALID_ARG;
    if (!aligned4(positions) || !aligned_to(freqs, 8)) return CQ_ERR_ALIGNMENT;
    cq::RopeArgs a{};
    const void* x[2] = {q, k};
    void* y[2] = {q_out, k_out};
    const float* w[2] = {q_norm, k_norm};
    const int64_t heads[2] = {q_heads, kv_heads}, xs[2] = {q_stride, k_stride}, ys[2] = {q_out_stride, k_out_stride};
    for (int i = 0; i < 2; ++i) {
        if (heads[i] == 0) continue;
        cq_status st = check_rows(x[i], xs[i], heads[i] * head_dim, bi);
        if (st == CQ_OK) st = check_rows(y[i], ys[i], heads[i] * head_dim, bo);
        if (st != CQ_OK) return st;
        if (!aligned16(w[i])) return CQ_ERR_ALIGNMENT;
        if (x[i] == y[i] && (in != out || xs[i] != ys[i])) return CQ_ERR_INVALID_ARG;
        a.x[i] = x[i]; a.y[i] = y[i]; a.w[i] = w[i];
        a.x_stride[i] = xs[i]; a.y_stride[i] = ys[i];
        a.heads[i] = static_cast<int>(heads[i]);
    }
    a.positions = positions; a.freqs = freqs; a.eps = eps;
    a.T = static_cast<int>(T); a.rot = static_cast<int>(rot_dim); a.adjacent = adjacent;
    cq::DeviceInfo dev;
    if (cq::device_info(&dev) != cudaSuccess) return CQ_ERR_CUDA;
    return status_of(cq::launch_qk_rope(dev, in, out, head_dim, a, static_cast<cudaStream_t>(stream)));
}

cq_status cq_tree_plan(int64_t R, int64_t T, const int32_t* kv_len, const int32_t* q_start, const int32_t* parent,
                       uint64_t* mask, int32_t* positions, void* stream) {
    if (R < 0 || T < 0) return CQ_ERR_INVALID_ARG;
    if (R > 16384 || T > INT_LIMIT) return CQ_ERR_SHAPE;
    if (T == 0 || (mask == nullptr && positions == nullptr)) return CQ_OK;
    if (parent == nullptr || (R > 0 && (kv_len == nullptr || q_start == nullptr))) return CQ_ERR_INVALID_ARG;
    if (!aligned4(kv_len) || !aligned4(q_start) || !aligned4(parent) || !aligned4(positions) || !aligned_to(mask, 8))
        return CQ_ERR_ALIGNMENT;
    cq::DeviceInfo dev;
    if (cq::device_info(&dev) != cudaSuccess) return CQ_ERR_CUDA;
    return status_of(cq::launch_tree_plan(dev, static_cast<int>(R), static_cast<int>(T), kv_len, q_start, parent, mask,
                                          positions, static_cast<cudaStream_t>(stream)));
}

cq_status cq_tree_verify(int64_t R, int64_t T, int64_t V, const float* logits, int64_t logits_stride, const float* draft,
                         int64_t draft_stride, const int32_t* tokens, const int32_t* parent, const int32_t* q_start,
                         const float* temperature, const float* u_accept, const float* u_sample, int64_t max_path,
                         int32_t* count, int32_t* path, int32_t* next, void* stream) {
    if (R < 0 || T < 0 || V < 1 || max_path < 1) return CQ_ERR_INVALID_ARG;
    if (R > 16384 || T > INT_LIMIT || V > 262144 || max_path > CQ_TREE_MAX) return CQ_ERR_SHAPE;
    if (R == 0) return CQ_OK;
    if (q_start == nullptr || temperature == nullptr || u_sample == nullptr || count == nullptr || path == nullptr || next == nullptr ||
        (T > 0 && (logits == nullptr || tokens == nullptr || parent == nullptr || u_accept == nullptr)))
        return CQ_ERR_INVALID_ARG;
    const int64_t most = int64_t(1) << 40;
    if (T > 0 && (logits_stride < V || logits_stride > most || (draft != nullptr && (draft_stride < V || draft_stride > most))))
        return CQ_ERR_SHAPE;
    const void* words[] = {logits, draft, tokens, parent, q_start, temperature, u_accept, u_sample, count, path, next};
    for (const void* p : words)
        if (!aligned4(p)) return CQ_ERR_ALIGNMENT;
    cq::DeviceInfo dev;
    if (cq::device_info(&dev) != cudaSuccess) return CQ_ERR_CUDA;
    cq::VerifyArgs a{};
    a.logits = logits; a.draft = draft;
    a.logits_stride = logits_stride; a.draft_stride = draft_stride;
    a.tokens = tokens; a.parent = parent; a.q_start = q_start;
    a.temperature = temperature; a.u_accept = u_accept; a.u_sample = u_sample;
    a.count = count; a.path = path; a.next = next;
    a.status = dev.status;
    a.R = static_cast<int>(R); a.T = static_cast<int>(T); a.V = static_cast<int>(V); a.max_path = static_cast<int>(max_path);
    return status_of(cq::launch_tree_verify(dev, a, static_cast<cudaStream_t>(stream)));
}

cq_status cq_kv_move(const cq_kv_cache* cache, int64_t R, const int32_t* block_table, int64_t max_blocks,
                     const int32_t* kv_len, const int32_t* q_start, const int32_t* count, const int32_t* path,
                     int64_t max_path, int32_t* new_len, void* stream) {
    if (R < 0 || max_blocks < 0 || max_path < 1) return CQ_ERR_INVALID_ARG;
    cq::KvView c;
    const cq_status st = check_cache(cache, &c);
    if (st != CQ_OK) return st;
    if (R > 16384 || max_path > CQ_TREE_MAX || max_blocks > (INT_LIMIT >> c.page_shift)) return CQ_ERR_SHAPE;
    if (R == 0) return CQ_OK;
    if (kv_len == nullptr || q_start == nullptr || count == nullptr || path == nullptr || (max_blocks > 0 && block_table == nullptr))
        return CQ_ERR_INVALID_ARG;
    const void* words[] = {block_table, kv_len, q_start, count, path, new_len};
    for (const void* p : words)
        if (!aligned4(p)) return CQ_ERR_ALIGNMENT;
    cq::DeviceInfo dev;
    if (cq::device_info(&dev) != cudaSuccess) return CQ_ERR_CUDA;
    const cq::MoveArgs a{block_table, kv_len, q_start, count, path, new_len, dev.status, max_blocks, static_cast<int>(R),
                         static_cast<int>(max_path)};
    return status_of(cq::launch_kv_move(dev, c, a, static_cast<cudaStream_t>(stream)));
}

cq_status cq_kv_release(int64_t R, int64_t page_size, const int32_t* block_table, int64_t max_blocks, int64_t num_pages,
                        const int32_t* old_len, const int32_t* new_len, int32_t* freed, int64_t capacity, int32_t* used,
                        void* stream) {
    if (R < 0 || max_blocks < 0 || num_pages < 0 || capacity < 0) return CQ_ERR_INVALID_ARG;
    const int shift = page_shift(page_size);
    if (shift < 0 || R > 16384 || capacity > INT_LIMIT || num_pages > INT_LIMIT || max_blocks > (INT_LIMIT >> shift))
        return CQ_ERR_SHAPE;
    if (used == nullptr || (capacity > 0 && freed == nullptr) ||
        (R > 0 && (old_len == nullptr || new_len == nullptr || (max_blocks > 0 && block_table == nullptr))))
        return CQ_ERR_INVALID_ARG;
    const void* words[] = {block_table, old_len, new_len, freed, used};
    for (const void* p : words)
        if (!aligned4(p)) return CQ_ERR_ALIGNMENT;
    cq::DeviceInfo dev;
    if (cq::device_info(&dev) != cudaSuccess) return CQ_ERR_CUDA;
    return status_of(cq::launch_kv_release(dev, static_cast<int>(R), shift, block_table, max_blocks, num_pages, old_len, new_len,
                                           freed, static_cast<int>(capacity), used, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
