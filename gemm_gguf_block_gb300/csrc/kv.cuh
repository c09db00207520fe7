// The 8-bit paged key/value cache inside the library: its view (cq_kv_cache in
// include/cq_kv.h), the launchers of its kernels and of the attention over it, and
// the conversions of the value types they take.
#pragma once
#include <cstdint>

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "cq_device.cuh"
#include "cq_internal.h"
#include "cq_kv.h"

namespace cq {

struct KvView {
    int8_t* k;
    int8_t* v;
    float* k_scale;
    float* v_scale;
    int64_t num_pages;
    int64_t page_stride;     // bytes
    int64_t scale_stride;    // floats
    int page_size;
    int page_shift;          // log2(page_size)
    int heads;
    int dim;
};

cudaError_t launch_kv_plan(const DeviceInfo& dev, int R, int page_shift, int64_t max_blocks, int64_t num_pages,
                           const int32_t* past, const int32_t* fresh, const int32_t* free_pages, int n_free,
                           int32_t* table, int T, int32_t* kv_len, int32_t* q_start, int64_t* slots,
                           int32_t* positions, int32_t* used, cudaStream_t s);
cudaError_t launch_kv_append(const DeviceInfo& dev, const KvView& c, int dtype, int64_t T, const void* k, int64_t ks,
                             const void* v, int64_t vs, const int64_t* slots, cudaStream_t s);
cudaError_t launch_kv_read(const DeviceInfo& dev, const KvView& c, int dtype, int64_t T, const int64_t* slots,
                           void* k, void* v, cudaStream_t s);

// Attention arguments past the cache view (cq_attn_paged).
struct AttnArgs {
    const void* q;
    void* out;
    float* lse;
    const int32_t* table;
    const int32_t* kv_len;
    const int32_t* q_start;
    int* status;
    void* ws;
    int64_t q_stride, out_stride;   // elements
    int64_t max_blocks, window;
    int64_t max_new;                // at most T
    float scale;
    int R, T, heads, causal;        // heads: query heads
};
size_t attn_workspace_size(int64_t head_dim);
cudaError_t launch_attn(const DeviceInfo& dev, const KvView& c, int dtype, const AttnArgs& a, cudaStream_t s);

// Four fp32 values rounded to nearest even, stored as 16 or 8 bytes.
__device__ __forceinline__ void store4(float* p, float4 v) { *reinterpret_cast<float4*>(p) = v; }
__device__ __forceinline__ void store4(__half* p, float4 v) {
    const __half2 a = __floats2half2_rn(v.x, v.y), b = __floats2half2_rn(v.z, v.w);
    *reinterpret_cast<uint2*>(p) =
        make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
}
__device__ __forceinline__ void store4(__nv_bfloat16* p, float4 v) {
    const __nv_bfloat162 a = __floats2bfloat162_rn(v.x, v.y), b = __floats2bfloat162_rn(v.z, v.w);
    *reinterpret_cast<uint2*>(p) =
        make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
}
}  // namespace cq
