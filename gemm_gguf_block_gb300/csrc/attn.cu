// Attention over the 8-bit paged cache (cq_attn_paged in include/cq.h).
//
// S = scale * q . (s_k k) over the visible keys, softmax in fp32 with a running
// maximum, out = sum p (s_v v) / sum p.
#include <algorithm>

#include "cq_device.cuh"
#include "cq_internal.h"
#include "kv.cuh"

namespace cq {
namespace {

// One warp per (token, query head): 32 keys at a time, a lane to a key for the
// scores and a lane to D / 32 values for the sum.
template <typename T, int D>
__global__ void __launch_bounds__(256) attn_simple_kernel(const KvView c, const AttnArgs a) {
    pdl_trigger();
    pdl_wait();
    __shared__ float qs[8][D];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t unit = static_cast<int64_t>(blockIdx.x) * 8 + warp;
    const int t = static_cast<int>(unit / a.heads), head = static_cast<int>(unit % a.heads);
    if (t >= a.T) return;
    int lo = 0, hi = a.R;                               // last request that starts at or before t
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (a.q_start[mid] <= t) lo = mid; else hi = mid;
    }
    const int r = lo;
    const int begin = a.q_start[r], end = min(a.q_start[r + 1], a.T);
    if (t < begin || t >= end) return;
    const int64_t limit = a.max_blocks << c.page_shift;
    const int kv = static_cast<int>(min(static_cast<int64_t>(max(a.kv_len[r], 0)), limit));
    const int64_t pos = static_cast<int64_t>(kv) - (a.q_start[r + 1] - begin) + (t - begin);
    const int stop = a.causal ? static_cast<int>(min(static_cast<int64_t>(kv), pos + 1)) : kv;
    const int from = a.window > 0 ? static_cast<int>(max(int64_t(0), pos - a.window + 1)) : 0;
    const int h = head / (a.heads / c.heads);
    const T* q = static_cast<const T*>(a.q) + t * a.q_stride + head * D;
    for (int d = lane; d < D; d += 32) qs[warp][d] = to_f32(q[d]) * a.scale;
    __syncwarp();
    float m = -INFINITY, l = 0.0f, acc[D / 32] = {};
    for (int j0 = from & ~15; j0 < stop; j0 += 16) {    // 16 keys: one page whatever its size
        const int page = a.table[r * a.max_blocks + (j0 >> c.page_shift)];
        if (page < 0 || page >= c.num_pages) {
            if (lane == 0) atomicOr(a.status, CQ_DEV_KV_PAGE);
            continue;
        }
        const int j = j0 + (lane & 15);
        const bool on = j >= from && j < stop;
        const int64_t at = page * c.page_stride + (static_cast<int64_t>(h) * c.page_size + (j0 & (c.page_size - 1))) * D;
        const int8_t* k = c.k + at + (lane & 15) * D + (lane >> 4) * (D / 2);
        float s = 0.0f;
        for (int d = 0; d < D / 2; ++d) s = fmaf(qs[warp][(lane >> 4) * (D / 2) + d], static_cast<float>(k[d]), s);
        s += __shfl_xor_sync(0xffffffffu, s, 16);
        s = on ? s * c.k_scale[page * c.scale_stride + h] : -INFINITY;
        float top = s;
#pragma unroll
        for (int o = 8; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
        const float m2 = fmaxf(m, top), base = m2 == -INFINITY ? 0.0f : m2;
        const float f = expf(m - base);
        const float e = on ? expf(s - base) : 0.0f;
        float sum = e;
#pragma unroll
        for (int o = 8; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        l = l * f + sum;
        m = m2;
        const float sv = c.v_scale[page * c.scale_stride + h];
#pragma unroll
        for (int i = 0; i < D / 32; ++i) acc[i] *= f;
        for (int jj = 0; jj < 16; ++jj) {
            if (j0 + jj < from || j0 + jj >= stop) continue;
            const float p = __shfl_sync(0xffffffffu, e, jj) * sv;
#pragma unroll
            for (int i = 0; i < D / 32; ++i) acc[i] = fmaf(p, static_cast<float>(c.v[at + jj * D + lane + 32 * i]), acc[i]);
        }
    }
    T* out = static_cast<T*>(a.out) + t * a.out_stride + head * D;
    const float inv = l == 0.0f ? 0.0f : 1.0f / l;      // l is 0 only where nothing was visible; NaN stays NaN
    for (int i = 0; i < D / 32; ++i) {
        const float v = acc[i] * inv;
        if constexpr (sizeof(T) == 4) out[lane + 32 * i] = v;
        else if constexpr (std::is_same<T, __half>::value) out[lane + 32 * i] = __float2half_rn(v);
        else out[lane + 32 * i] = __float2bfloat16_rn(v);
    }
    if (a.lse != nullptr && lane == 0) a.lse[static_cast<int64_t>(t) * a.heads + head] = m + logf(l);
}

template <typename T>
cudaError_t launch_simple(const KvView& c, const AttnArgs& a, cudaStream_t s) {
    const int64_t ctas = (static_cast<int64_t>(a.T) * a.heads + 7) / 8;
    if (ctas > 0x7fffffff) return cudaErrorInvalidConfiguration;
    return launch_kernel(c.dim == 64 ? attn_simple_kernel<T, 64> : attn_simple_kernel<T, 128>,
                         dim3(static_cast<unsigned>(ctas)), dim3(256), 0, s, c, a);
}

}  // namespace

size_t attn_workspace_size(int64_t, int64_t, int64_t) { return 256; }

cudaError_t launch_attn(const DeviceInfo&, const KvView& c, int dtype, const AttnArgs& a, cudaStream_t s) {
    switch (dtype) {
    case CQ_F32: return launch_simple<float>(c, a, s);
    case CQ_F16: return launch_simple<__half>(c, a, s);
    case CQ_BF16: return launch_simple<__nv_bfloat16>(c, a, s);
    default: return cudaErrorInvalidValue;
    }
}

}  // namespace cq
