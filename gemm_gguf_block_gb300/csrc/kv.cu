// The 8-bit paged key/value cache: block tables and slot maps from request
// lengths, writing and reading rows (include/cq.h: cq_kv_plan, cq_kv_append,
// cq_kv_read).
#include <algorithm>

#include "cq_device.cuh"
#include "cq_internal.h"
#include "kv.cuh"

namespace cq {
namespace {

constexpr int PLAN_THREADS = 512;

struct PlanParams {
    const int32_t* past;
    const int32_t* fresh;
    const int32_t* free_pages;
    int32_t* table;
    int32_t* kv_len;
    int32_t* q_start;
    int64_t* slots;
    int32_t* positions;
    int32_t* used;
    int64_t max_blocks, num_pages;
    int R, T, n_free, shift;
};

// Last index i of the ascending v[0..n] with v[i] <= x, given v[0] <= x < v[n].
__device__ __forceinline__ int last_le(const int* v, int n, int x) {
    int lo = 0, hi = n;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (v[mid] <= x) lo = mid; else hi = mid;
    }
    return lo;
}

// Every CTA scans all requests' (new tokens, new pages) into shared memory --
// at most 16384 of each, read from L2 -- and then fills its share of the new
// table entries and of the tokens, finding each one's request by bisection. One
// launch without a second pass over the requests, and no CTA waits for
// another: the entries that the tokens' slots need are computed from the free
// list, not read from the table that others are writing.
__global__ void __launch_bounds__(PLAN_THREADS) kv_plan_kernel(const PlanParams p) {
    pdl_trigger();
    pdl_wait();
    extern __shared__ int plan_smem[];
    int* qs = plan_smem;                  // [R + 1] first token of each request (stops at T)
    int* ps = plan_smem + p.R + 1;        // [R + 1] first new page of each request (stops at n_free)
    __shared__ int64_t warp_sum[2][PLAN_THREADS / 32];
    __shared__ int flags;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int P1 = (1 << p.shift) - 1;
    if (tid == 0) flags = 0;
    __syncthreads();
    int64_t carry[2] = {0, 0};
    int bad = 0;
    for (int r0 = 0; r0 < p.R; r0 += PLAN_THREADS) {
        const int r = r0 + tid;
        int64_t x[2] = {0, 0};
        if (r < p.R) {
            int past = p.past[r], fresh = p.fresh[r];
            if (past < 0 || fresh < 0) { bad |= CQ_DEV_KV_LENGTH; past = max(past, 0); fresh = max(fresh, 0); }
            const int64_t kv = static_cast<int64_t>(past) + fresh;
            const int64_t b0 = (past + int64_t(P1)) >> p.shift, b1 = (kv + P1) >> p.shift;
            if (b1 > p.max_blocks) bad |= CQ_DEV_KV_BLOCKS;
            x[0] = fresh;
            x[1] = min(b1, p.max_blocks) - min(b0, p.max_blocks);
            if (blockIdx.x == 0) p.kv_len[r] = static_cast<int32_t>(min(kv, p.max_blocks << p.shift));
        }
        int64_t s[2] = {x[0], x[1]};
#pragma unroll
        for (int o = 1; o < 32; o <<= 1)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                const int64_t up = __shfl_up_sync(0xffffffffu, s[c], o);
                if (lane >= o) s[c] += up;
            }
        if (lane == 31) { warp_sum[0][warp] = s[0]; warp_sum[1][warp] = s[1]; }
        __syncthreads();
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            int64_t before = 0, all = 0;
            for (int w = 0; w < PLAN_THREADS / 32; ++w) {
                if (w < warp) before += warp_sum[c][w];
                all += warp_sum[c][w];
            }
            const int64_t start = carry[c] + before + s[c] - x[c];
            if (r < p.R) (c == 0 ? qs : ps)[r] = static_cast<int>(min(start, static_cast<int64_t>(c == 0 ? p.T : p.n_free)));
            carry[c] += all;
        }
        __syncthreads();
    }
    if (carry[0] > p.T) bad |= CQ_DEV_KV_TOKENS;
    if (carry[1] > p.n_free) bad |= CQ_DEV_KV_PAGES;
    const int total = static_cast<int>(min(carry[0], static_cast<int64_t>(p.T)));
    const int pages = static_cast<int>(min(carry[1], static_cast<int64_t>(p.n_free)));
    if (tid == 0) { qs[p.R] = total; ps[p.R] = pages; }
    if (bad) atomicOr(&flags, bad);
    __syncthreads();
    const int step = gridDim.x * PLAN_THREADS, first = blockIdx.x * PLAN_THREADS + tid;
    for (int r = first; r <= p.R; r += step) p.q_start[r] = qs[r];
    // Entries that no free page is left for.
    if (carry[1] > p.n_free) {
        for (int r = first; r < p.R; r += step) {
            const int past = max(p.past[r], 0);
            const int64_t b0 = min((past + int64_t(P1)) >> p.shift, p.max_blocks);
            const int64_t b1 = min((static_cast<int64_t>(past) + max(p.fresh[r], 0) + P1) >> p.shift, p.max_blocks);
            for (int64_t b = b0 + (ps[r + 1] - ps[r]); b < b1; ++b) p.table[r * p.max_blocks + b] = -1;
        }
    }
    for (int j = first; j < pages; j += step) {
        const int r = last_le(ps, p.R, j);
        const int64_t b0 = (max(p.past[r], 0) + int64_t(P1)) >> p.shift;
        int page = p.free_pages[j];
        if (page < 0 || page >= p.num_pages) page = -1;
        p.table[r * p.max_blocks + b0 + (j - ps[r])] = page;
    }
    for (int t = first; t < p.T; t += step) {
        int64_t slot = -1;
        int pos = -1;
        if (t < total) {
            const int r = last_le(qs, p.R, t);
            const int past = max(p.past[r], 0);
            pos = past + (t - qs[r]);
            const int64_t b0 = (past + int64_t(P1)) >> p.shift, b = pos >> p.shift;
            int page = -1;
            if (b < p.max_blocks) {
                if (b < b0) page = p.table[r * p.max_blocks + b];
                else if (b - b0 < ps[r + 1] - ps[r]) page = p.free_pages[ps[r] + (b - b0)];
            }
            if (page >= 0 && page < p.num_pages) slot = (static_cast<int64_t>(page) << p.shift) + (pos & P1);
        }
        p.slots[t] = slot;
        p.positions[t] = pos;
    }
    // The status is CTA 0's alone, so that no CTA has to clear it for the others:
    // it looks over every page id that the step uses.
    if (blockIdx.x == 0) {
        int fault = 0;
        for (int j = tid; j < pages; j += PLAN_THREADS) {
            const int page = p.free_pages[j];
            if (page < 0 || page >= p.num_pages) fault = CQ_DEV_KV_PAGE;
        }
        for (int r = tid; r < p.R; r += PLAN_THREADS) {
            const int past = max(p.past[r], 0);
            const int64_t b = past >> p.shift;
            if ((past & P1) == 0 || qs[r + 1] <= qs[r] || b >= p.max_blocks) continue;
            const int page = p.table[r * p.max_blocks + b];
            if (page < 0 || page >= p.num_pages) fault = CQ_DEV_KV_PAGE;
        }
        if (fault) atomicOr(&flags, fault);
        __syncthreads();
        if (tid == 0) { p.used[0] = pages; p.used[1] = flags; }
    }
}

__device__ __forceinline__ float warp_max_bits(float a) {
    // |x| as an integer keeps the order of the values and puts infinities and NaN on top
    return __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(a)));
}

template <typename T>
struct AppendParams {
    KvView c;
    const T* x[2];           // keys, values
    int64_t stride[2];       // elements
    const int64_t* slots;
    int* status;
    int T_;
};

__device__ __forceinline__ uint32_t pack4(int a, int b, int c, int d) {
    return (static_cast<uint32_t>(a) & 0xffu) | ((static_cast<uint32_t>(b) & 0xffu) << 8) |
           ((static_cast<uint32_t>(c) & 0xffu) << 16) | (static_cast<uint32_t>(d) << 24);
}

// A warp takes one (run of tokens that share a page, head, keys or values): it
// owns that block's scale and rows, so nothing is shared between warps. A run
// begins at a token whose slot does not follow its neighbour's or begins a
// page; the warps of the other tokens leave at once.
template <typename T, int D>
__global__ void __launch_bounds__(256) kv_append_kernel(const AppendParams<T> p) {
    pdl_trigger();
    pdl_wait();
    const int lane = threadIdx.x & 31;
    const int64_t unit = (static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x) >> 5;
    const int per = 2 * p.c.heads;
    const int64_t t0 = unit / per;
    if (t0 >= p.T_) return;
    const int which = static_cast<int>(unit - t0 * per) & 1, head = static_cast<int>(unit - t0 * per) >> 1;
    const int P = p.c.page_size;
    const int64_t slot = p.slots[t0];
    if (slot < 0) return;
    const int64_t page = slot >> p.c.page_shift;
    const int off = static_cast<int>(slot & (P - 1));
    if (page >= p.c.num_pages) {
        if (lane == 0) atomicOr(p.status, CQ_DEV_KV_PAGE);
        return;
    }
    if (off != 0 && t0 > 0 && p.slots[t0 - 1] == slot - 1) return;
    int n = 1;
    for (bool on = true; on && off + n < P;) {
        const bool next = off + n + lane < P && t0 + n + lane < p.T_ && p.slots[t0 + n + lane] == slot + n + lane;
        const uint32_t m = __ballot_sync(0xffffffffu, next);
        const int got = m == 0xffffffffu ? 32 : __ffs(~m) - 1;
        n += got;
        on = got == 32;
    }
    // Four values a lane: a row of 128 is a warp's width, two rows of 64 are.
    constexpr int RPW = 128 / D;
    const int sub = lane / (D / 4), col = (lane % (D / 4)) * 4;
    const T* x = p.x[which] + t0 * p.stride[which] + head * D + col;
    const int64_t xs = p.stride[which];
    float a = 0.0f;
    for (int i = sub; i < n; i += RPW) {
        const float4 v = load4(x + i * xs);
        const uint32_t u = max(max(__float_as_uint(fabsf(v.x)), __float_as_uint(fabsf(v.y))),
                               max(__float_as_uint(fabsf(v.z)), __float_as_uint(fabsf(v.w))));
        a = __uint_as_float(max(__float_as_uint(a), u));
    }
    a = warp_max_bits(a);
    float* sp = (which ? p.c.v_scale : p.c.k_scale) + page * p.c.scale_stride + head;
    int8_t* q = (which ? p.c.v : p.c.k) + page * p.c.page_stride + (static_cast<int64_t>(head) * P) * D + col;
    const float old = off == 0 ? 0.0f : *sp;
    float want = q8_scale(a);
    if (want < 1.17549435e-38f) want = 0.0f;
    float s = fmaxf(old, want);
    if (!(a < INFINITY) || old != old) s = __uint_as_float(0x7fffffffu);
    const float inv = s > 0.0f ? __frcp_rn(s) : 0.0f;      // 0 for NaN too: the rows hold zeros then
    if (s != old && off > 0) {
        const float ratio = s > 0.0f ? __fdiv_rn(old, s) : 0.0f;
        for (int i = sub; i < off; i += RPW) {
            const uint32_t w = *reinterpret_cast<const uint32_t*>(q + i * D);
            int r[4];
#pragma unroll
            for (int b = 0; b < 4; ++b) {
                const float h = static_cast<float>(static_cast<int8_t>(w >> (8 * b)));
                r[b] = static_cast<int>(roundf(__fmul_rn(h, ratio)));
            }
            *reinterpret_cast<uint32_t*>(q + i * D) = pack4(r[0], r[1], r[2], r[3]);
        }
    }
    for (int i = sub; i < n; i += RPW) {
        const float4 v = load4(x + i * xs);
        const uint32_t w = inv > 0.0f ? pack4(quant_q8(v.x, inv), quant_q8(v.y, inv), quant_q8(v.z, inv), quant_q8(v.w, inv)) : 0u;
        *reinterpret_cast<uint32_t*>(q + (off + i) * D) = w;
    }
    __syncwarp();
    if (lane == 0) *sp = s;
}

template <typename T>
struct ReadParams {
    KvView c;
    T* out[2];
    const int64_t* slots;
    int* status;
    int64_t n4;              // groups of four values in one output
};

template <typename T, int D>
__global__ void __launch_bounds__(256) kv_read_kernel(const ReadParams<T> p) {
    pdl_trigger();
    pdl_wait();
    const int row4 = p.c.heads * (D / 4);
    const int64_t step = static_cast<int64_t>(gridDim.x) * blockDim.x;
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x; i < p.n4; i += step) {
        const int64_t t = i / row4;
        const int in = static_cast<int>(i - t * row4), head = in / (D / 4), col = (in % (D / 4)) * 4;
        const int64_t slot = p.slots[t];
        const int64_t page = slot >> p.c.page_shift;
        const bool on = slot >= 0 && page < p.c.num_pages;
        if (slot >= 0 && !on) atomicOr(p.status, CQ_DEV_KV_PAGE);
#pragma unroll
        for (int w = 0; w < 2; ++w) {
            if (p.out[w] == nullptr) continue;
            float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            if (on) {
                const int row = static_cast<int>(slot & (p.c.page_size - 1));
                const int8_t* q = (w ? p.c.v : p.c.k) + page * p.c.page_stride + (static_cast<int64_t>(head) * p.c.page_size + row) * D + col;
                const uint32_t u = *reinterpret_cast<const uint32_t*>(q);
                const float s = (w ? p.c.v_scale : p.c.k_scale)[page * p.c.scale_stride + head];
                v = make_float4(s * static_cast<int8_t>(u), s * static_cast<int8_t>(u >> 8),
                                s * static_cast<int8_t>(u >> 16), s * static_cast<int8_t>(u >> 24));
            }
            store4(p.out[w] + i * 4, v);
        }
    }
}

template <typename T>
cudaError_t append_t(const DeviceInfo& dev, const KvView& c, int64_t T_, const void* k, int64_t ks, const void* v,
                     int64_t vs, const int64_t* slots, cudaStream_t s) {
    AppendParams<T> p{c, {static_cast<const T*>(k), static_cast<const T*>(v)}, {ks, vs}, slots, dev.status,
                      static_cast<int>(T_)};
    const int64_t ctas = (T_ * 2 * c.heads + 7) / 8;
    if (ctas > 0x7fffffff) return cudaErrorInvalidConfiguration;
    return launch_kernel(c.dim == 64 ? kv_append_kernel<T, 64> : kv_append_kernel<T, 128>,
                         dim3(static_cast<unsigned>(ctas)), dim3(256), 0, s, p);
}

template <typename T>
cudaError_t read_t(const DeviceInfo& dev, const KvView& c, int64_t T_, const int64_t* slots, void* k, void* v,
                   cudaStream_t s) {
    ReadParams<T> p{c, {static_cast<T*>(k), static_cast<T*>(v)}, slots, dev.status, T_ * c.heads * (c.dim / 4)};
    const int64_t ctas = std::min<int64_t>((p.n4 + 255) / 256, static_cast<int64_t>(dev.sm_count) * 64);
    return launch_kernel(c.dim == 64 ? kv_read_kernel<T, 64> : kv_read_kernel<T, 128>,
                         dim3(static_cast<unsigned>(ctas)), dim3(256), 0, s, p);
}

}  // namespace

cudaError_t launch_kv_plan(const DeviceInfo& dev, int R, int page_shift, int64_t max_blocks, int64_t num_pages,
                           const int32_t* past, const int32_t* fresh, const int32_t* free_pages, int n_free,
                           int32_t* table, int T, int32_t* kv_len, int32_t* q_start, int64_t* slots,
                           int32_t* positions, int32_t* used, cudaStream_t s) {
    PlanParams p{past, fresh, free_pages, table, kv_len, q_start, slots, positions, used,
                 max_blocks, num_pages, R, T, n_free, page_shift};
    const int smem = 2 * (R + 1) * 4;
    cudaError_t e = raise_smem_limit(reinterpret_cast<const void*>(kv_plan_kernel), smem);
    if (e != cudaSuccess) return e;
    const int work = std::max(T, R + 1);
    const int ctas = std::min(dev.sm_count, (work + PLAN_THREADS - 1) / PLAN_THREADS);
    return launch_kernel(kv_plan_kernel, dim3(static_cast<unsigned>(ctas)), dim3(PLAN_THREADS), static_cast<size_t>(smem), s, p);
}

cudaError_t launch_kv_append(const DeviceInfo& dev, const KvView& c, int dtype, int64_t T, const void* k, int64_t ks,
                             const void* v, int64_t vs, const int64_t* slots, cudaStream_t s) {
    switch (dtype) {
    case CQ_F32: return append_t<float>(dev, c, T, k, ks, v, vs, slots, s);
    case CQ_F16: return append_t<__half>(dev, c, T, k, ks, v, vs, slots, s);
    case CQ_BF16: return append_t<__nv_bfloat16>(dev, c, T, k, ks, v, vs, slots, s);
    default: return cudaErrorInvalidValue;
    }
}

cudaError_t launch_kv_read(const DeviceInfo& dev, const KvView& c, int dtype, int64_t T, const int64_t* slots,
                           void* k, void* v, cudaStream_t s) {
    switch (dtype) {
    case CQ_F32: return read_t<float>(dev, c, T, slots, k, v, s);
    case CQ_F16: return read_t<__half>(dev, c, T, slots, k, v, s);
    case CQ_BF16: return read_t<__nv_bfloat16>(dev, c, T, slots, k, v, s);
    default: return cudaErrorInvalidValue;
    }
}

}  // namespace cq
