// The 8-bit paged key/value cache: block tables and slot maps from request
// lengths, writing and reading rows (include/cq_kv.h: cq_kv_plan, cq_kv_append,
// cq_kv_read).
#include <algorithm>
#include <type_traits>

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
    // (indices in 64 bits: pages and T may be near 2^31, where a step more passes 32)
    for (int64_t j = first; j < pages; j += step) {
        const int r = last_le(ps, p.R, static_cast<int>(j));
        const int64_t b0 = (max(p.past[r], 0) + int64_t(P1)) >> p.shift;
        int page = p.free_pages[j];
        if (page < 0 || page >= p.num_pages) page = -1;
        p.table[r * p.max_blocks + b0 + (j - ps[r])] = page;
    }
    for (int64_t t = first; t < p.T; t += step) {
        int64_t slot = -1;
        int pos = -1;
        if (t < total) {
            const int r = last_le(qs, p.R, static_cast<int>(t));
            const int past = max(p.past[r], 0);
            const int64_t at = static_cast<int64_t>(past) + (t - qs[r]);         // passes 32 bits where past + new does
            const int64_t b0 = (past + int64_t(P1)) >> p.shift, b = at >> p.shift;
            int page = -1;
            if (b < p.max_blocks) {
                if (b < b0) page = p.table[r * p.max_blocks + b];
                else if (b - b0 < ps[r + 1] - ps[r]) page = p.free_pages[ps[r] + (b - b0)];
            }
            if (page >= 0 && page < p.num_pages) slot = (static_cast<int64_t>(page) << p.shift) + (at & P1);
            if (at <= 0x7fffffff) pos = static_cast<int>(at);
        }
        p.slots[t] = slot;
        p.positions[t] = pos;
    }
    // The status is CTA 0's alone, so that no CTA has to clear it for the others:
    // it looks over every page id that the step uses.
    if (blockIdx.x == 0) {
        int fault = 0;
        for (int64_t j = tid; j < pages; j += PLAN_THREADS) {
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

template <typename T>
struct AppendParams {
    KvView c;
    const T* xk;
    const T* xv;
    int64_t k_stride, v_stride;      // elements
    const int64_t* slots;
    int* status;
    int T_;
    int slice;               // tokens whose runs one CTA takes, at most 128
};

__device__ __forceinline__ float max3_nan(float a, float b, float c) {      // NaN if any is
    float y;
    asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(y) : "f"(a), "f"(b), "f"(c));
    return y;
}

constexpr int APPEND_WARPS = 8;

// A run is a stretch of tokens that lie one after another in one page: it begins
// at a token whose slot does not follow its neighbour's or begins a page. A CTA
// takes the runs that begin in a slice of tokens, for one head's keys or values:
// it alone changes those blocks' scales and rows. A run belongs to one warp for
// every 16 tokens of a page, each holding its 16 rows in registers between the
// largest value and the rounding, so that the new rows are read once, all of
// a warp's loads in flight together (8 KB at fp32).
template <typename T, int D>
__global__ void __launch_bounds__(APPEND_WARPS * 32) kv_append_kernel(const AppendParams<T> p) {
    pdl_trigger();
    pdl_wait();
    __shared__ int64_t slot_of[2 * 128 + 1];   // slots of tokens t0 - 1 .. t0 + slice + P - 1
    __shared__ int16_t start[128];             // the runs' first tokens, from t0
    __shared__ int runs;
    __shared__ uint32_t top[APPEND_WARPS];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int P = p.c.page_size, head = blockIdx.y >> 1, which = blockIdx.y & 1;
    const int64_t t0 = static_cast<int64_t>(blockIdx.x) * p.slice, stride = which ? p.v_stride : p.k_stride;
    for (int i = tid; i <= p.slice + P; i += APPEND_WARPS * 32) {
        const int64_t t = t0 - 1 + i;
        slot_of[i] = t >= 0 && t < p.T_ ? p.slots[t] : -2;
    }
    __syncthreads();
    if (warp == 0) {
        int count = 0;
        for (int i0 = 0; i0 < p.slice; i0 += 32) {
            const int i = i0 + lane;
            bool begins = false;
            if (i < p.slice) {
                const int64_t s = slot_of[i + 1];
                const bool inside = s >= 0 && (s >> p.c.page_shift) < p.c.num_pages;
                begins = inside && ((s & (P - 1)) == 0 || slot_of[i] != s - 1);
                if (s >= 0 && !inside) atomicOr(p.status, CQ_DEV_KV_PAGE);
            }
            const uint32_t m = __ballot_sync(0xffffffffu, begins);
            if (begins) start[count + __popc(m & ((1u << lane) - 1))] = static_cast<int16_t>(i);
            count += __popc(m);
        }
        if (lane == 0) runs = count;
    }
    __syncthreads();
    const int wpr = P / 16;                                     // warps of a run
    const int group = warp / wpr, part = warp % wpr, groups = APPEND_WARPS / wpr;
    constexpr int RPW = 128 / D, NL = 16 / RPW;                 // rows of a load, loads
    const int sub = lane / (D / 4), col = (lane % (D / 4)) * 4;
    for (int r = group; r < runs; r += groups) {
        const int i0 = start[r];
        const int64_t slot = slot_of[i0 + 1], page = slot >> p.c.page_shift;
        const int off = static_cast<int>(slot & (P - 1));
        int n = 1;                                              // tokens of the run
        for (bool on = true; on && off + n < P;) {
            const bool next = off + n + lane < P && slot_of[i0 + 1 + min(n + lane, P)] == slot + n + lane;
            const uint32_t m = __ballot_sync(0xffffffffu, next);
            const int got = m == 0xffffffffu ? 32 : __ffs(~m) - 1;
            n += got;
            on = got == 32;
        }
        float* sp = (which ? p.c.v_scale : p.c.k_scale) + page * p.c.scale_stride + head;
        const float old = off == 0 ? 0.0f : *sp;
        const T* x = (which ? p.xv : p.xk) + (t0 + i0) * stride + head * D + col;
        Raw4<T> v[NL];
        const int row0 = 16 * part + sub;
        const T* xr = x + row0 * stride;
#pragma unroll
        for (int k = 0; k < NL; ++k) {
            v[k].zero();
            if (row0 + k * RPW < n) v[k].load(xr);
            xr += RPW * stride;
        }
        float far = 0.0f;
#pragma unroll
        for (int k = 0; k < NL; ++k) {
            const float4 f = v[k].value();
            far = max3_nan(max3_nan(far, fabsf(f.x), fabsf(f.y)), fabsf(f.z), fabsf(f.w));
        }
        uint32_t a = __float_as_uint(far);                      // as an integer: the same order, infinities and NaN on top
        a = __reduce_max_sync(0xffffffffu, a);
        if (wpr > 1) {
            if (lane == 0) top[warp] = a;
            asm volatile("bar.sync %0, %1;" ::"r"(1 + group), "r"(32 * wpr) : "memory");
            for (int w = 0; w < wpr; ++w) a = max(a, top[group * wpr + w]);
        }
        float want = q8_scale(__uint_as_float(a));
        if (want < 1.17549435e-38f) want = 0.0f;
        float s = fmaxf(old, want);
        if (a >= 0x7f800000u || old != old) s = __uint_as_float(0x7fffffffu);
        const float inv = s > 0.0f ? __frcp_rn(s) : 0.0f;       // 0 for NaN too: the rows hold zeros then
        int8_t* q = (which ? p.c.v : p.c.k) + page * p.c.page_stride + static_cast<int64_t>(head) * P * D + col;
        if (s != old && off > 0) {
            const float ratio = s > 0.0f ? __fdiv_rn(old, s) : 0.0f;
            for (int i = row0; i < min(off, 16 * part + 16); i += RPW) {
                const uint32_t w = *reinterpret_cast<const uint32_t*>(q + i * D);
                int z[4];
#pragma unroll
                for (int b = 0; b < 4; ++b) {
                    const float h = static_cast<float>(static_cast<int8_t>(w >> (8 * b)));
                    z[b] = round_away(__fmul_rn(h, ratio));
                }
                *reinterpret_cast<uint32_t*>(q + i * D) = pack4(z[0], z[1], z[2], z[3]);
            }
        }
#pragma unroll
        for (int k = 0; k < NL; ++k) {
            const int i = row0 + k * RPW;
            const float4 f = v[k].value();
            const uint32_t w = inv > 0.0f ? pack4(round_away(__fmul_rn(f.x, inv)), round_away(__fmul_rn(f.y, inv)),
                                              round_away(__fmul_rn(f.z, inv)), round_away(__fmul_rn(f.w, inv))) : 0u;
            if (i < n) *reinterpret_cast<uint32_t*>(q + static_cast<int64_t>(off + i) * D) = w;
        }
        // every warp has the old scale before it is replaced, and the largest values before the next run's
        if (wpr > 1) asm volatile("bar.sync %0, %1;" ::"r"(1 + group), "r"(32 * wpr) : "memory");
        if (part == 0 && lane == 0) *sp = s;
    }
}

template <typename T>
struct ReadParams {
    KvView c;
    T* k_out;
    T* v_out;
    const int64_t* slots;
    int* status;
    int T_;
};

// A thread keeps its place in a row (head, four dimensions) and goes down the tokens,
// four of them in flight: rows are read and written whole by neighbouring threads.
template <typename T, int D>
__global__ void __launch_bounds__(256) kv_read_kernel(const ReadParams<T> p) {
    pdl_trigger();
    pdl_wait();
    constexpr int BATCH = 4;
    const int row4 = p.c.heads * (D / 4);
    const int per = row4 < 256 ? 256 / row4 : 1;                // tokens of a CTA side by side
    const int sub = row4 < 256 ? threadIdx.x / row4 : 0;
    if (sub >= per) return;
    const int shift = p.c.page_shift, mask = p.c.page_size - 1;
    for (int in = row4 < 256 ? threadIdx.x - sub * row4 : threadIdx.x; in < row4; in += 256) {
        const int head = in / (D / 4), col = (in % (D / 4)) * 4;
        for (int64_t tb = static_cast<int64_t>(blockIdx.x) * per * BATCH + sub; tb < p.T_; tb += static_cast<int64_t>(gridDim.x) * per * BATCH) {
            int64_t slot[BATCH];
            uint32_t u[2][BATCH];
            float sc[2][BATCH];
#pragma unroll
            for (int b = 0; b < BATCH; ++b) {
                const int64_t t = tb + b * per;
                slot[b] = t < p.T_ ? p.slots[t] : -1;
                if (slot[b] >= 0 && (slot[b] >> shift) >= p.c.num_pages) {
                    atomicOr(p.status, CQ_DEV_KV_PAGE);
                    slot[b] = -1;
                }
            }
#pragma unroll
            for (int b = 0; b < BATCH; ++b) {
                const int64_t page = slot[b] >> shift;
                const int64_t at = page * p.c.page_stride + (static_cast<int64_t>(head) * p.c.page_size + (slot[b] & mask)) * D + col;
#pragma unroll
                for (int w = 0; w < 2; ++w) {
                    u[w][b] = 0;
                    sc[w][b] = 0.0f;
                    if (slot[b] >= 0 && (w ? p.v_out : p.k_out) != nullptr) {
                        u[w][b] = *reinterpret_cast<const uint32_t*>((w ? p.c.v : p.c.k) + at);
                        sc[w][b] = (w ? p.c.v_scale : p.c.k_scale)[page * p.c.scale_stride + head];
                    }
                }
            }
#pragma unroll
            for (int b = 0; b < BATCH; ++b) {
                const int64_t t = tb + b * per;
                if (t >= p.T_) continue;
#pragma unroll
                for (int w = 0; w < 2; ++w)
                    if ((w ? p.v_out : p.k_out) != nullptr)
                        store4((w ? p.v_out : p.k_out) + t * (row4 * 4) + in * 4,
                               make_float4(sc[w][b] * static_cast<int8_t>(u[w][b]), sc[w][b] * static_cast<int8_t>(u[w][b] >> 8),
                                           sc[w][b] * static_cast<int8_t>(u[w][b] >> 16), sc[w][b] * static_cast<int8_t>(u[w][b] >> 24)));
            }
        }
    }
}

template <typename T>
cudaError_t append_t(const DeviceInfo& dev, const KvView& c, int64_t T_, const void* k, int64_t ks, const void* v,
                     int64_t vs, const int64_t* slots, cudaStream_t s) {
    // Runs for all of a CTA's warps: 128 tokens where there are plenty (a page for each group of
    // warps); with few tokens, whose runs are short, a token for each group.
    const int groups = APPEND_WARPS / (c.page_size / 16);
    const int slice = (T_ + 127) / 128 * 2 * c.heads >= dev.sm_count ? 128 : groups;
    AppendParams<T> p{c, static_cast<const T*>(k), static_cast<const T*>(v), ks, vs, slots, dev.status,
                      static_cast<int>(T_), slice};
    return launch_kernel(c.dim == 64 ? kv_append_kernel<T, 64> : kv_append_kernel<T, 128>,
                         dim3(static_cast<unsigned>((T_ + slice - 1) / slice), 2 * c.heads), dim3(APPEND_WARPS * 32), 0, s, p);
}

template <typename T>
cudaError_t read_t(const DeviceInfo& dev, const KvView& c, int64_t T_, const int64_t* slots, void* k, void* v,
                   cudaStream_t s) {
    ReadParams<T> p{c, static_cast<T*>(k), static_cast<T*>(v), slots, dev.status, static_cast<int>(T_)};
    const int row4 = c.heads * (c.dim / 4), per = row4 < 256 ? 256 / row4 : 1;
    const int64_t ctas = std::min<int64_t>((T_ + per * 4 - 1) / (per * 4), static_cast<int64_t>(dev.sm_count) * 32);
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
    const int64_t work = std::max(T, R + 1);
    const int64_t ctas = std::min<int64_t>(dev.sm_count, (work + PLAN_THREADS - 1) / PLAN_THREADS);
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
