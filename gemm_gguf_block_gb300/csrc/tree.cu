// A tree step's bookkeeping (include/cq_tree.h): masks and positions from parents,
// the rows of the kept tokens moved together in the cache, pages given back.
#include <algorithm>

#include "tree.cuh"

namespace cq {
namespace {

constexpr int MAX = CQ_TREE_MAX;

// First token, new tokens (both clipped to T) and length of request r.
__device__ __forceinline__ void tokens_of(const int32_t* q_start, int T, int r, int& first, int& n) {
    first = min(max(q_start[r], 0), T);
    n = max(min(q_start[r + 1], T) - first, 0);
}

constexpr int PLAN_THREADS = 256;
constexpr int GROUPS = PLAN_THREADS / MAX;         // requests of a CTA at a time

// A thread a token walks up its own ancestors in shared memory: trees are a few
// generations deep, and the longest walk is 63 reads of about 30 cycles. Bounded by the
// launch: a round of requests is a load, a barrier and the walks.
__global__ void __launch_bounds__(PLAN_THREADS) tree_plan_kernel(int R, int T, const int32_t* kv_len, const int32_t* q_start,
                                                                 const int32_t* parent, uint64_t* mask, int32_t* positions,
                                                                 int* status) {
    pdl_trigger();
    pdl_wait();
    __shared__ int8_t up[GROUPS][MAX];
    const int tid = threadIdx.x, grp = tid / MAX, i = tid % MAX;
    auto write = [&](int64_t t, uint64_t m, int64_t pos) {
        if (mask != nullptr) mask[t] = m;
        if (positions != nullptr) positions[t] = pos >= 0 && pos <= 0x7fffffff ? static_cast<int32_t>(pos) : -1;
    };
    for (int r0 = blockIdx.x * GROUPS; r0 < R; r0 += gridDim.x * GROUPS) {
        const int r = r0 + grp;
        int first = 0, n = 0;
        int64_t base = 0;
        if (r < R) {
            tokens_of(q_start, T, r, first, n);
            base = static_cast<int64_t>(kv_len[r]) - n;
        }
        if (i < n && n <= MAX) {
            int p = parent[first + i];
            if (p < -1 || p >= i) {
                atomicOr(status, CQ_DEV_TREE);
                p = -1;
            }
            up[grp][i] = static_cast<int8_t>(p);
        }
        __syncthreads();
        if (n > MAX) {
            for (int64_t t = i; t < n; t += MAX) write(first + t, 0, base + t);      // (n may be near 2^31, where a step more passes 32 bits)
        } else if (i < n) {
            uint64_t m = 0;
            int depth = -1;
            for (int j = i; j >= 0; j = up[grp][j]) {      // each step goes to a smaller index
                m |= uint64_t(1) << j;
                ++depth;
            }
            write(static_cast<int64_t>(first) + i, m, base + depth);
        }
        __syncthreads();
    }
    // padding
    const int begin = R > 0 ? min(max(q_start[0], 0), T) : 0, end = R > 0 ? min(max(q_start[R], 0), T) : 0;
    const int64_t me = static_cast<int64_t>(blockIdx.x) * PLAN_THREADS + tid, all = static_cast<int64_t>(gridDim.x) * PLAN_THREADS;
    for (int64_t t = me; t < begin; t += all) write(t, 0, -1);
    for (int64_t t = end + me; t < T; t += all) write(t, 0, -1);
}

constexpr int MOVE_THREADS = 128;
constexpr int MOST_PAGES = MAX / 16 + 1;           // pages that 64 positions touch, at most

// A CTA moves the rows of one (request, head) of the keys or the values: all of them, and the scales
// of their pages, are in shared memory before anything is written, so that the path may be any. One
// CTA owns those blocks: nothing waits for another. Bounded by the launch and four dependent loads
// (lengths, path, table, rows): the rows of a step are a few megabytes.
template <int D>
__global__ void __launch_bounds__(MOVE_THREADS) kv_move_kernel(const KvView c, const MoveArgs a) {
    pdl_trigger();
    pdl_wait();
    __shared__ __align__(16) uint32_t rows[MAX][D / 4];
    __shared__ int16_t src[MAX];                   // where row i comes from: its index, or -1: it stays
    __shared__ int page[MOST_PAGES];               // of the request's new tokens; -1: none
    __shared__ float old[MOST_PAGES], now[MOST_PAGES];
    __shared__ int gets[MOST_PAGES];               // whether rows come to it
    const int tid = threadIdx.x, r = blockIdx.x, head = blockIdx.y >> 1, which = blockIdx.y & 1;
    const bool lead = blockIdx.y == 0 && tid == 0; // notes faults and the new length
    const int P = c.page_size, shift = c.page_shift;
    const int n0 = a.q_start[r], n1 = a.q_start[r + 1], kv = a.kv_len[r], asked = a.count[r];
    const int n = n1 > n0 ? static_cast<int>(min(static_cast<int64_t>(n1) - n0, static_cast<int64_t>(INT32_MAX))) : 0;
    if (n > MAX) {                                 // no tree: a prompt beside them keeps its tokens
        if (lead && a.new_len != nullptr) a.new_len[r] = max(kv, 0);
        return;
    }
    const int count = min(min(max(asked, 0), n), a.max_path);
    const int64_t base = static_cast<int64_t>(kv) - n;
    if (lead) {
        if (count != asked) atomicOr(a.status, CQ_DEV_TREE);
        if (a.new_len != nullptr) a.new_len[r] = static_cast<int32_t>(max(base + count, int64_t(0)));
    }
    if (count == 0) return;
    float* scales = which ? c.v_scale : c.k_scale;
    int8_t* values = which ? c.v : c.k;
    // (a length shorter than its new tokens: the first of them have no position)
    const int64_t b0 = (base < 0 ? 0 : base) >> shift;
    if (tid < MAX) {
        int from = -1;
        if (tid < count) {
            from = a.path[static_cast<int64_t>(r) * a.max_path + tid];
            if (from < 0 || from >= n) {
                if (blockIdx.y == 0) atomicOr(a.status, CQ_DEV_TREE);
                from = -1;
            } else if (from == tid) {
                from = -1;
            } else if (base + from < 0 || base + tid < 0) {
                if (blockIdx.y == 0) atomicOr(a.status, CQ_DEV_KV_PAGE);
                from = -1;
            }
        }
        src[tid] = static_cast<int16_t>(from);
    } else if (tid < MAX + MOST_PAGES) {
        const int k = tid - MAX;
        int p = -1;
        if (base + n > 0 && b0 + k <= (base + n - 1) >> shift && b0 + k < a.max_blocks) {
            p = a.table[r * a.max_blocks + b0 + k];
            if (p < 0 || p >= c.num_pages) p = -1;
        }
        page[k] = p;
        if (p >= 0) old[k] = now[k] = scales[p * c.scale_stride + head];
    }
    __syncthreads();
    auto block_of = [&](int i) { return static_cast<int>(((base + i) >> shift) - b0); };
    auto row_of = [&](int p, int i) {
        return values + static_cast<int64_t>(p) * c.page_stride + (static_cast<int64_t>(head) * P + ((base + i) & (P - 1))) * D;
    };
    if (tid < MAX && src[tid] >= 0 && (page[block_of(tid)] < 0 || page[block_of(src[tid])] < 0)) {
        if (blockIdx.y == 0) atomicOr(a.status, CQ_DEV_KV_PAGE);
        src[tid] = -1;
    }
    __syncthreads();
    // the rows as they were, and the pages' new scales
    constexpr int WPR = D / 16;                    // 16-byte pieces of a row
    for (int x = tid; x < count * WPR; x += MOVE_THREADS) {
        const int i = x / WPR, w = x % WPR;
        if (src[i] >= 0)
            *reinterpret_cast<uint4*>(&rows[i][4 * w]) = *reinterpret_cast<const uint4*>(row_of(page[block_of(src[i])], src[i]) + 16 * w);
    }
    if (tid < MOST_PAGES && page[tid] >= 0) {
        float s = old[tid];
        bool bad = s != s, any = false;
        for (int i = 0; i < count; ++i)
            if (src[i] >= 0 && block_of(i) == tid) {
                const float f = old[block_of(src[i])];
                any = true;
                bad |= f != f;
                s = fmaxf(s, f);
            }
        now[tid] = bad ? __uint_as_float(0x7fffffffu) : s;
        gets[tid] = any;
    }
    __syncthreads();
    auto scaled = [](uint32_t w, float ratio) {
        int z[4];
#pragma unroll
        for (int b = 0; b < 4; ++b) z[b] = round_away(__fmul_rn(static_cast<float>(static_cast<int8_t>(w >> (8 * b))), ratio));
        return pack4(z[0], z[1], z[2], z[3]);
    };
    auto ratio_of = [](float from, float to) { return to > 0.0f ? __fdiv_rn(from, to) : 0.0f; };
    // pages whose scale grows: their other rows (those that get one are written below)
    for (int k = 0; k < MOST_PAGES; ++k) {
        if (page[k] < 0 || !gets[k] || now[k] == old[k]) continue;
        const float ratio = ratio_of(old[k], now[k]);
        int8_t* q = values + static_cast<int64_t>(page[k]) * c.page_stride + static_cast<int64_t>(head) * P * D;
        for (int x = tid; x < P * (D / 4); x += MOVE_THREADS) {
            const int row = x / (D / 4), w = x % (D / 4);
            const int64_t i = ((b0 + k) << shift) + row - base;               // index among the new tokens
            if (i >= 0 && i < count && src[i] >= 0) continue;
            uint32_t* p = reinterpret_cast<uint32_t*>(q + row * D) + w;
            *p = scaled(*p, ratio);
        }
        if (tid == 0) scales[page[k] * c.scale_stride + head] = now[k];
    }
    for (int x = tid; x < count * (D / 4); x += MOVE_THREADS) {
        const int i = x / (D / 4), w = x % (D / 4);
        if (src[i] < 0) continue;
        const float from = old[block_of(src[i])], to = now[block_of(i)];
        const uint32_t v = rows[i][w];
        *(reinterpret_cast<uint32_t*>(row_of(page[block_of(i)], i)) + w) = from == to && to > 0.0f ? v : scaled(v, ratio_of(from, to));
    }
}

constexpr int FREE_THREADS = 512;

// Every CTA scans all requests' pages into shared memory (at most 16384 of them, read from L2), then
// copies its share of the list, each place's request found by bisection: one launch, nothing waits.
__global__ void __launch_bounds__(FREE_THREADS) kv_release_kernel(int R, int shift, const int32_t* table, int64_t max_blocks,
                                                                  int64_t num_pages, const int32_t* old_len,
                                                                  const int32_t* new_len, int32_t* freed, int capacity,
                                                                  int32_t* used) {
    pdl_trigger();
    pdl_wait();
    extern __shared__ int64_t before[];            // [R + 1] pages of the requests in front
    __shared__ int64_t warp_sum[FREE_THREADS / 32];
    __shared__ int flags;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, P1 = (1 << shift) - 1;
    if (tid == 0) flags = 0;
    __syncthreads();
    int64_t carry = 0;
    int bad = 0;
    auto blocks = [&](int len) { return min((static_cast<int64_t>(max(len, 0)) + P1) >> shift, max_blocks); };
    for (int r0 = 0; r0 < R; r0 += FREE_THREADS) {
        const int r = r0 + tid;
        int64_t x = 0;
        if (r < R) {
            const int o = old_len[r], w = new_len[r];
            if (o < 0 || w < 0) bad |= CQ_DEV_KV_LENGTH;
            if (((static_cast<int64_t>(max(o, 0)) + P1) >> shift) > max_blocks) bad |= CQ_DEV_KV_BLOCKS;
            x = max(blocks(o) - blocks(w), int64_t(0));
        }
        int64_t s = x;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t up = __shfl_up_sync(0xffffffffu, s, o);
            if (lane >= o) s += up;
        }
        if (lane == 31) warp_sum[warp] = s;
        __syncthreads();
        int64_t front = carry, all = 0;
        for (int w = 0; w < FREE_THREADS / 32; ++w) {
            if (w < warp) front += warp_sum[w];
            all += warp_sum[w];
        }
        if (r < R) before[r] = front + s - x;
        carry += all;
        __syncthreads();
    }
    if (tid == 0) before[R] = carry;
    if (carry > capacity) bad |= CQ_DEV_KV_PAGES;
    if (bad) atomicOr(&flags, bad);
    __syncthreads();
    const int64_t total = min(carry, static_cast<int64_t>(capacity));
    auto entry = [&](int64_t j) {
        int lo = 0, hi = R;                        // the last request with before <= j
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (before[mid] <= j) lo = mid; else hi = mid;
        }
        const int page = table[lo * max_blocks + blocks(new_len[lo]) + (j - before[lo])];
        return page >= 0 && page < num_pages ? page : -1;
    };
    const int64_t step = static_cast<int64_t>(gridDim.x) * FREE_THREADS;
    for (int64_t j = static_cast<int64_t>(blockIdx.x) * FREE_THREADS + tid; j < capacity; j += step) freed[j] = j < total ? entry(j) : -1;
    // the status is CTA 0's alone: it looks over every entry that is given back
    if (blockIdx.x == 0) {
        int fault = 0;
        for (int64_t j = tid; j < total; j += FREE_THREADS)
            if (entry(j) < 0) fault = CQ_DEV_KV_PAGE;
        if (fault) atomicOr(&flags, fault);
        __syncthreads();
        if (tid == 0) { used[0] = static_cast<int>(total); used[1] = flags; }
    }
}

}  // namespace

cudaError_t launch_tree_plan(const DeviceInfo& dev, int R, int T, const int32_t* kv_len, const int32_t* q_start,
                             const int32_t* parent, uint64_t* mask, int32_t* positions, cudaStream_t s) {
    const int ctas = std::max(1, std::min((R + GROUPS - 1) / GROUPS, dev.sm_count * 8));
    return launch_kernel(tree_plan_kernel, dim3(static_cast<unsigned>(ctas)), dim3(PLAN_THREADS), 0, s, R, T, kv_len, q_start,
                         parent, mask, positions, dev.status);
}

cudaError_t launch_kv_move(const DeviceInfo&, const KvView& c, const MoveArgs& a, cudaStream_t s) {
    const dim3 grid(static_cast<unsigned>(a.R), static_cast<unsigned>(2 * c.heads));
    return launch_kernel(c.dim == 64 ? kv_move_kernel<64> : kv_move_kernel<128>, grid, dim3(MOVE_THREADS), 0, s, c, a);
}

cudaError_t launch_kv_release(const DeviceInfo& dev, int R, int page_shift, const int32_t* table, int64_t max_blocks,
                              int64_t num_pages, const int32_t* old_len, const int32_t* new_len, int32_t* freed,
                              int capacity, int32_t* used, cudaStream_t s) {
    const int smem = (R + 1) * 8;
    cudaError_t e = raise_smem_limit(reinterpret_cast<const void*>(kv_release_kernel), smem);
    if (e != cudaSuccess) return e;
    const int64_t work = std::max<int64_t>(capacity, 1);
    const int64_t ctas = std::min<int64_t>(dev.sm_count, (work + FREE_THREADS - 1) / FREE_THREADS);
    return launch_kernel(kv_release_kernel, dim3(static_cast<unsigned>(ctas)), dim3(FREE_THREADS), static_cast<size_t>(smem), s, R,
                         page_shift, table, max_blocks, num_pages, old_len, new_len, freed, capacity, used);
}

}  // namespace cq
