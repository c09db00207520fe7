// Verification of drafted tokens (cq_tree_verify in include/cq_tree.h).
//
// A cluster of CTAs walks one request's tree from its first token: only the rows on the path of
// kept tokens are read, each CTA its slice of the vocabulary, which stays in shared memory for as
// long as the row is looked at. Probabilities are whole numbers,
//   w_v = 2^45 * 2^((z_v - max z) log2(e) / temperature), rounded,
// so that sums are exact whatever their order, W = sum w <= 2^63 for 2^18 values, and the
// rounding moves a value of the distribution function by 2^-45 sqrt(V) of the largest, not by
// fp32's 2^-24: a random number that falls near a border of a 10^5-value distribution still gives
// the token that 64 bits give. The exponential of fp32 units would not do, and fp64 runs at a
// sixty-fourth of fp32's rate; whole-number arithmetic costs about 45 instructions a value.
//
// After k rejected children the distribution is r_k = max(w - q A_k, 0) with A_k = R_0 + .. +
// R_(k-1), R_i the sum of r_i: max(max(a - b, 0) - c, 0) = max(a - b - c, 0) for b, c >= 0, so that
// one number stands for all rejections, and a rejection is one pass over the slice. Without draft
// probabilities a rejection only takes the child's own weight away.
//
// Every CTA decides by the same numbers: what a decision needs is spread over the cluster's shared
// memory (the request's tokens by CTA 0, maxima, sums and the children's logits by their owners),
// so that the CTAs meet at the same barriers whatever else writes to the inputs meanwhile.
#include <algorithm>
#include <climits>

#include "tc.cuh"
#include "tree.cuh"

namespace cq {
namespace {

constexpr int THREADS = 256;
constexpr int WARPS = THREADS / 32;
constexpr int MAX_CLUSTER = 16;
constexpr int MAX = CQ_TREE_MAX;
constexpr int PIECE = 128;                         // values that a warp takes at a time, four neighbours a lane
constexpr float CUT = -46.0f;                      // below 2^CUT of the largest: 0 (less than half a unit)

// 2^(i / 256) in units of 2^-45: the exponential's series in fp64, worked out by the compiler.
struct Pow2Table { unsigned long long v[256]; };
constexpr Pow2Table pow2_table() {
    Pow2Table t{};
    for (int i = 0; i < 256; ++i) {
        const double x = i * (0.69314718055994530942 / 256.0);
        double sum = 1.0, term = 1.0;
        for (int k = 1; k < 24; ++k) {
            term *= x / k;
            sum += term;
        }
        t.v[i] = static_cast<unsigned long long>(sum * 35184372088832.0 + 0.5);
    }
    return t;
}
__constant__ Pow2Table POW2 = pow2_table();

// What a request is decided by: CTA 0 reads it, the others copy it.
struct Request {
    int first, n, greedy;
    float c_hi, c_lo;                              // log2(e) / temperature in two parts
    unsigned long long u_sample;
    unsigned long long u[MAX];                     // in units of 2^-64
    int token[MAX];
    int parent[MAX];
};

__device__ __forceinline__ uint32_t mapa(uint32_t addr, uint32_t rank) {
    uint32_t r;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
    return r;
}
__device__ __forceinline__ void st_cluster(uint32_t addr, uint64_t v) {
    asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(addr), "l"(v) : "memory");
}
__device__ __forceinline__ uint32_t ld_cluster32(uint32_t addr) {
    uint32_t v;
    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
    return v;
}
// All threads of the cluster; what the first two warps wrote to others' shared memory is visible behind it.
// (A release by every warp is a fence by every warp.)
__device__ __forceinline__ void cluster_sync() {
    if (threadIdx.x < MAX) asm volatile("fence.acq_rel.cluster;" ::: "memory");
    asm volatile("barrier.cluster.arrive.relaxed;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
}
// Four values from global memory, those from n on 0.
__device__ __forceinline__ float4 load4(const float* p, int n, bool aligned) {
    if (aligned && n >= 4) return *reinterpret_cast<const float4*>(p);
    return make_float4(n > 0 ? p[0] : 0.0f, n > 1 ? p[1] : 0.0f, n > 2 ? p[2] : 0.0f, n > 3 ? p[3] : 0.0f);
}
__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}

// u in [0, 1) in units of 2^-64, exact (a float has 24 bits and is at least 2^-149).
__device__ __forceinline__ uint64_t unit64(float u) {
    if (!(u > 0.0f)) return 0;
    return __float2ull_rz(fminf(u, 0.99999994f) * 18446744073709551616.0f);
}
// A probability: 1 is 2^64 - 1.
__device__ __forceinline__ uint64_t prob64(float q) { return q > 0.0f ? __float2ull_rz(fminf(q, 1.0f) * 18446744073709551616.0f) : 0; }

__device__ __forceinline__ float max_nan(float a, float b) {      // NaN if either is
    float y;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
    return y;
}
__device__ __forceinline__ float exp2_fast(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// The whole-number part of an exponential: t0, t1, t2 are x's parts in units of 1, 2^-20 and 2^-40, each with 1.5 * 2^23 added.
// 2^x = 2^I * table[8 bits] * (1 + y + y^2 / 2 + y^3 / 6), y < 2^-8.5 in units of 2^-40; the next term is 2^-38.
__device__ __forceinline__ uint64_t weight_of(float t0, float t1, float t2, const unsigned long long* table) {
    const uint64_t above = static_cast<uint64_t>(__float_as_uint(t0) - 0x4b400000u) << 40 | __float_as_uint(t2);
    const uint64_t x = above + (static_cast<uint64_t>(__float_as_uint(t1)) << 20) - (0x4b400000ull << 20) - 0x4b400000ull;
    const int down = -(static_cast<int>(x >> 32) >> 8);                                 // 0 .. 47
    const uint32_t g = static_cast<uint32_t>(x);
    const uint64_t t = table[static_cast<uint32_t>(x >> 32) & 255u];
    const uint32_t y = __umulhi(g, 2977044472u);                                        // ln 2 in units of 2^-32
    const uint32_t y2 = __umulhi(y, y) >> 9;
    const uint32_t y3 = __umulhi(y2 * 683u, y) >> 19;                                   // 683 / 2048: a third
    const uint64_t w = t + ((static_cast<uint64_t>(static_cast<uint32_t>(t >> 15)) * (y + y2 + y3)) >> 25);
    return (w + ((uint64_t(1) << down) >> 1)) >> down;
}

constexpr float CUTTER = 12582912.0f;              // 0x4b400000: adding it leaves a whole number

// w of two logits beside the row's largest, m (finite); c = log2(e) / temperature. The exponent
// x = (z - m) c is held to 2^-40: the difference and its rounding error, times c in two parts; it is cut into whole
// numbers by additions (conversions run at an eighth of their rate). The fp32 steps go two logits at a time (115 us one
// at a time, 112 so, at 64 chains of 5 drafts over 128256 values; 109 since the CTAs meet once a row).
struct Two { uint64_t a, b; };
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
    uint64_t y;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(y) : "l"(a), "l"(b));
    return y;
}
__device__ __forceinline__ Two weights(float z0, float z1, float m, float c_hi, float c_lo, const unsigned long long* table) {
    auto both = [](float x) { return tc::pk(x, x); };
    const uint64_t z = tc::pk(z0, z1), less = both(-1.0f), nm = both(-m), ch = both(c_hi), cut = both(CUTTER);
    const uint64_t d = tc::add2(z, nm), np = mul2(d, both(-c_hi));                      // -p
    const uint64_t bb = tc::fma2(z, less, d);
    const uint64_t err = tc::add2(tc::fma2(tc::fma2(bb, less, d), less, z), tc::fma2(bb, less, nm));
    const uint64_t e = tc::fma2(err, ch, tc::fma2(d, both(c_lo), tc::fma2(d, ch, np)));
    const uint64_t t0 = tc::fma2(np, less, cut), nf = tc::add2(np, tc::add2(t0, both(-CUTTER)));      // -f
    const uint64_t t1 = tc::fma2(nf, both(-1048576.0f), cut);
    const uint64_t nf2 = tc::fma2(tc::add2(t1, both(-CUTTER)), both(9.5367431640625e-07f), nf);
    const uint64_t t2 = tc::fma2(tc::fma2(nf2, less, e), both(1099511627776.0f), cut);
    float p0, p1, a0, a1, b0, b1, c0, c1;
    tc::upk(np, p0, p1);
    tc::upk(t0, a0, a1);
    tc::upk(t1, b0, b1);
    tc::upk(t2, c0, c1);
    return Two{p0 < -CUT ? weight_of(a0, b0, c0, table) : 0, p1 < -CUT ? weight_of(a1, b1, c1, table) : 0};
}

// One logit's, by the same steps: what is taken from a sum is what went into it.
__device__ __forceinline__ uint64_t weight(float z, float m, float c_hi, float c_lo, const unsigned long long* table) {
    return weights(z, z, m, c_hi, c_lo, table).a;
}

// max(w - q A, 0), A = a_hi 2^64 + a_lo; q a probability: 24 bits, q = f 2^-s.
__device__ __forceinline__ uint64_t without(uint64_t w, float q, uint64_t a_lo, uint32_t a_hi) {
    const uint32_t b = __float_as_uint(fminf(fmaxf(q, 0.0f), 1.0f));                    // (NaN: 0)
    const uint32_t f = (b & 0x7fffffu) | 0x800000u;
    const int s = 150 - static_cast<int>(b >> 23);                                      // 23 (q = 1) .. 150 (0 and subnormal: nothing is left)
    // f A: 24 bits by 70
    const uint64_t lo = static_cast<uint64_t>(f) * static_cast<uint32_t>(a_lo);
    const uint64_t hi = static_cast<uint64_t>(f) * static_cast<uint32_t>(a_lo >> 32) + (lo >> 32);      // < 2^57
    uint64_t t;
    if (a_hi == 0) {
        t = s >= 96 ? 0 : s >= 32 ? hi >> (s - 32) : hi << (32 - s) | static_cast<uint32_t>(lo) >> s;
    } else {
        const uint64_t top = static_cast<uint64_t>(f) * a_hi;                           // < 2^31, in units of 2^64
        if (s < 64 && top >> s != 0) return 0;
        t = s >= 96 ? 0 : s >= 32 ? hi >> (s - 32) : hi << (32 - s) | static_cast<uint32_t>(lo) >> s;
        const uint64_t more = s >= 128 ? 0 : s >= 64 ? top >> (s - 64) : top << (64 - s);
        if (t + more < t) return 0;
        t += more;
    }
    return w > t ? w - t : 0;
}

struct Shared {
    unsigned long long table[256];
    unsigned long long xchg[2][MAX_CLUSTER];       // what the CTAs spread, alternately
    unsigned long long tot[MAX_CLUSTER];           // the CTAs' sums of r
    unsigned long long parts[2][WARPS];            // the warps' sums over their own stretch of the slice, alternately
    unsigned long long children[2][MAX];           // logit and draft probability of a node's children, alternately
    unsigned long long weight[MAX];                // their w
    float2 top[WARPS];                             // largest logits and sums of exponentials
    Request rq;
    int gone[MAX], gone_at[MAX];                   // tokens rejected at this node, and whose (no draft probabilities)
};

template <bool DRAFT>
__global__ void __launch_bounds__(THREADS, 3) tree_verify_kernel(const VerifyArgs a, const int cluster, const int slice, const int stretch, const bool few) {
    pdl_trigger();
    extern __shared__ __align__(16) float row[];   // [WARPS * stretch]: the node's logits, -infinity past the slice
    __shared__ Shared sh;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int r = blockIdx.x / cluster;
    const uint32_t rank = cluster_rank();
    if (tid < 256) sh.table[tid] = POW2.v[tid];
    pdl_wait();
    const int lo = static_cast<int>(min(static_cast<int64_t>(rank) * slice, static_cast<int64_t>(a.V)));
    const int len = min(slice, a.V - lo);          // this CTA's values; 0 for none
    // a warp's values: whole pieces, four neighbours a lane; a thread reads what it has brought itself
    const int w0 = warp * stretch + 4 * lane, w1 = min((warp + 1) * stretch, (len + 3) & ~3);
    if (rank == 0) {
        const int first = min(max(a.q_start[r], 0), a.T);
        const int n = max(min(a.q_start[r + 1], a.T) - first, 0);
        if (tid == 0) {
            const float t = a.temperature[r];
            const bool greedy = !(t >= 5.421010862427522e-20f);                          // 2^-64
            const double c = 1.4426950408889634 / (greedy ? 1.0 : static_cast<double>(fminf(t, 1.8446744073709552e19f)));
            sh.rq.first = first;
            sh.rq.n = n;
            sh.rq.greedy = greedy;
            sh.rq.c_hi = static_cast<float>(c);
            sh.rq.c_lo = static_cast<float>(c - static_cast<double>(sh.rq.c_hi));
            sh.rq.u_sample = unit64(a.u_sample[r]);
        }
        if (n <= MAX && tid < n) {
            int p = a.parent[first + tid];
            if (p < -1 || p >= tid) {
                atomicOr(a.status, CQ_DEV_TREE);
                p = -1;
            }
            sh.rq.parent[tid] = p;
            sh.rq.token[tid] = a.tokens[first + tid];
            sh.rq.u[tid] = unit64(a.u_accept[first + tid]);
        }
    }
    cluster_sync();
    if (rank != 0) {
        const uint32_t from = mapa(smem_u32(&sh.rq), 0);
        static_assert(sizeof(Request) % 4 == 0, "copied as words");
        for (int i = tid; i < static_cast<int>(sizeof(Request) / 4); i += THREADS)
            reinterpret_cast<uint32_t*>(&sh.rq)[i] = ld_cluster32(from + 4 * i);
        __syncthreads();
    }
    const int n = sh.rq.n, first = sh.rq.first;
    const bool lead = rank == 0 && tid == 0;
    int32_t* path = a.path + static_cast<int64_t>(r) * a.max_path;
    int kept = 0, next = -1;

    // Spreads a CTA's number and gives all of them, each CTA's in its place. (A buffer is written again two
    // turns on: by then every CTA has passed the barrier between, and read it.)
    int turn = 0;
    auto spread = [&](uint64_t mine) {
        if (tid < cluster) st_cluster(mapa(smem_u32(&sh.xchg[turn][rank]), tid), mine);
        cluster_sync();
        turn ^= 1;
        return sh.xchg[turn ^ 1];
    };
    // The warps' sums to `part` and the CTA's to all threads. (A buffer is written again two barriers on.)
    int side = 0;
    unsigned long long* part = sh.parts[0];
    auto sum_of = [&](uint64_t s) {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
        part = sh.parts[side];
        side ^= 1;
        if (lane == 0) part[warp] = s;
        __syncthreads();
        uint64_t all = 0;
#pragma unroll
        for (int w = 0; w < WARPS; ++w) all += part[w];
        return all;
    };
    // A row's slice on its way into L2.
    auto ahead = [&](const float* p) {
        const uintptr_t p0 = (reinterpret_cast<uintptr_t>(p) + 15) & ~uintptr_t(15), p1 = reinterpret_cast<uintptr_t>(p + len) & ~uintptr_t(15);
        if (tid == 0 && p1 > p0) bulk_prefetch_l2(reinterpret_cast<const void*>(p0), static_cast<uint32_t>(p1 - p0));
    };
    // The CTAs' sums of r spread and held in sh.tot; the sum of all.
    auto totals = [&](uint64_t mine) {
        const unsigned long long* got = spread(mine);
        uint64_t all = 0;
        for (int c = 0; c < cluster; ++c) all += got[c];
        if (all != 0) {
            if (tid < cluster) sh.tot[tid] = got[tid];
            __syncthreads();
        }
        return all;
    };

    if (n > 0 && n <= MAX) {
        int node = 0;
        kept = 1;
        if (lead) path[0] = 0;
        const float c_hi = sh.rq.c_hi, c_lo = sh.rq.c_lo;
        const bool greedy = sh.rq.greedy != 0;
        for (;;) {
            // ---- the node's row: into shared memory
            const float* z = a.logits + static_cast<int64_t>(first + node) * a.logits_stride + lo;
            const float* dr = DRAFT ? a.draft + static_cast<int64_t>(first + node) * a.draft_stride + lo : nullptr;
            const bool al = (reinterpret_cast<uintptr_t>(z) & 15) == 0, al_d = (reinterpret_cast<uintptr_t>(dr) & 15) == 0;
            __syncthreads();                       // nobody looks at the last row any more
            for (int i = w0; i < (warp + 1) * stretch; i += PIECE) {
                if (al && i + 4 <= len) {
                    cp_async16(row + i, z + i);
                } else {
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        if (i + k < len) cp_async4(row + i + k, z + i + k, 4);
                        else row[i + k] = -INFINITY;
                    }
                }
            }
            cp_async_commit();
            // ---- its children, one bit each
            uint64_t children = 0;
            if (kept < a.max_path) {
                const uint32_t c0 = __ballot_sync(0xffffffffu, lane < n && sh.rq.parent[lane] == node && lane > 0);
                const uint32_t c1 = __ballot_sync(0xffffffffu, lane + 32 < n && sh.rq.parent[lane + 32] == node);
                children = static_cast<uint64_t>(c1) << 32 | c0;
            }
            // the thread's child, where this CTA has its token, and its draft probability
            const int own = tid < MAX && (children >> tid & 1) != 0 ? sh.rq.token[tid] - lo : -1;
            const bool owns = own >= 0 && own < len;
            const float own_q = DRAFT && owns ? dr[own] : 0.0f;
            if (few && children != 0)               // the row that is likeliest next
                ahead(a.logits + static_cast<int64_t>(first + __ffsll(static_cast<long long>(children)) - 1) * a.logits_stride + lo);
            // ---- its largest logit, NaN if any is, and where a child is to be tested the sum of its exponentials in fp32: each
            // warp's beside its own largest, so that the CTAs meet once for both
            cp_async_wait_all();
            float m = -INFINITY, sum = 0.0f;
#pragma unroll 4
            for (int i = w0; i < w1; i += PIECE) {
                const float4 v = *reinterpret_cast<const float4*>(row + i);
                m = max_nan(max_nan(m, max_nan(v.x, v.y)), max_nan(v.z, v.w));
            }
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
            if (children != 0 && !greedy && m > -INFINITY) {
#pragma unroll 4
                for (int i = w0; i < w1; i += PIECE) {
                    const float4 v = *reinterpret_cast<const float4*>(row + i);
                    sum += (exp2_fast((v.x - m) * c_hi) + exp2_fast((v.y - m) * c_hi)) + (exp2_fast((v.z - m) * c_hi) + exp2_fast((v.w - m) * c_hi));
                }
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
            }
            // (largest, sum) of some stretches as those of all of them; a stretch without a finite value has a sum of 0
            auto joined = [&](const float2* part_of, int count) {
                float top = -INFINITY, all = 0.0f;
                for (int k = 0; k < count; ++k) top = max_nan(top, part_of[k].x);
                for (int k = 0; k < count; ++k)
                    if (part_of[k].y > 0.0f) all = fmaf(part_of[k].y, exp2_fast((part_of[k].x - top) * c_hi), all);
                return make_float2(top, all);
            };
            if (lane == 0) sh.top[warp] = make_float2(m, sum);
            __syncthreads();
            const float2 here = joined(sh.top, WARPS);
            // the children's logits and draft probabilities, from the CTA that has them (to a place of its own: another CTA may
            // still be at the node before)
            unsigned long long* const child = sh.children[kept & 1];
            if (owns) {
                const uint64_t v = static_cast<uint64_t>(__float_as_uint(own_q)) << 32 | __float_as_uint(row[own]);
                for (int c = 0; c < cluster; ++c) st_cluster(mapa(smem_u32(&child[tid]), c), v);
            }
            const unsigned long long* got = spread(static_cast<uint64_t>(__float_as_uint(here.y)) << 32 | __float_as_uint(here.x));
            const float2 row_of = joined(reinterpret_cast<const float2*>(got), cluster);
            m = row_of.x;
            if (!(fabsf(m) < INFINITY)) {
                if (lead) atomicOr(a.status, CQ_DEV_LOGITS);
                break;
            }
            int taken = -1;
            if (greedy) {
                // the largest logit's smallest index
                int at = INT_MAX;
                for (int i = w0; i < w1 && at == INT_MAX; i += PIECE)
#pragma unroll
                    for (int k = 3; k >= 0; --k)
                        if (row[i + k] == m) at = lo + i + k;
                at = __reduce_min_sync(0xffffffffu, at);
                part = sh.parts[side];
                side ^= 1;
                if (lane == 0) part[warp] = at;
                __syncthreads();
                for (int w = 0; w < WARPS; ++w) at = min(at, static_cast<int>(part[w]));
                got = spread(at);
                for (int c = 0; c < cluster; ++c) at = min(at, static_cast<int>(got[c]));
                for (uint64_t left = children; left != 0 && taken < 0; left &= left - 1) {
                    const int j = __ffsll(static_cast<long long>(left)) - 1;
                    if (sh.rq.token[j] == at) taken = j;
                }
                if (taken < 0) next = at;
            } else {
                // The sum of w: exactly, with the warps' and the CTAs' parts; the path's rows in front of the last need it only
                // to tell on which side of it a random number falls.
                auto exact = [&]() {
                    uint64_t s = 0;
                    for (int i = w0; i < w1; i += PIECE) {
                        const float4 v = *reinterpret_cast<const float4*>(row + i);
                        const Two x = weights(v.x, v.y, m, c_hi, c_lo, sh.table), y = weights(v.z, v.w, m, c_hi, c_lo, sh.table);
                        s += (x.a + x.b) + (y.a + y.b);
                    }
                    return totals(sum_of(s));
                };
                uint64_t R = 0, below = 0, above = 0;       // the sum of r (0: not known yet) and bounds on it
                if (children != 0) {
                    // Terms good to 2^-17 (arguments up to 46, three roundings), brought to the row's largest in two steps
                    // more, in sums of some tens: within 2^-15.
                    above = __float2ull_rn(row_of.y * 35184372088832.0f);
                    below = above - (above >> 15);
                    above += above >> 15;
                    if (tid < MAX && (children >> tid & 1) != 0)
                        sh.weight[tid] = weight(__uint_as_float(static_cast<uint32_t>(child[tid])), m, c_hi, c_lo, sh.table);
                    __syncthreads();
                }
                uint64_t a_lo = 0;
                uint32_t a_hi = 0;
                int gone = 0;
                for (uint64_t left = children; left != 0 && taken < 0; left &= left - 1) {
                    const int j = __ffsll(static_cast<long long>(left)) - 1, x = sh.rq.token[j];
                    if (x < 0 || x >= a.V) continue;
                    const uint64_t u = sh.rq.u[j];
                    uint64_t w = sh.weight[j];
                    if constexpr (DRAFT) {
                        const float q1 = __uint_as_float(static_cast<uint32_t>(child[j] >> 32));
                        const uint64_t q = prob64(q1);
                        if (R == 0) {
                            if (__umul64hi(u, __umul64hi(q, above)) < w) {
                                taken = j;
                                break;
                            }
                            ahead(dr);
                            R = exact();
                        }
                        w = without(w, q1, a_lo, a_hi);
                        if (__umul64hi(u, __umul64hi(q, R)) < w) {
                            taken = j;
                            break;
                        }
                        // one pass for the next distribution's sums
                        const uint64_t n_lo = a_lo + R;
                        const uint32_t n_hi = a_hi + (n_lo < a_lo);
                        uint64_t rs = 0;
                        auto next_q = [&](int i) { return load4(dr + i, i < w1 ? len - i : 0, al_d); };
                        float4 d0 = next_q(w0), d1 = next_q(w0 + PIECE);
                        for (int i = w0; i < w1; i += PIECE) {
                            const float4 v = *reinterpret_cast<const float4*>(row + i), d = d0;
                            d0 = d1;
                            d1 = next_q(i + 2 * PIECE);
                            const Two x = weights(v.x, v.y, m, c_hi, c_lo, sh.table), y = weights(v.z, v.w, m, c_hi, c_lo, sh.table);
                            rs += (without(x.a, d.x, n_lo, n_hi) + without(x.b, d.y, n_lo, n_hi)) +
                                  (without(y.a, d.z, n_lo, n_hi) + without(y.b, d.w, n_lo, n_hi));
                        }
                        unsigned long long* before = part;                              // kept where nothing is left
                        const uint64_t sum = totals(sum_of(rs));
                        if (sum != 0) {
                            R = sum;
                            a_lo = n_lo;
                            a_hi = n_hi;
                        } else {
                            part = before;
                            side ^= 1;                                                  // the next sums do not go there
                        }
                    } else {
                        for (int k = 0; k < gone; ++k)
                            if (sh.gone[k] == x) w = 0;
                        if (__umul64hi(u, above) < w) {
                            taken = j;
                            break;
                        }
                        if (R == 0 && __umul64hi(u, below) < w) {                      // between the bounds: exactly, then
                            R = exact();
                            for (int k = 0; k < gone; ++k) R -= sh.weight[sh.gone_at[k]];
                            above = below = R;
                            if (__umul64hi(u, R) < w) {
                                taken = j;
                                break;
                            }
                        }
                        // (its weight may be all that is left only where the bounds are exact: else something of r is beside it)
                        if (w != 0 && w != above) {
                            above -= w;
                            below = below > w ? below - w : 0;
                            if (R != 0) R -= w;
                            __syncthreads();
                            if (tid == 0) {
                                sh.gone[gone] = x;
                                sh.gone_at[gone] = j;
                            }
                            ++gone;
                            __syncthreads();
                        }
                    }
                }
                if (taken < 0) {
                    // ---- the next token: the CTA, the warp's stretch and the place in it where the sums pass u R
                    if (R == 0) {
                        R = exact();
                        for (int k = 0; k < gone; ++k) R -= sh.weight[sh.gone_at[k]];
                    }
                    if (!DRAFT && gone > 0) {
                        __syncthreads();
                        if (tid == 0)
                            for (int k = 0; k < gone; ++k) {
                                const int x = sh.gone[k], owner = x / slice;
                                sh.tot[owner] -= sh.weight[sh.gone_at[k]];
                                if (owner == static_cast<int>(rank)) part[(x - lo) / stretch] -= sh.weight[sh.gone_at[k]];
                            }
                        __syncthreads();
                    }
                    uint64_t t = __umul64hi(sh.rq.u_sample, R);
                    int owner = 0;
                    while (owner < cluster - 1 && t >= sh.tot[owner]) t -= sh.tot[owner++];
                    if (owner == static_cast<int>(rank)) {
                        int w = 0;
                        while (w < WARPS - 1 && t >= part[w]) t -= part[w++];
                        const int s0 = min(w * stretch, len), s1 = min(s0 + stretch, len);
                        const int per = (stretch + THREADS - 1) / THREADS, i0 = s0 + tid * per, i1 = min(i0 + per, s1);
                        auto value = [&](int i) {
                            uint64_t v = weight(row[i], m, c_hi, c_lo, sh.table);
                            if constexpr (DRAFT) {
                                if ((a_lo | a_hi) != 0) v = without(v, dr[i], a_lo, a_hi);
                            } else {
                                for (int k = 0; k < gone; ++k)
                                    if (sh.gone[k] == lo + i) v = 0;
                            }
                            return v;
                        };
                        uint64_t mine = 0;
                        for (int i = i0; i < i1; ++i) mine += value(i);
                        uint64_t upto = mine;
#pragma unroll
                        for (int o = 1; o < 32; o <<= 1) {
                            const uint64_t up = __shfl_up_sync(0xffffffffu, upto, o);
                            if (lane >= o) upto += up;
                        }
                        part = sh.parts[side];
                        side ^= 1;
                        if (lane == 31) part[warp] = upto;
                        __syncthreads();
                        for (int k = 0; k < warp; ++k) upto += part[k];
                        if (t < upto && t >= upto - mine) {                          // one thread
                            uint64_t c = upto - mine;
                            int i = i0;
                            for (; i < i1 - 1; ++i) {
                                c += value(i);
                                if (t < c) break;
                            }
                            a.next[r] = lo + i;
                        }
                    }
                    next = -2;                     // written by its owner
                }
            }
            if (taken < 0) break;
            node = taken;
            if (lead) path[kept] = node;
            ++kept;
        }
    }
    if (rank == 0) {
        for (int i = kept + tid; i < a.max_path; i += THREADS) path[i] = -1;
        if (tid == 0) {
            a.count[r] = kept;
            if (next != -2) a.next[r] = next;
        }
    }
    cluster_sync();                                // nobody leaves while another may look at its shared memory
}

template <bool DRAFT>
cudaError_t launch_t(const DeviceInfo& dev, const VerifyArgs& a, cudaStream_t s) {
    // CTAs of a request: a slice of 4096 values is sixteen a thread. Eight, whose slices of 2^18 values fit in shared
    // memory, or sixteen where requests are few: 1 / 16 / 64 chains of 5 drafts over 128256 values take 40 / 56 / 117 us
    // with eight, 29 / 46 / 134 with sixteen (27 / 43 / 109 now, by this rule).
    const int most = static_cast<int64_t>(a.R) * MAX_CLUSTER <= 2 * dev.sm_count ? MAX_CLUSTER : MAX_CLUSTER / 2;
    int cluster = 1;
    while (cluster < most && a.V > 4096 * cluster) cluster *= 2;
    const int slice = ((a.V + cluster - 1) / cluster + 3) / 4 * 4, stretch = ((slice + WARPS - 1) / WARPS + PIECE - 1) / PIECE * PIECE;
    const int smem = WARPS * stretch * 4;
    // Where the CTAs are few, a row that may not be needed costs nobody's bandwidth.
    const bool few = static_cast<int64_t>(a.R) * cluster <= 2 * dev.sm_count;
    if (smem > dev.smem_optin - static_cast<int>(sizeof(Shared)) - 1024) return cudaErrorInvalidConfiguration;
    cudaError_t e = raise_smem_limit(reinterpret_cast<const void*>(tree_verify_kernel<DRAFT>), smem);
    if (e != cudaSuccess) return e;
    if (cluster > 8) {                             // more than every GPU takes: asked for
        e = cudaFuncSetAttribute(tree_verify_kernel<DRAFT>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
        if (e != cudaSuccess) return e;
    }
    return launch_kernel_cluster(tree_verify_kernel<DRAFT>, dim3(static_cast<unsigned>(a.R * cluster)), dim3(THREADS),
                                 static_cast<size_t>(smem), s, dim3(cluster), a, cluster, slice, stretch, few);
}

}  // namespace

cudaError_t launch_tree_verify(const DeviceInfo& dev, const VerifyArgs& a, cudaStream_t s) {
    return a.draft != nullptr ? launch_t<true>(dev, a, s) : launch_t<false>(dev, a, s);
}

}  // namespace cq
