// Shared pieces of the attention kernels: lengths and visible ranges, query
// scaling, streaming loads, output rows.
#pragma once
#include <cstdint>
#include <type_traits>

#include "cq_device.cuh"
#include "cq_internal.h"
#include "cq_tree.h"
#include "kv.cuh"

namespace cq {

// CTAs that share the partial results of a call: the workspace has two slots
// and a counter for each.
constexpr int ATTN_MAX_CTAS = 640;

// CTAs of the tiles kernel when it splits its items over the keys (one an SM at
// most), the reference offset of its results, and what a shared item's first
// CTA writes down for the join.
constexpr int ATTN_TILE_CTAS = 256;
constexpr float TILES_OFF = 7.0f;
struct TileShare {
    int parts;           // CTAs that share the item; below 2: none
    int rows, row0;      // its rows, and the first among its request's rows of the kv head
    int first, h;        // the request's first token, the kv head
    int any;             // whether the call splits items at all
    int pad[2];
};

struct RowsPlan {
    int* count;          // [ATTN_MAX_CTAS], zero between calls
    float* part;         // [ATTN_MAX_CTAS][2][16][head_dim + 4]
    TileShare* share;    // [ATTN_TILE_CTAS]
    float* tile_part;    // [ATTN_TILE_CTAS][256][head_dim + 4]
    int sms;             // CTAs that the tiles kernel may split its items into
    int after_tiles;     // the rows kernel follows the tiles kernel and runs beside it
    int one_tile;        // 16-bit calls under masks: the tiles kernel's build with one row tile a CTA
    int tile_rows;       // a request with at least so many rows of a kv head is attn_tiles.cu's; INT_MAX: none is
};

// Requests that each kernel takes: n new tokens, G query heads a kv head.
__device__ __forceinline__ bool tiles_take(const RowsPlan& pl, int n, int G) { return static_cast<int64_t>(n) * G >= pl.tile_rows; }
__device__ __forceinline__ bool rows_take(const RowsPlan& pl, int n, int G) { return n > 0 && !tiles_take(pl, n, G); }

// a / b for 0 <= a, 0 < b, by a 32-bit division where both allow it.
__device__ __forceinline__ int64_t quot(int64_t a, int64_t b) {
    if (((a | b) >> 32) == 0) return static_cast<uint32_t>(a) / static_cast<uint32_t>(b);
    return a / b;
}

// First token, new tokens (clipped to T) and length (clipped to the table) of request r.
__device__ __forceinline__ void request_of(const KvView& c, const AttnArgs& a, int r, int& first, int& n, int& kv) {
    const int s = a.q_start[r], e = a.q_start[r + 1];
    first = min(max(s, 0), a.T);
    n = max(min(e, a.T) - first, 0);
    kv = static_cast<int>(min(static_cast<int64_t>(max(a.kv_len[r], 0)), a.max_blocks << c.page_shift));
}

// Keys [from, stop) that the request's token t of n sees; 0, 0 if none.
__device__ __forceinline__ void row_range(const AttnArgs& a, int n, int kv, int t, int& from, int& stop) {
    const int64_t pos = static_cast<int64_t>(kv) - n + t;
    int64_t s = a.causal ? min(static_cast<int64_t>(kv), pos + 1) : kv;
    int64_t f = a.window > 0 ? max(int64_t(0), pos - a.window + 1) : 0;
    if (s <= f) s = f = 0;
    from = static_cast<int>(f);
    stop = static_cast<int>(s);
}

// Trees (cq_attn_tree): a request of at most CQ_TREE_MAX new tokens sees the keys in front of them, and of
// them those whose bits are set in the row's mask; a longer one is causal.
__device__ __forceinline__ bool is_tree(int n) { return n <= CQ_TREE_MAX; }

// What token t sees of its own request's new tokens, by their index; 0 where the request is causal.
__device__ __forceinline__ uint64_t tree_mask(const AttnArgs& a, int first, int n, int t) {
    if (!is_tree(n)) return 0;
    const uint64_t m = a.tree[first + t];
    return n == 64 ? m : m & ((uint64_t(1) << n) - 1);
}

// Of the request's tokens t0..t1 (t0 <= t1): the first key that one of them may see, the keys [all_from, all_stop) that all see, the
// end of what one of them may see. A tree's masks are not looked at: its new tokens count as seen by some.
template <bool TREE>
__device__ __forceinline__ void tile_range(const AttnArgs& a, int n, int kv, int t0, int t1, int& from, int& all_from,
                                           int& all_stop, int& stop) {
    if (TREE && is_tree(n)) {
        from = all_from = 0;
        all_stop = max(kv - n, 0);
        stop = kv;
        return;
    }
    row_range(a, n, kv, t0, from, all_stop);
    row_range(a, n, kv, t1, all_from, stop);
}

// Token t's keys [from, stop), those of a tree's mask apart.
template <bool TREE>
__device__ __forceinline__ void token_range(const AttnArgs& a, int n, int kv, int t, int& from, int& stop) {
    if (TREE && is_tree(n)) {
        from = 0;
        stop = max(kv - n, 0);
        return;
    }
    row_range(a, n, kv, t, from, stop);
}

// From the bits of a row's largest |value|: the power of two that brings it to
// [2^8, 2^9) and its inverse; NaN for a row that is not finite.
__device__ __forceinline__ void row_scale(uint32_t top, float& mul, float& back) {
    const int e = static_cast<int>(top >> 23);              // biased exponent, 0 for zero and subnormal
    if (e == 255) { mul = back = __uint_as_float(0x7fffffffu); return; }
    const int up = min(135 - max(e, 1), 126);               // 2^up; stays a normal number
    mul = __uint_as_float(static_cast<uint32_t>(127 + up) << 23);
    back = __uint_as_float(static_cast<uint32_t>(127 - up) << 23);
}

__device__ __forceinline__ float exp2_approx(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// A block of zeros (value scale 0) adds to the sum alone. Its P must not set the reference that
// the other blocks' are held to, whatever their scale, so it takes part as if its scale were
// 2^ZERO_LOG: at 1, a row whose other blocks have scales of 1e-6 lost its bits in binary16 (85
// times its error bound at 1e-8, and 0 at 1e-10). Its P stays a normal number beside scales of up
// to 2^45, with 24 bits below its largest.
constexpr float ZERO_LOG = -64.0f;

// The sums of P / s_v are held without a factor 2^SUM_LOG: for scales down to append's smallest,
// 2^-126, P up to 2^15 and 2^20 keys they stay below 2^128 (with nothing taken out they were
// infinite from 2^-116 down), and up to scales of 2^96 a row's sum is a normal number: its
// largest P is at least 2^7.
constexpr float SUM_LOG = 34.0f, SUM_DOWN = 1.0f / 17179869184.0f;        // 2^-SUM_LOG

__device__ __forceinline__ float log2_approx(float x) {
    float y;
    asm("lg2.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float rcp_approx(float x) {
    float y;
    asm("rcp.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// What a value scale s gives its block: the offset of its scores, log2 s, and the factor of its
// P in the sums; for the 16-bit types approximations to 2^-22, as the exponentials themselves are,
// the same in both kernels. Finite whatever s is: the factor meets sums of 0 where a row sees nothing.
template <bool EXACT>
__device__ __forceinline__ void value_factors(float s, float& offset, float& weight) {
    if (s == 0.0f) {
        offset = ZERO_LOG;
        weight = exp2f(-ZERO_LOG - SUM_LOG);
        return;
    }
    offset = EXACT ? log2f(s) : log2_approx(s);
    weight = fminf(EXACT ? __frcp_rn(s) : rcp_approx(s), 3.402823466e38f) * SUM_DOWN;
}

// What a row's result is multiplied by, one factor after the other: 2^-SUM_LOG / l in two steps
// that neither pass fp32's range nor fall below it where the result does not. 0 for a row that saw nothing.
__device__ __forceinline__ void row_factors(float l, float& f, float& down) {
    f = l == 0.0f ? 0.0f : __frcp_rn(l);
    down = SUM_DOWN;
    if (f > 1.0f) {
        f *= SUM_DOWN;
        down = 1.0f;
    }
}

__device__ __forceinline__ float max3(float a, float b, float c) {
    float y;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(y) : "f"(a), "f"(b), "f"(c));
    return y;
}

// Two binary16 integers of at most 8 bits as bfloat16 (exact).
__device__ __forceinline__ uint32_t half_to_bf16(uint32_t h) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
    return __byte_perm(__float_as_uint(f.x), __float_as_uint(f.y), 0x7632);
}

// Four signed bytes as bfloat16 integers, in byte order: each flipped to 128 + b
// under the exponent of 2^23, the offset taken away, the upper halves kept.
__device__ __forceinline__ void s8x4_bf16(uint32_t w, uint32_t& o0, uint32_t& o1) {
    const uint32_t u = w ^ 0x80808080u;
    float f[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = __uint_as_float(__byte_perm(u, 0x4b000000u, 0x7440 + i)) - 8388736.0f;
    o0 = __byte_perm(__float_as_uint(f[0]), __float_as_uint(f[1]), 0x7632);
    o1 = __byte_perm(__float_as_uint(f[2]), __float_as_uint(f[3]), 0x7632);
}

// Two consecutive values as they were loaded: converted only when they are used, so
// that several loads can be in flight.
template <typename T> struct Raw2 {
    uint32_t u[sizeof(T) / 2];
    __device__ __forceinline__ void load(const T* p) {
        if constexpr (sizeof(T) == 4) {
            const uint2 v = *reinterpret_cast<const uint2*>(p);
            u[0] = v.x;
            u[1] = v.y;
        } else {
            u[0] = *reinterpret_cast<const uint32_t*>(p);
        }
    }
    __device__ __forceinline__ float2 value() const {
        if constexpr (sizeof(T) == 4) return make_float2(__uint_as_float(u[0]), __uint_as_float(u[1]));
        else if constexpr (std::is_same<T, __half>::value) return __half22float2(*reinterpret_cast<const __half2*>(&u[0]));
        else return make_float2(__uint_as_float(u[0] << 16), __uint_as_float(u[0] & 0xffff0000u));
    }
};

// Eight of them, 16-byte aligned.
template <typename T> struct Raw8 {
    uint4 u[sizeof(T) / 2];
    __device__ __forceinline__ void load(const T* p) {
#pragma unroll
        for (int i = 0; i < static_cast<int>(sizeof(T) / 2); ++i) u[i] = reinterpret_cast<const uint4*>(p)[i];
    }
    __device__ __forceinline__ void values(float (&x)[8]) const {
        const uint32_t w[4] = {u[0].x, u[0].y, u[0].z, u[0].w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (sizeof(T) == 4) {
                const uint32_t z[4] = {u[1].x, u[1].y, u[1].z, u[1].w};
                x[i] = __uint_as_float(w[i]);
                x[4 + i] = __uint_as_float(z[i]);
            } else if constexpr (std::is_same<T, __half>::value) {
                const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
                x[2 * i] = f.x;
                x[2 * i + 1] = f.y;
            } else {
                x[2 * i] = __uint_as_float(w[i] << 16);
                x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
            }
        }
    }
};

// Cache rows are read once: past L1.
__device__ __forceinline__ uint4 ldg_stream16(const void* p) {
    uint4 v;
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
    return v;
}
__device__ __forceinline__ uint2 ldg_stream8(const void* p) {
    uint2 v;
    asm volatile("ld.global.L1::no_allocate.v2.u32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "l"(p));
    return v;
}

// Four values of an output row from the sums: rho counts the rows (token,
// head) of the request's kv head; acc in units of 2^(m - off), l in 2^(m - off + SUM_LOG).
template <typename T, int D>
__device__ __forceinline__ void write_row(const AttnArgs& a, int first, int h, int G, int rho, int col, float4 acc,
                                          float m, float l, float off) {
    const int64_t tok = first + rho / G;
    const int head = h * G + rho % G;
    float inv, down;
    row_factors(l, inv, down);
    store4(static_cast<T*>(a.out) + tok * a.out_stride + head * D + col,
           make_float4(acc.x * inv * down, acc.y * inv * down, acc.z * inv * down, acc.w * inv * down));
    if (col == 0 && a.lse != nullptr)
        a.lse[tok * a.heads + head] = l == 0.0f ? -INFINITY : 0.6931471805599453f * (m - off + SUM_LOG + log2f(l));
}

cudaError_t launch_attn_tiles(const DeviceInfo& dev, const KvView& c, int dtype, const AttnArgs& a, const RowsPlan& pl,
                              cudaStream_t s);
cudaError_t launch_attn_rows(const DeviceInfo& dev, const KvView& c, int dtype, const AttnArgs& a, const RowsPlan& pl,
                             cudaStream_t s);

}  // namespace cq
