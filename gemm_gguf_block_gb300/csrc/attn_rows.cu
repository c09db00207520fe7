// Attention over the 8-bit paged cache for few query rows a (request, kv head):
// decoding and verification (cq_attn_paged in include/cq_kv.h).
//
// With x_j = log2(e) * scale * s_k * (q . k_j) + log2(s_v), the int8 values k_j, v_j
// and their blocks' scales s_k, s_v:
//   P_j = 2^(x_j - M + OFF),  out = (sum_j P_j v_j) / (sum_j P_j / s_v),
//   lse = ln 2 * (M - OFF + log2(sum_j P_j / s_v)),
// so both scales cost one fused multiply-add a score and the tensor cores see
// the stored integers (exact in binary16). M is a running reference, raised
// only when a score passes it by RAISE: P_j then stays below 2^15, and a value
// that is small against the largest keeps its 11 bits down to 2^-21 of it.
//
// Both products are mma.sync m16n8k16 with the cache as the A operand: 16 keys
// against 8 query rows (token, head of the kv head's group), and 16 head
// dimensions against the 8 rows, so one decoded token of up to eight heads wastes
// no row. The cache is read once, straight from global memory into the A
// fragments' registers: a key row's 16-byte piece holds four k-steps of its lane,
// a value row's piece its lane's dimensions of all row tiles. Only the
// probabilities change lanes (one 8 x 8 transpose for 8 keys). fp32 queries and
// probabilities enter as two binary16 parts (22 bits).
//
// Work: every (request, kv head, tile of 8 or 16 rows) is a group of units of 64 keys; the
// units of all groups, in order, are split evenly over the CTAs, whatever the
// lengths. A CTA's warps take its piece's tiles in turn and merge in shared
// memory; pieces of a group that several CTAs share go to the workspace, and the
// CTA that arrives last at the group's counter joins them in order.
#include <algorithm>
#include <type_traits>

#include "attn_common.cuh"
#include "cq_device.cuh"
#include "cq_internal.h"
#include "kv.cuh"
#include "tc.cuh"

namespace cq {
namespace {

constexpr int NW = 4;                     // warps a CTA
constexpr int THREADS = NW * 32;
constexpr int UNIT = 64;                  // keys of a work unit
constexpr int MIN_UNITS = 2;              // a CTA is worth at least so many
constexpr int SETUP = 4;                  // units that beginning and merging a group is worth
constexpr int JOIN = 8;                   // partial results joined at a time
constexpr int AHEAD = 2;                  // tiles that a warp has on their way into L2
constexpr int KNOWN = THREADS;            // requests whose lengths stay in shared memory
// fp32: probabilities below this would be held to less than 17 bits by two binary16
// parts (which end at 2^-25). They enter as two bfloat16 parts instead, in the tiles that
// have any: 2^-20 of the largest and less, rare unless the softmax is very peaked.
constexpr float SMALL = 1.0f / 256.0f;

__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ void mma16816_bf16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t bf16_pair(float a, float b) {
    const __nv_bfloat162 x = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&x);
}

// A CTA's part of one group: what its rows are and see, and the keys to read.
struct Piece {
    int r, h, i;             // request, kv head, row tile
    int first, n, kv;        // the request's first token, new tokens, length
    int rows;                // of the tile
    int units, piece0, piece1;      // the group's units, and the piece's among them
    int all_from, all_stop;  // keys that every row sees
    int k_begin, k_end, ntile;
    int64_t group_u;         // the group's first unit
};

// Keys [from, stop) that some row of the request sees.
__device__ __forceinline__ void request_range(const AttnArgs& a, int n, int kv, int& from, int& stop) {
    from = 0;
    stop = kv;
    if (a.window > 0) {
        const int64_t f = static_cast<int64_t>(kv) - n + 1 - a.window;
        if (f > 0) from = static_cast<int>(min(f, static_cast<int64_t>(kv)));
    }
}

__device__ __forceinline__ int request_units(const AttnArgs& a, int n, int kv) {
    int from, stop;
    request_range(a, n, kv, from, stop);
    return max((stop - 1) / UNIT + 1 - from / UNIT, 1);      // (stop may be near 2^31)
}

__device__ __forceinline__ int atomic_inc_acq_rel(int* p) {
    int v;
    asm volatile("atom.acq_rel.gpu.global.add.s32 %0, [%1], 1;" : "=r"(v) : "l"(p) : "memory");
    return v;
}

// Transposes an 8 x 8 matrix of 16-bit values held as fragments (lane: row
// lane / 4, columns 2 (lane % 4), 2 (lane % 4) + 1).
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

// The items that the tiles kernel split over their keys, 16 rows of one at a time, over
// this grid's CTAs: parts in order, weighted by their references.
template <typename T, int D>
__device__ __forceinline__ void join_tiles(const AttnArgs& a, const RowsPlan& pl, int G) {
    constexpr int ROWF = D + 4;
    if (__ldcg(&pl.share->any) == 0) return;
    for (int w = blockIdx.x; w < pl.sms * 16; w += gridDim.x) {
        const int b = w >> 4, chunk = (w & 15) * 16;
        const int4* sp = reinterpret_cast<const int4*>(pl.share + b);
        const int4 s0 = __ldcg(sp), s1 = __ldcg(sp + 1);
        const TileShare sh{s0.x, s0.y, s0.z, s0.w, s1.x, s1.y, {0, 0}};
        if (sh.parts < 2 || chunk >= sh.rows) continue;
        for (int x = threadIdx.x; x < min(16, sh.rows - chunk) * (D / 4); x += THREADS) {
            const int row = chunk + x / (D / 4), col = (x % (D / 4)) * 4;
            const float* src = pl.tile_part + static_cast<int64_t>(b) * (256 * ROWF) + row * ROWF;
            float m = -INFINITY;
            for (int k = 0; k < sh.parts; ++k) m = fmaxf(m, __ldcg(src + static_cast<int64_t>(k) * (256 * ROWF) + D));
            const float base = m == -INFINITY ? 0.0f : m;
            float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            float lt = 0.0f;
#pragma unroll 4
            for (int k = 0; k < sh.parts; ++k) {
                const float* p = src + static_cast<int64_t>(k) * (256 * ROWF);
                const float f = exp2_approx(__ldcg(p + D) - base);
                const float4 v = __ldcg(reinterpret_cast<const float4*>(p + col));
                lt = fmaf(__ldcg(p + D + 1), f, lt);
                acc.x = fmaf(v.x, f, acc.x);
                acc.y = fmaf(v.y, f, acc.y);
                acc.z = fmaf(v.z, f, acc.z);
                acc.w = fmaf(v.w, f, acc.w);
            }
            write_row<T, D>(a, sh.first, sh.h, G, sh.row0 + row, col, acc, m, lt, TILES_OFF);
        }
    }
}

template <typename T, int D, int NB> struct Rows {
    static constexpr bool F32 = std::is_same<T, float>::value;
    static constexpr int RT = 8 * NB;                       // rows of a tile
    // The largest probability lies between 2^OFF and 2^(OFF + RAISE) = 2^15. fp32 raises its
    // reference sooner, so that fewer are SMALL.
    static constexpr float OFF = F32 ? 12.0f : 7.0f, RAISE = 15.0f - OFF;
    static constexpr int CTAS = NB == 1 && !F32 ? 4 : 3;    // an SM's CTAs (registers): one's merge hides behind the others' loads
    static constexpr int ROWF = D + 4;                      // floats of a merge row
    static constexpr int QF = (F32 ? 2 : 1) * NB * (D / 16) * 32;   // query fragments, 8 bytes each
    static int smem(int R) { return (((R + 1) * 8 + 15) & ~15) + QF * 8 + RT * 4 + NW * RT * (ROWF + 2) * 4; }
};

template <typename T, int D, int NB>
__global__ void __launch_bounds__(THREADS, Rows<T, D, NB>::CTAS) attn_rows_kernel(const KvView c, const AttnArgs a, const RowsPlan pl) {
    pdl_trigger();
    // Behind the tiles kernel this one runs beside it: every CTA of that one has waited for what
    // came before (see its first lines), and each CTA of this one waits for its end before it
    // leaves, so that this grid's end is the end of both.
    if (pl.after_tiles) __threadfence();
    else pdl_wait();
    auto leave = [&]() {
        if (!pl.after_tiles) return;
        pdl_wait();
        join_tiles<T, D>(a, pl, a.heads / c.heads);
    };
    using W = Rows<T, D, NB>;
    constexpr bool F32 = W::F32;
    // Probabilities enter as two binary16 parts (22 bits) where the result has 11 bits or more, else
    // as one: in bfloat16 the second part moved no error against 64 bits (1.7e-3 is the result's
    // rounding) and cost 62 -> 66 us at 64 ragged contexts; in binary16 it takes 2.5e-4 to 2.1e-4.
    constexpr bool SPLIT_P = !std::is_same<T, __nv_bfloat16>::value;
    constexpr int RT = W::RT, ROWF = W::ROWF;
    constexpr float OFF = W::OFF, RAISE = W::RAISE;
    constexpr int NSUB = 128 / D, KST = D / 16, MT = D / 16;      // a tile: NSUB blocks of 16 keys, 2 KB of keys
    constexpr int TK = 16 * NSUB;                                 // keys of a tile
    constexpr int BT = 32 / NSUB;                                 // tiles of a batch of page ids
    extern __shared__ __align__(16) uint8_t rows_smem[];
    int64_t* cum = reinterpret_cast<int64_t*>(rows_smem);                     // [R + 1] first unit of each request
    uint2* qf = reinterpret_cast<uint2*>(rows_smem + (((a.R + 1) * 8 + 15) & ~15));   // [1 or 2][KST][NB][32] B fragments
    float* merge = reinterpret_cast<float*>(qf + W::QF);                      // [NW][RT][ROWF]
    float* ml = merge + NW * RT * ROWF;                                       // [NW][RT][2]
    float* rowf = ml + NW * RT * 2;                                           // [RT] factor of each row's scores
    __shared__ int64_t wsum[NW];
    __shared__ int last_flag[2];
    __shared__ Piece held[2];                                                 // pieces of groups that other CTAs share
    __shared__ int held_on[2];
    __shared__ int known[KNOWN][3];
    __shared__ Piece pieces[2];                                               // this one and the next
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, tq = lane & 3;
    const int G = a.heads / c.heads;

    if (tid < 2) held_on[tid] = 0;
    // ---- every CTA counts all requests' units
    int64_t carry = 0;
    for (int r0 = 0; r0 < a.R; r0 += THREADS) {
        const int r = r0 + tid;
        int64_t x = 0;
        if (r < a.R) {
            int first, n, kv;
            request_of(c, a, r, first, n, kv);
            if (r < KNOWN) { known[r][0] = first; known[r][1] = n; known[r][2] = kv; }
            if (rows_take(pl, n, G)) x = static_cast<int64_t>(SETUP + request_units(a, n, kv)) * c.heads * ((static_cast<int64_t>(n) * G + RT - 1) / RT);
        }
        int64_t s = x;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t up = __shfl_up_sync(0xffffffffu, s, o);
            if (lane >= o) s += up;
        }
        if (lane == 31) wsum[warp] = s;
        __syncthreads();
        int64_t before = carry, all = 0;
#pragma unroll
        for (int w = 0; w < NW; ++w) {
            if (w < warp) before += wsum[w];
            all += wsum[w];
        }
        if (r < a.R) cum[r] = before + s - x;
        carry += all;
        __syncthreads();
    }
    if (tid == 0) cum[a.R] = carry;
    __syncthreads();
    const int64_t U = carry;
    if (U == 0) return leave();
    const int64_t nact = min(static_cast<int64_t>(gridDim.x), (U + MIN_UNITS - 1) / MIN_UNITS);
    const int64_t me = blockIdx.x;
    if (me >= nact) return leave();
    int64_t u = quot(me * U, nact);
    const int64_t u_end = quot((me + 1) * U, nact);
    const float lscale = fabsf(a.scale) * 1.4426950408889634f;
    bool first_piece = true;

    // The piece that begins at unit u.
    auto locate = [&](int64_t u, Piece& pc) {
        int lo = 0, hi = a.R;
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (cum[mid] <= u) lo = mid; else hi = mid;
        }
        pc.r = lo;
        if (lo < KNOWN) { pc.first = known[lo][0]; pc.n = known[lo][1]; pc.kv = known[lo][2]; }
        else request_of(c, a, lo, pc.first, pc.n, pc.kv);
        int from, stop;
        request_range(a, pc.n, pc.kv, from, stop);
        const int u0 = (from / UNIT) * UNIT;
        pc.units = request_units(a, pc.n, pc.kv);
        const int64_t in = u - cum[lo], gi = quot(in, SETUP + pc.units);
        pc.group_u = u - (in - gi * (SETUP + pc.units));
        pc.piece0 = static_cast<int>(max(u - pc.group_u - SETUP, int64_t(0)));
        const int nrt = (pc.n * G + RT - 1) / RT;
        pc.h = static_cast<int>(quot(gi, nrt));
        pc.i = static_cast<int>(gi - static_cast<int64_t>(pc.h) * nrt);
        pc.piece1 = static_cast<int>(min(static_cast<int64_t>(pc.units), u_end - pc.group_u - SETUP));
        pc.rows = min(RT, pc.n * G - RT * pc.i);
        // from the last row's first key to the first row's last
        int tfrom, tstop;
        row_range(a, pc.n, pc.kv, (RT * pc.i) / G, tfrom, pc.all_stop);
        row_range(a, pc.n, pc.kv, (RT * pc.i + pc.rows - 1) / G, pc.all_from, tstop);
        pc.k_begin = max(u0 + pc.piece0 * UNIT, (tfrom / TK) * TK);
        pc.k_end = static_cast<int>(min(u0 + static_cast<int64_t>(pc.piece1) * UNIT, static_cast<int64_t>(tstop)));
        pc.ntile = pc.k_end > pc.k_begin ? (pc.k_end - 1 - pc.k_begin) / TK + 1 : 0;
    };
    // What the loop over the tiles needs of its piece; the rest waits in shared memory.
    int k_begin = 0, k_end = 0, all_from = 0, all_stop = 0, turn = 0;
    int mine = 0;                                                 // the warp's tiles: warp, warp + NW, ...
    // Lane b of a batch holds the place and scales of sub-block b of the warp's
    // next 32; its page and scales of the batch after it (n_) are on their way meanwhile.
    int64_t head_off = 0;
    int n_page = -1;
    float n_ks = 0.0f, n_vs = 0.0f;
    int64_t b_at = -1;                                                      // offset of the sub-block's keys (and values)
    float b_ks = 0.0f, b_lv = 0.0f, b_rv = 0.0f;
    auto place = [&](int tl) { return k_begin + (warp + tl * NW) * TK + (lane % NSUB) * 16; };
    auto fetch_batch = [&](const Piece& pc, int t0) {
        const int tl = t0 + lane / NSUB, j0 = place(tl);                    // the warp's tile, its first key
        n_page = -1;
        if (tl < mine && j0 < k_end) {
            const int page = a.table[pc.r * a.max_blocks + (j0 >> c.page_shift)];
            if (page >= 0 && page < c.num_pages) {
                n_page = page;
                n_ks = c.k_scale[page * c.scale_stride + pc.h];
                n_vs = c.v_scale[page * c.scale_stride + pc.h];
            } else {
                atomicOr(a.status, CQ_DEV_KV_PAGE);
            }
        }
    };
    auto offset_of = [&](int page, int j0) {
        return page * c.page_stride + head_off + static_cast<int64_t>(j0 & (c.page_size - 1)) * D;
    };
    auto next_place = [&](int t0) { b_at = n_page >= 0 ? offset_of(n_page, place(t0 + lane / NSUB)) : -1; };
    auto next_scales = [&]() {
        b_ks = n_ks;
        value_factors<F32>(n_vs, b_lv, b_rv);
    };
    // Tile t begins its way into L2: the lanes that hold it in its batch.
    auto prefetch = [&](int t, bool next) {
        if (lane / NSUB != t % BT) return;
        const int64_t at = !next ? b_at : n_page >= 0 ? offset_of(n_page, place(t)) : -1;
        if (at >= 0) { bulk_prefetch_l2(c.k + at, 16 * D); bulk_prefetch_l2(c.v + at, 16 * D); }
    };
    uint4 kr[NSUB][2][D / 64];          // [sub-block][key g, g + 8][64 dimensions]
    uint32_t vr[NSUB][4][D / 32];       // [sub-block][its keys 2t, 2t+1, 2t+8, 2t+9][words]
    auto load_k = [&](int t) {
        const int at = (t % BT) * NSUB;
#pragma unroll
        for (int s = 0; s < NSUB; ++s) {
            const int64_t off = __shfl_sync(0xffffffffu, b_at, at + s);
            if (off < 0) continue;
            const int8_t* p = c.k + off + g * D + 16 * tq;
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int j = 0; j < D / 64; ++j) kr[s][i][j] = ldg_stream16(p + 8 * i * D + 64 * j);
        }
    };
    auto load_v = [&](int t) {
        const int at = (t % BT) * NSUB;
#pragma unroll
        for (int s = 0; s < NSUB; ++s) {
            const int64_t off = __shfl_sync(0xffffffffu, b_at, at + s);
            if (off < 0) continue;
            const int8_t* p = c.v + off + 2 * tq * D + g * (D / 8);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int8_t* q = p + ((i & 1) + 8 * (i >> 1)) * D;
                if constexpr (D == 128) {
                    const uint4 x = ldg_stream16(q);
                    vr[s][i][0] = x.x; vr[s][i][1] = x.y; vr[s][i][2] = x.z; vr[s][i][3] = x.w;
                } else {
                    const uint2 x = ldg_stream8(q);
                    vr[s][i][0] = x.x; vr[s][i][1] = x.y;
                }
            }
        }
    };
    // The query rows of the piece: consecutive dimensions of a lane, rows of a warp.
    constexpr int PER = D / 32, WR = RT / NW;
    Raw2<T> q[WR][PER / 2];                                       // as loaded: converted when the piece begins
    auto load_q = [&](const Piece& pc) {
#pragma unroll
        for (int w = 0; w < WR; ++w) {
            const int rho = RT * pc.i + min(warp + w * NW, pc.rows - 1);     // rows past the last are the last
            const int64_t tok = pc.first + rho / G;
            const T* src = static_cast<const T*>(a.q) + tok * a.q_stride + (pc.h * G + rho % G) * D + lane * PER;
#pragma unroll
            for (int i = 0; i < PER / 2; ++i) q[w][i].load(src + 2 * i);
        }
    };
    // A piece's first loads, all on their way before anything is waited for: the
    // next piece's while this one is merged.
    auto begin = [&](int64_t u) {
        Piece pc;
        locate(u, pc);
        k_begin = pc.k_begin;
        k_end = pc.k_end;
        all_from = pc.all_from;
        all_stop = pc.all_stop;
        head_off = static_cast<int64_t>(pc.h) * c.page_size * D;
        mine = pc.ntile > warp ? (pc.ntile - warp + NW - 1) / NW : 0;
        load_q(pc);
        if (mine > 0) fetch_batch(pc, 0);
        turn ^= 1;
        if (tid == 0) pieces[turn] = pc;
        return pc.piece1 > pc.piece0;
    };
    auto begin_tiles = [&]() {
        if (mine > 0) {
            next_place(0);
            load_k(0);
            load_v(0);
            for (int t = 1; t < AHEAD; ++t) prefetch(t, false);
            next_scales();
        }
    };
    if (!begin(u)) return leave();                                        // a part of one group's setup
    begin_tiles();

    for (;;) {
        // ---- query fragments: k-step (j, s) of lane (g, t) holds dimensions 64j + 16t + 4s + 0..3 of row g
        // (the barrier at the previous piece's merge is behind the last reader of its fragments)
#pragma unroll
        for (int w = 0; w < WR; ++w) {
            const int row = warp + w * NW;
            // A power of two brings the row's largest value to [2^8, 2^9): exact, and
            // nothing that matters is below binary16's range. NaN for a row that is not finite.
            uint32_t top = 0;
            float2 x[PER / 2];
#pragma unroll
            for (int i = 0; i < PER / 2; ++i) {
                x[i] = q[w][i].value();
                top = max(top, max(__float_as_uint(fabsf(x[i].x)), __float_as_uint(fabsf(x[i].y))));
            }
            top = __reduce_max_sync(0xffffffffu, top);
            float mul, back;
            row_scale(top, mul, back);
            if (a.scale < 0.0f) mul = -mul;
            if (lane == 0) rowf[row] = back * lscale;
#pragma unroll
            for (int i = 0; i < PER; i += 2) {
                const int d = lane * PER + i;
                const int j = d >> 6, t = (d >> 4) & 3, s = (d >> 2) & 3, half = (d >> 1) & 1;
                const float v0 = x[i / 2].x * mul, v1 = x[i / 2].y * mul;
                const __half2 hi = __floats2half2_rn(v0, v1);
                uint32_t* dst = reinterpret_cast<uint32_t*>(qf + ((4 * j + s) * NB + (row >> 3)) * 32 + 4 * (row & 7) + t) + half;
                *dst = *reinterpret_cast<const uint32_t*>(&hi);
                if constexpr (F32) {
                    const float2 back2 = __half22float2(hi);
                    const __half2 lo = __floats2half2_rn(v0 - back2.x, v1 - back2.y);
                    dst[KST * NB * 32 * 2] = *reinterpret_cast<const uint32_t*>(&lo);
                }
            }
        }
        __syncthreads();
        // this lane's rows, 8b + 2t + e: what they see, their scores' factors, running reference and sum
        int rfrom[NB][2], rstop[NB][2];
        float rf[NB][2], M[NB][2], l[NB][2];
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int row = 8 * b + 2 * tq + e;
                const Piece& pc = pieces[turn];
                row_range(a, pc.n, pc.kv, (RT * pc.i + row) / G, rfrom[b][e], rstop[b][e]);
                if (row >= pc.rows) rfrom[b][e] = rstop[b][e] = 0;
                rf[b][e] = rowf[row];
                M[b][e] = -INFINITY;
                l[b][e] = 0.0f;
            }
        uint2 qh[NB == 1 ? KST : 1];                              // one block's fragments stay in registers
        if constexpr (NB == 1) {
#pragma unroll
            for (int ks = 0; ks < KST; ++ks) qh[ks] = qf[ks * 32 + lane];
        }
        float o[NB][MT][4];                                       // dimensions (D / 8) g + 2i (0, 1) and + 2i + 1 (2, 3) of rows 2t, 2t + 1
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
            for (int i = 0; i < MT; ++i) o[b][i][0] = o[b][i][1] = o[b][i][2] = o[b][i][3] = 0.0f;

        for (int t = 0; t < mine; ++t) {
            // what belongs to this tile, before the batch moves on
            bool on[NSUB];
            float ks_[NSUB], lv_[NSUB], rv_[NSUB];
#pragma unroll
            for (int s = 0; s < NSUB; ++s) {
                const int at = (t % BT) * NSUB + s;
                on[s] = __shfl_sync(0xffffffffu, b_at, at) >= 0;
                ks_[s] = __shfl_sync(0xffffffffu, b_ks, at);
                lv_[s] = __shfl_sync(0xffffffffu, b_lv, at);
                rv_[s] = __shfl_sync(0xffffffffu, b_rv, at);
            }
            if (t % BT == BT / 2) fetch_batch(pieces[turn], t - BT / 2 + BT);
            prefetch(t + AHEAD, t % BT + AHEAD >= BT);
            float sc[NSUB][NB][4] = {}, sl[F32 ? NSUB : 1][F32 ? NB : 1][4] = {};    // fp32: the lower parts' scores, a chain of their own
#pragma unroll
            for (int ks = 0; ks < KST; ++ks) {
                uint2 qa[NB], ql[NB];
#pragma unroll
                for (int b = 0; b < NB; ++b) {
                    if constexpr (NB == 1) qa[b] = qh[ks];
                    else qa[b] = qf[(ks * NB + b) * 32 + lane];
                    if constexpr (F32) ql[b] = qf[((KST + ks) * NB + b) * 32 + lane];
                }
#pragma unroll
                for (int s = 0; s < NSUB; ++s) {
                    uint32_t w[2], ka[4];
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const uint4& kk = kr[s][i][ks >> 2];
                        w[i] = (ks & 3) == 0 ? kk.x : (ks & 3) == 1 ? kk.y : (ks & 3) == 2 ? kk.z : kk.w;
                        tc::s8x4_half(w[i], ka[i], ka[2 + i]);
                    }
#pragma unroll
                    for (int b = 0; b < NB; ++b) {
                        mma16816(sc[s][b], ka, qa[b].x, qa[b].y);
                        if constexpr (F32) mma16816(sl[s][b], ka, ql[b].x, ql[b].y);
                    }
                }
            }
            // the next tile's keys come in behind the softmax and the second product, its values behind the next scores
            const bool more = t + 1 < mine;
            if (more) {
                if ((t + 1) % BT == 0) { next_place(t + 1); next_scales(); }
                load_k(t + 1);
            }
#pragma unroll
            for (int s = 0; s < NSUB; ++s) {
                if (!on[s]) continue;                                           // warp-uniform
                const int j0 = k_begin + (warp + t * NW) * TK + s * 16;
                // x_j, hidden keys at -inf
                const bool whole = j0 >= all_from && j0 + 16 <= all_stop;
                bool raise = false;
                float top[NB][2];
#pragma unroll
                for (int b = 0; b < NB; ++b) {
                    const float f[2] = {ks_[s] * rf[b][0], ks_[s] * rf[b][1]};
#pragma unroll
                    for (int e = 0; e < 4; ++e) {                               // key g + 8 (e / 2), row 2t + e % 2
                        if constexpr (F32) sc[s][b][e] += sl[s][b][e];
                        float x = fmaf(sc[s][b][e], f[e & 1], lv_[s]);
                        if (!whole) {
                            const int j = j0 + g + 8 * (e >> 1);
                            if (j < rfrom[b][e & 1] || j >= rstop[b][e & 1]) x = -INFINITY;
                        }
                        sc[s][b][e] = x;
                    }
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        top[b][e] = fmaxf(sc[s][b][e], sc[s][b][2 + e]);
                        raise |= top[b][e] > M[b][e] + RAISE;
                    }
                }
                if (__any_sync(0xffffffffu, raise)) {
#pragma unroll
                    for (int b = 0; b < NB; ++b)
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            float m = top[b][e];
                            m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 4));
                            m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 8));
                            m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 16));
                            const float old = M[b][e];
                            if (m > old + RAISE) {                              // the row's own, the same in its eight lanes
                                M[b][e] = m;
                                const float f = exp2_approx(old - m);           // 0 from -inf
                                l[b][e] *= f;
#pragma unroll
                                for (int i = 0; i < MT; ++i) { o[b][i][e] *= f; o[b][i][2 + e] *= f; }
                            }
                        }
                }
                uint2 ph[NB], plo[NB], ps[NB], pt[NB];
                bool small = false;                         // (hidden keys' zeros too: the tiles at the edges)
#pragma unroll
                for (int b = 0; b < NB; ++b) {
                    float sum[2] = {0.0f, 0.0f};
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float m = M[b][e & 1], base = m == -INFINITY ? 0.0f : m - OFF;
                        const float p = exp2_approx(sc[s][b][e] - base);
                        sum[e & 1] += p;                                        // unrounded: lse is held to fp32
                        if constexpr (F32) small |= p < SMALL;
                        sc[s][b][e] = p;
                    }
                    // a row that sees nothing here must not meet a scale that is not finite
                    l[b][0] += sum[0] != 0.0f ? sum[0] * rv_[s] : 0.0f;
                    l[b][1] += sum[1] != 0.0f ? sum[1] * rv_[s] : 0.0f;
                }
                if constexpr (F32) {
                    small = __any_sync(0xffffffffu, small);
                    if (small) {
#pragma unroll
                        for (int b = 0; b < NB; ++b) {
                            float sm[4];
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                sm[e] = sc[s][b][e] < SMALL ? sc[s][b][e] : 0.0f;
                                sc[s][b][e] -= sm[e];
                            }
                            const uint32_t s0 = bf16_pair(sm[0], sm[1]), s1 = bf16_pair(sm[2], sm[3]);
                            const uint32_t t0 = bf16_pair(sm[0] - __uint_as_float(s0 << 16), sm[1] - __uint_as_float(s0 & 0xffff0000u));
                            const uint32_t t1 = bf16_pair(sm[2] - __uint_as_float(s1 << 16), sm[3] - __uint_as_float(s1 & 0xffff0000u));
                            ps[b] = make_uint2(transpose8(s0), transpose8(s1));
                            pt[b] = make_uint2(transpose8(t0), transpose8(t1));
                        }
                    }
                }
#pragma unroll
                for (int b = 0; b < NB; ++b) {
                    const float (&p)[4] = sc[s][b];
                    const __half2 h0 = __floats2half2_rn(p[0], p[1]), h1 = __floats2half2_rn(p[2], p[3]);
                    ph[b] = make_uint2(transpose8(*reinterpret_cast<const uint32_t*>(&h0)),
                                       transpose8(*reinterpret_cast<const uint32_t*>(&h1)));
                    if constexpr (SPLIT_P) {
                        const float2 f0 = __half22float2(h0), f1 = __half22float2(h1);
                        const __half2 l0 = __floats2half2_rn(p[0] - f0.x, p[1] - f0.y), l1 = __floats2half2_rn(p[2] - f1.x, p[3] - f1.y);
                        plo[b] = make_uint2(transpose8(*reinterpret_cast<const uint32_t*>(&l0)),
                                            transpose8(*reinterpret_cast<const uint32_t*>(&l1)));
                    }
                }
                // The second product follows at once: a later sub-block may raise M.
#pragma unroll
                for (int w = 0; w < D / 32; ++w) {
                    // four dimensions of keys (2t, 2t+1) and (2t+8, 2t+9), as pairs of keys: two row tiles
                    uint32_t va[2][4];
                    tc::s8x4_half(__byte_perm(vr[s][0][w], vr[s][1][w], 0x5140), va[0][0], va[0][1]);
                    tc::s8x4_half(__byte_perm(vr[s][0][w], vr[s][1][w], 0x7362), va[1][0], va[1][1]);
                    tc::s8x4_half(__byte_perm(vr[s][2][w], vr[s][3][w], 0x5140), va[0][2], va[0][3]);
                    tc::s8x4_half(__byte_perm(vr[s][2][w], vr[s][3][w], 0x7362), va[1][2], va[1][3]);
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
#pragma unroll
                        for (int b = 0; b < NB; ++b) {
                            mma16816(o[b][2 * w + x], va[x], ph[b].x, ph[b].y);
                            if constexpr (SPLIT_P) mma16816(o[b][2 * w + x], va[x], plo[b].x, plo[b].y);
                        }
                        if constexpr (F32) {
                            if (small) {
                                uint32_t vb[4];
#pragma unroll
                                for (int i = 0; i < 4; ++i) vb[i] = half_to_bf16(va[x][i]);
#pragma unroll
                                for (int b = 0; b < NB; ++b) {
                                    mma16816_bf16(o[b][2 * w + x], vb, ps[b].x, ps[b].y);
                                    mma16816_bf16(o[b][2 * w + x], vb, pt[b].x, pt[b].y);
                                }
                            }
                        }
                    }
                }
            }
            if (more) load_v(t + 1);
        }

        // ---- the warps' parts of the piece
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float lt = l[b][e];
                lt += __shfl_xor_sync(0xffffffffu, lt, 4);
                lt += __shfl_xor_sync(0xffffffffu, lt, 8);
                lt += __shfl_xor_sync(0xffffffffu, lt, 16);
                const int row = 8 * b + 2 * tq + e;
                if (row < pieces[turn].rows) {
                    if (g == 0) { ml[(warp * RT + row) * 2] = M[b][e]; ml[(warp * RT + row) * 2 + 1] = lt; }
                    float* dst = merge + (warp * RT + row) * ROWF + g * (D / 8);
#pragma unroll
                    for (int i = 0; i < MT; i += 2)
                        *reinterpret_cast<float4*>(dst + 2 * i) = make_float4(o[b][i][e], o[b][i][2 + e], o[b][i + 1][e], o[b][i + 1][2 + e]);
                }
            }
        const Piece& done = pieces[turn];
        const int rows = done.rows;
        u = done.group_u + SETUP + done.piece1;
        const bool more = u + SETUP < u_end;                       // u begins a group, or u_end was in this one
        if (more) (void)begin(u);
        __syncthreads();
        if (more) begin_tiles();
        const int used = min(NW, max(done.ntile, 1));                               // warps that had a tile (warp 0 always counts)
        const bool whole = done.piece0 == 0 && done.piece1 == done.units;
        const int slot = first_piece ? 0 : 1;                                  // only a first and a last piece may be parts
        float* part = pl.part + (me * 2 + slot) * (16 * ROWF);
        first_piece = false;
        if (!whole && tid == 0) { held[slot] = done; held_on[slot] = 1; }
        for (int x = tid; x < rows * (D / 4); x += THREADS) {
            const int row = x / (D / 4), col = (x % (D / 4)) * 4;
            float m = -INFINITY;
            for (int w = 0; w < used; ++w) m = fmaxf(m, ml[(w * RT + row) * 2]);
            const float base = m == -INFINITY ? 0.0f : m;
            float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            float lt = 0.0f;
            for (int w = 0; w < used; ++w) {
                const float f = exp2_approx(ml[(w * RT + row) * 2] - base);
                const float4 v = *reinterpret_cast<const float4*>(merge + (w * RT + row) * ROWF + col);
                lt = fmaf(ml[(w * RT + row) * 2 + 1], f, lt);
                acc.x = fmaf(v.x, f, acc.x);
                acc.y = fmaf(v.y, f, acc.y);
                acc.z = fmaf(v.z, f, acc.z);
                acc.w = fmaf(v.w, f, acc.w);
            }
            if (whole) {
                write_row<T, D>(a, done.first, done.h, G, RT * done.i + row, col, acc, m, lt, OFF);
            } else {
                *reinterpret_cast<float4*>(part + row * ROWF + col) = acc;
                if (col == 0) { part[row * ROWF + D] = m; part[row * ROWF + D + 1] = lt; }
            }
        }
        if (!more) break;
        // the merge region and the fragments are free once every warp is here
        __syncthreads();
    }

    // ---- Groups that this CTA has a part of lie with CTAs c0..c1; the last of them to arrive at
    // the group's counter joins the parts. Both of this CTA's arrive here, together: the fence and
    // the counters' latency are paid once.
    __syncthreads();
    auto first_cta = [&](const Piece& pc) { return quot((pc.group_u + SETUP + 1) * nact - 1, U); };
    auto last_cta = [&](const Piece& pc) { return quot((pc.group_u + SETUP + pc.units) * nact - 1, U); };
    if (tid < 2) {
        last_flag[tid] = 0;
        if (held_on[tid]) {
            const int64_t c0 = first_cta(held[tid]), c1 = last_cta(held[tid]);
            // (releases what the CTA wrote before the barrier, and acquires the others' parts)
            last_flag[tid] = atomic_inc_acq_rel(pl.count + c0) == static_cast<int>(c1 - c0);
            if (last_flag[tid]) pl.count[c0] = 0;                              // as the next call wants it
        }
    }
    __syncthreads();
    for (int hs = 0; hs < 2; ++hs) {
        if (!last_flag[hs]) continue;
        const Piece& pc = held[hs];
        const int64_t c0 = first_cta(pc), c1 = last_cta(pc);
        // The first CTA holds the group in its second slot unless the group begins with it; the others
        // begin inside the group: their first.
        const int slot0 = quot(c0 * U, nact) < pc.group_u;
        for (int x = tid; x < pc.rows * (D / 4); x += THREADS) {
            const int row = x / (D / 4), col = (x % (D / 4)) * 4;
            float m = -INFINITY;
            float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            float lt = 0.0f;
            // in order, so that the result does not depend on who joins; eight at a time, their loads in flight together
            for (int64_t cb = c0; cb <= c1; cb += JOIN) {
                float mc[JOIN], lc[JOIN];
                float4 v[JOIN];
#pragma unroll
                for (int k = 0; k < JOIN; ++k) {
                    const int64_t cc = min(cb + k, c1);
                    const float* src = pl.part + (cc * 2 + (cc == c0 ? slot0 : 0)) * (16 * ROWF) + row * ROWF;
                    mc[k] = cb + k <= c1 ? __ldcg(src + D) : -INFINITY;
                    lc[k] = __ldcg(src + D + 1);
                    v[k] = __ldcg(reinterpret_cast<const float4*>(src + col));
                }
#pragma unroll
                for (int k = 0; k < JOIN; ++k) {
                    if (cb + k > c1) continue;
                    const float m2 = fmaxf(m, mc[k]), base = m2 == -INFINITY ? 0.0f : m2;
                    const float f = exp2_approx(m - base), fc = exp2_approx(mc[k] - base);
                    lt = lt * f + lc[k] * fc;
                    acc.x = acc.x * f + v[k].x * fc;
                    acc.y = acc.y * f + v[k].y * fc;
                    acc.z = acc.z * f + v[k].z * fc;
                    acc.w = acc.w * f + v[k].w * fc;
                    m = m2;
                }
            }
            write_row<T, D>(a, pc.first, pc.h, G, RT * pc.i + row, col, acc, m, lt, OFF);
        }
    }
    leave();
}

template <typename T, int D, int NB>
cudaError_t launch_rows_n(const DeviceInfo& dev, const KvView& c, const AttnArgs& a, const RowsPlan& pl, cudaStream_t s) {
    using W = Rows<T, D, NB>;
    const int smem = W::smem(a.R);
    if (smem > dev.smem_optin) return cudaErrorInvalidConfiguration;
    cudaError_t e = raise_smem_limit(reinterpret_cast<const void*>(attn_rows_kernel<T, D, NB>), smem);
    if (e != cudaSuccess) return e;
    const int ctas = std::min(dev.sm_count * W::CTAS, ATTN_MAX_CTAS);
    return launch_kernel(attn_rows_kernel<T, D, NB>, dim3(static_cast<unsigned>(ctas)), dim3(THREADS), static_cast<size_t>(smem), s, c, a, pl);
}

// Tiles of 8 rows where a request's rows of one kv head fit them, else of 16: the
// conversion of the cache's bytes is then shared by two row blocks.
template <typename T, int D>
cudaError_t launch_rows_t(const DeviceInfo& dev, const KvView& c, const AttnArgs& a, const RowsPlan& pl, cudaStream_t s) {
    return a.max_new * (a.heads / c.heads) <= 8 ? launch_rows_n<T, D, 1>(dev, c, a, pl, s) : launch_rows_n<T, D, 2>(dev, c, a, pl, s);
}

}  // namespace

cudaError_t launch_attn_rows(const DeviceInfo& dev, const KvView& c, int dtype, const AttnArgs& a, const RowsPlan& pl,
                             cudaStream_t s) {
    const bool d64 = c.dim == 64;
    switch (dtype) {
    case CQ_F32: return d64 ? launch_rows_t<float, 64>(dev, c, a, pl, s) : launch_rows_t<float, 128>(dev, c, a, pl, s);
    case CQ_F16: return d64 ? launch_rows_t<__half, 64>(dev, c, a, pl, s) : launch_rows_t<__half, 128>(dev, c, a, pl, s);
    case CQ_BF16:
        return d64 ? launch_rows_t<__nv_bfloat16, 64>(dev, c, a, pl, s) : launch_rows_t<__nv_bfloat16, 128>(dev, c, a, pl, s);
    default: return cudaErrorInvalidValue;
    }
}

}  // namespace cq
