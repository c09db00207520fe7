// Attention over the 8-bit paged cache for many query rows a (request, kv head):
// prompts and chunks of them (cq_attn_paged in include/cq_kv.h), trees of drafts
// (cq_attn_tree in include/cq_tree.h).
//
// The mathematics is attn_rows.cu's: x_j = log2(e) scale s_k (q . k_j) + log2(s_v),
// P_j = 2^(x_j - M + OFF), out = sum P_j v_j / sum (P_j / s_v). Here the products
// run on tcgen05 with the accumulators in tensor memory: a CTA takes 256 rows
// (token, head of the kv head's group) as two tiles of 128 -- fp32: 128 rows --
// against 128 keys at a time.
//   S = Q K^T: both from shared memory, K-major, 128-byte swizzle; K the stored
//     integers as binary16 (exact). fp32 queries are two binary16 parts, two MMAs.
//   O += P V: P from tensor memory, V from shared memory as it lies in the cache (keys
//     as rows, MN-major). fp32: P is three bfloat16 parts (24 bits over fp32's whole
//     range), and V bfloat16.
// Warps: 0-7 softmax, a thread to a row (fp32: two threads, 64 keys each); 8-11
// convert the cache's bytes to operands, two stages of keys and two of values;
// 12 issues the MMAs, 13-15 only fill the last warpgroup, whose registers the softmax
// gets. The tiles are half a step apart: while one's softmax runs, the other's MMAs do.
// (Two threads a row, 16 softmax warps, are 5% slower at the prompt below: the exchange of
// the rows' largest costs more than the shorter loops gain. Eight converter warps leave the
// softmax 168 registers or fewer, it spills, and the prompt takes a quarter longer.)
// Measured, 8192 tokens, 32 heads on 8, dim 128, bf16: 437 us, 1.26 PFLOP/s. The softmax
// (3000 of a step's 3500 cycles) and the converters bound it together: without the
// converters' loads and stores it takes 12% less, without the exponentials no less.
// Few items are split over their keys; the rows kernel, which always follows, joins
// the parts.
// Trees: TREE builds have the rows' masks in the steps that are not whole. NARROW ones take a tile of 128 rows alone, two
// threads a row, with eight converter warps that copy the bytes asynchronously: 64 contexts of 200-8190 keys, 32
// heads on 8 of 128, bf16, 12 to 36 rows take 113 us (two tiles: 162 together with the rows kernel). A step takes
// 2400 cycles whatever the rows: 900 of them a thread's exponentials, the rest one wait behind another (scores, meeting,
// product, converters); an item's beginning and end 9 us. Tried for NARROW without gain: 64 keys a step and two CTAs
// an SM (the same time), the queries in tensor memory, two steps' P.
// A block of 16 keys carries (s_k, log2 s_v, 1 / s_v) in shared memory; a block outside
// the cache or the request's keys has s_k = 0 and log2 s_v = -inf, so P = 0 whatever
// integers its place holds.
#include <algorithm>
#include <climits>
#include <type_traits>

#include "attn_common.cuh"
#include "cq_device.cuh"
#include "cq_internal.h"
#include "kv.cuh"
#include "tc.cuh"

namespace cq {
namespace {

constexpr float OFF = TILES_OFF, RAISE = 8.0f;
constexpr int MIN_STEPS = 3;              // a part of an item has at least so many, where it has parts
constexpr int INFO = 4;                   // steps whose scales are kept

enum { B_Q = 0, B_K_FULL = 1, B_K_EMPTY = 3, B_V_FULL = 5, B_V_EMPTY = 7, B_S = 9, B_P = 11, B_O = 13, B_INFO = 15, B_FREE = 19, B_DRAINED = 21 };

// Token and head of a kv head's group of an item's rows: rows count on from row0 = tok0 * G +
// head0. The quotient by G <= 1024 of a number below 1280, by a reciprocal in 21 bits: exact,
// since the number times the reciprocal's error (below G) stays under 2^21.
struct RowMap {
    int tok0, head0, G;
    uint32_t inv;
    __device__ __forceinline__ RowMap(int row0, int g) : tok0(row0 / g), head0(row0 % g), G(g), inv(((1u << 21) + g - 1) / g) {}
    __device__ __forceinline__ void of(int row, int& tok, int& head) const {
        const int x = head0 + row, t = static_cast<int>((x * inv) >> 21);
        tok = tok0 + t;
        head = x - t * G;
    }
};

template <typename T, int D, bool TREE, bool NARROW> struct Tiles {
    static constexpr bool F32 = std::is_same<T, float>::value;
    static_assert(!(F32 && NARROW), "fp32 has one row tile always");
    // binary16 trees: P in two parts (21 bits), so that a tree's precision, 22 bits in the rows kernel, does not hang on
    // what stands beside it in the call. (64 contexts of 200-8190, 12-36 rows: 128 us, 114 with one part.) bfloat16's
    // results have 8 bits: one part.
    static constexpr bool PAIR = NARROW && std::is_same<T, __half>::value;
    static constexpr int PARTS = F32 ? 3 : PAIR ? 2 : 1;   // of P
    // Trees: the MMAs' sums are cut off at each addition, up to 5e-9 of a result a key, 1e-8 with P in two parts (fp32: 7e-5 at
    // 60000 random keys, 2e-4 at 40000 of one sign, where sums that round are 1e-6 off; binary16 7e-4 at 65536 of one sign, its
    // own rounding 2e-4). So a result begins anew every FLUSH steps, and the softmax threads add the last one to totals of their
    // own: every 512 keys for fp32 (1.1e-6 at any length; every eighth step leaves 1.7e-6), every 4096 for binary16 in two parts and 8192 in
    // one (4e-5 at most), every 32768 for bfloat16 (2e-4, a twentieth of half a step). 64 contexts of 200-8190 keys, 12-36 rows of 128: fp32 212 us,
    // 201 with one result throughout, binary16 128 and 124, bfloat16 113 and 111 (whose contexts are too short to come here).
    static constexpr int FLUSH = !TREE ? 0 : F32 ? 4 : PAIR ? 32 : std::is_same<T, __half>::value ? 64 : 256;
    // Two row tiles a CTA and four converter warps; NARROW: one tile, a row's keys halved between two threads as in fp32,
    // and eight converter warps.
    static constexpr int KEYS = 128;                       // keys of a step
    static constexpr int SOFT = 256;                       // softmax threads
    static constexpr int CONV = NARROW ? 256 : 128;        // converter threads
    static constexpr int THREADS = SOFT + CONV + 128;      // the last four warps: one issues the MMAs
    // Registers a thread of each role; the roles' sum is what the launch gives. 512 threads have 128
    // each: 256 * 176 + 128 * 104 + 128 * 56 = 512 * 128. 640 have 96: 256 * 128 + 256 * 80 + 128 * 64 = 640 * 96.
    static constexpr int REGS_SOFT = NARROW ? 128 : 176, REGS_CONV = NARROW ? 80 : 104, REGS_MMA = NARROW ? 64 : 56;
    static constexpr int KW = KEYS / (CONV / 32);          // keys of a converter warp
    static constexpr int NBK = KW / 16;                    // their blocks of 16
    static constexpr int MT = F32 || NARROW ? 1 : 2;       // row tiles
    static constexpr int ROWS = 128 * MT;
    static constexpr int SPLIT = SOFT / (128 * MT);        // softmax threads of a row
    static constexpr int KT = KEYS / SPLIT;                // their keys
    static constexpr int OC = D / SPLIT;                   // and their columns of the result
    static constexpr int QB = 128 * D * 2;                 // one query operand
    static constexpr int KB = KEYS * D * 2;
    static constexpr int OFF_Q = 1024;
    static constexpr int OFF_K = OFF_Q + (NARROW ? 1 : 2) * QB;
    static constexpr int OFF_V = OFF_K + 2 * KB;
    // NARROW: the cache's bytes on their way, a step's keys or values a slot
    static constexpr int SLOTS = NARROW ? 3 : 0, SLOT = KEYS * D;
    static constexpr int OFF_RAW = OFF_V + 2 * KB;
    static constexpr int SMEM = OFF_RAW + SLOTS * SLOT + 1024;     // + alignment slack of the dynamic base
    // Tensor memory columns. 16-bit types: the scores of one tile at a time, both tiles' P, both
    // results. (A tile's scores are there only until its softmax has them in registers, so the
    // other's next ones follow while the first is at work: no softmax waits for its own P's
    // product. With 128 columns of scores a tile, P over them, the prompt takes 2% longer.)
    // fp32: scores -- two steps' where that fits, so that one step's are there before the
    // other's softmax is done --, overlaid by the first two parts of P, the third part, and two
    // results: of P's first part and of the other two. (The MMAs' sums are cut off, not rounded:
    // the small parts' 16 additions a step would cost a sum of full size as much as the first
    // part's 8.)
    // NARROW: two steps' scores, P in columns of its own. (Two steps' P as well gain nothing.)
    static constexpr int SBUF = (F32 && D == 64) || NARROW ? 2 : 1;
    static constexpr uint32_t S0 = 0, S1 = 128;
    static constexpr uint32_t SP = 128 * SBUF;             // P, 64 columns a tile; fp32: P's third part
    static constexpr uint32_t O0 = SP + 64 * MT;
    static constexpr uint32_t O1 = O0 + (F32 ? D : NARROW ? 0 : 128);   // fp32: the smaller result; two tiles: the second's
    static constexpr uint32_t P2 = 448;                    // P's second part
    static constexpr uint32_t T0 = 448;                    // FLUSH: totals, from a thread's 32nd column on
    static_assert(!F32 || FLUSH == 0 || OC == 32 || (OC == 64 && O1 + D <= T0), "totals");
    static_assert(O1 + D <= (PAIR ? P2 : 512), "tensor memory");
};

template <typename T, int D, bool TREE, bool NARROW>
__global__ void __launch_bounds__(Tiles<T, D, TREE, NARROW>::THREADS, 1) attn_tiles_kernel(const KvView c, const AttnArgs a, const RowsPlan pl) {
    // The rows kernel that follows begins when every CTA of this one has passed here, and
    // does not wait for the end of it: what both read is complete by then.
    pdl_wait();
    pdl_trigger();
    using W = Tiles<T, D, TREE, NARROW>;
    constexpr bool F32 = W::F32;
    constexpr int KEYS = W::KEYS, SOFT = W::SOFT, CONV = W::CONV, THREADS = W::THREADS;
    constexpr int MT = W::MT, ROWS = W::ROWS, SPLIT = W::SPLIT, KT = W::KT, OC = W::OC, SBUF = W::SBUF;
    extern __shared__ uint8_t tiles_smem[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(tiles_smem) + 1023) & ~uintptr_t(1023));
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem);
    __shared__ uint32_t tmem_holder;
    __shared__ int abort_word;
    __shared__ int item[4];                                // request, its first token, new tokens, length
    __shared__ int item_at;                                // index inside the request
    __shared__ int64_t scan[THREADS / 32];
    __shared__ __align__(16) float info[INFO][3][KEYS / 16];   // s_k, log2 s_v, 1 / s_v of a step's blocks
    __shared__ float rowf[ROWS];                           // the rows' factors
    __shared__ float exch[2][SPLIT][ROWS];                 // [step's parity]
    const SmemFlag abort_flag{smem_u32(&abort_word)};
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int G = a.heads / c.heads;

    // ---- this CTA's item: requests in order; inside one the last rows (the longest) first, heads together.
    // Where the items are too few for half the SMs, each is split over its keys into parts of about
    // equal length, together one CTA an SM.
    if (tid == 0) { item[0] = -1; abort_word = 0; }
    auto items_of = [&](int n_) {
        return tiles_take(pl, n_, G) ? static_cast<int>((static_cast<int64_t>(n_) * G + ROWS - 1) / ROWS) : 0;
    };
    // Keys and steps of row tile i of a request: what some row sees, and what all rows see.
    auto range_of = [&](int n_, int kv_, int i, int& key0_, int& stop_, int& all_from_, int& all_stop_) {
        const int last = min((i + 1) * ROWS, n_ * G) - 1;
        tile_range<TREE>(a, n_, kv_, i * ROWS / G, last / G, key0_, all_from_, all_stop_, stop_);
        key0_ = key0_ / KEYS * KEYS;
        return stop_ > key0_ ? (stop_ - 1 - key0_) / KEYS + 1 : 0;       // (stop may be near 2^31)
    };
    // Trees: long requests first, where they are few enough to be put in order: the items that begin last are short.
    // (64 contexts of 200-8190, trees of 3-9 tokens: 123 us when it was brought in, in the requests' order 158)
    constexpr int SORTED = 128;
    __shared__ int sort_len[TREE ? SORTED : 1];
    __shared__ int4 in_order[TREE ? SORTED : 1];            // request, first token, new tokens, length
    const bool sorted = TREE && a.R <= SORTED;
    if constexpr (TREE) {
        if (sorted) {
            int f_ = 0, n_ = 0, kv_ = 0;
            if (tid < a.R) {
                request_of(c, a, tid, f_, n_, kv_);
                sort_len[tid] = kv_;
            }
            __syncthreads();
            if (tid < a.R) {
                int rank = 0;
                for (int i = 0; i < a.R; ++i) rank += sort_len[i] > kv_ || (sort_len[i] == kv_ && i < tid);
                in_order[rank] = make_int4(tid, f_, n_, kv_);
            }
            __syncthreads();
        }
    }
    // The sum of count(n, kv) over the requests; where the CTA's index falls into a request's
    // count, notes the request and the index in it.
    auto over_requests = [&](auto&& count) {
        int64_t carry = 0;
        for (int r0 = 0; r0 < a.R; r0 += THREADS) {
            int r_ = r0 + tid;
            int f_ = 0, n_ = 0, kv_ = 0;
            int64_t x = 0;
            if (r_ < a.R) {
                if (TREE && sorted) {
                    const int4 q_ = in_order[r_];
                    r_ = q_.x; f_ = q_.y; n_ = q_.z; kv_ = q_.w;
                } else {
                    request_of(c, a, r_, f_, n_, kv_);
                }
                x = count(n_, kv_);
            }
            int64_t s = x;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int64_t up = __shfl_up_sync(0xffffffffu, s, o);
                if (lane >= o) s += up;
            }
            if (lane == 31) scan[warp] = s;
            __syncthreads();
            int64_t before = carry, all = 0;
            for (int w = 0; w < THREADS / 32; ++w) {
                if (TREE && r0 + 32 * w >= a.R) break;       // (a tree call's few requests are a few warps')
                if (w < warp) before += scan[w];
                all += scan[w];
            }
            const int64_t in = static_cast<int64_t>(blockIdx.x) - (before + s - x);
            if (in >= 0 && in < x) {
                item[0] = r_; item[1] = f_; item[2] = n_; item[3] = kv_;
                item_at = static_cast<int>(in);
            }
            carry += all;
            __syncthreads();
        }
        return carry;
    };
    __syncthreads();
    const int64_t items = over_requests([&](int n_, int) { return static_cast<int64_t>(items_of(n_)) * c.heads; });
    int parts = 1, mine = 0, tile = 0, h = 0;                   // parts of the item, this one, row tile, kv head
    const bool split = 2 * items <= pl.sms && items > 0;
    if (split) {
        auto steps_of = [&](int n_, int kv_, int per) {         // per > 0: parts of that many steps instead
            int64_t total = 0;
            int x[4];
            for (int i = 0; i < items_of(n_); ++i) {
                const int st = max(range_of(n_, kv_, i, x[0], x[1], x[2], x[3]), 1);
                total += per > 0 ? (st + per - 1) / per : st;
            }
            return total * c.heads;
        };
        // The rows kernel's requests want SMs at the same time: a step takes an SM as long as
        // about six of its units (64 keys, 16 rows).
        auto units_of = [&](int n_, int kv_) {
            if (!rows_take(pl, n_, G)) return int64_t(0);
            int f0, s0, f1, s1;
            tile_range<TREE>(a, n_, kv_, 0, n_ - 1, f0, f1, s0, s1);
            return static_cast<int64_t>((max(s1 - f0, 0) >> 6) + 1) * ((n_ * G + 15) >> 4) * c.heads;
        };
        const int64_t steps_all = over_requests([&](int n_, int kv_) { return steps_of(n_, kv_, 0); });
        const int64_t units_all = over_requests(units_of);
        const int64_t share = pl.sms * 6 * steps_all / (6 * steps_all + units_all);
        const int64_t room = max(share - items, int64_t(1));
        int per = max(MIN_STEPS, static_cast<int>(min((steps_all + room - 1) / room, static_cast<int64_t>(INT_MAX / 2))));
        if constexpr (TREE) {
            // That leaves SMs idle where a few parts a little shorter would fit: the shortest of some lengths that does.
            // (4 contexts of 30k-60k: 32 items, 128 parts of 93 steps by the rule above)
            for (int k = 0, fine = max(MIN_STEPS, static_cast<int>((steps_all + share - 1) / max(share, int64_t(1)))); k < 8 && fine < per; ++k, fine += fine / 16 + 1)
                if (over_requests([&](int n_, int kv_) { return steps_of(n_, kv_, fine); }) <= share) per = fine;
        }
        if (tid == 0) item[0] = -1;
        __syncthreads();
        over_requests([&](int n_, int kv_) { return steps_of(n_, kv_, per); });
        if (item[0] >= 0) {
            int x[4];
            mine = item_at;
            for (tile = items_of(item[2]) - 1;; --tile) {
                parts = (max(range_of(item[2], item[3], tile, x[0], x[1], x[2], x[3]), 1) + per - 1) / per;
                if (mine < parts * c.heads || tile == 0) break;
                mine -= parts * c.heads;
            }
            h = mine / parts;
            mine -= h * parts;
        }
    } else if (item[0] >= 0) {
        tile = items_of(item[2]) - 1 - item_at / c.heads;
        h = item_at % c.heads;
    }
    const int r = item[0], first = item[1], n = item[2], kv = item[3];
    const int row0 = tile * ROWS, rows = min(ROWS, n * G - row0);
    if (tid == 0 && blockIdx.x < ATTN_TILE_CTAS)
        pl.share[blockIdx.x] = TileShare{r >= 0 && mine == 0 ? parts : 0, rows, row0, first, h, split, {0, 0}};
    if (r < 0) return;
    int key0, tstop, all_from, all_stop;
    int steps = range_of(n, kv, tile, key0, tstop, all_from, all_stop);
    if (parts > 1) {
        const int s0 = static_cast<int>(static_cast<int64_t>(mine) * steps / parts),
                  s1 = static_cast<int>(static_cast<int64_t>(mine + 1) * steps / parts);
        key0 += s0 * KEYS;
        steps = s1 - s0;
    }

    if (tid == 0) {
        mbar_init(&bars[B_Q], SOFT);
        for (int i = 0; i < 2; ++i) {
            mbar_init(&bars[B_K_FULL + i], CONV);
            mbar_init(&bars[B_K_EMPTY + i], 1);
            mbar_init(&bars[B_V_FULL + i], CONV);
            mbar_init(&bars[B_V_EMPTY + i], 1);
            mbar_init(&bars[B_S + i], 1);
            mbar_init(&bars[B_P + i], SOFT / 32 / MT);
            mbar_init(&bars[B_O + i], 1);
            mbar_init(&bars[B_FREE + i], SOFT / 32 / MT);
        }
        for (int i = 0; i < INFO; ++i) mbar_init(&bars[B_INFO + i], CONV / 32);
        mbar_init(&bars[B_DRAINED], 1);
        fence_mbar_init();
    }
    if (warp == (SOFT + CONV) / 32) {
        tc::tmem_alloc(&tmem_holder, 512);
        tc::tmem_relinquish();
    }
    tc::fence_before();
    __syncthreads();
    tc::fence_after();
    const uint32_t tmem = tmem_holder;

    if (warp < SOFT / 32) {
        // ------------------------------------------------------------ softmax
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(W::REGS_SOFT));
        const int mt = (warp >> 2) / SPLIT, part = (warp >> 2) % SPLIT;      // row tile, part of the keys
        const int lrow = (warp & 3) * 32 + lane;            // row of the tile, lane of tensor memory
        const int row = 128 * mt + lrow;                    // of the item
        // fp32: the warps that share these 32 rows meet here (the same number of times each, come what may)
        auto meet = [&]() { asm volatile("bar.sync %0, %1;" ::"r"(1 + 4 * mt + (warp & 3)), "n"(32 * SPLIT) : "memory"); };
        const RowMap map(row0, G);
        int my_tok, my_head;
        map.of(row, my_tok, my_head);
        const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
        {
            // The rows as operand, each scaled to [2^8, 2^9) by a power of two: four lanes a
            // row, each with every fourth chunk of 8 values; all of a warp's loads in flight.
            constexpr int NCH = D / 32, PASS = ROWS / (SOFT / 32) / 8;
            const int quad = lane & 3, w0 = warp * (ROWS / (SOFT / 32)) + (lane >> 2);
            Raw8<T> v[PASS][NCH];                              // rows past the last are the last
#pragma unroll
            for (int b = 0; b < PASS; ++b) {
                int tk, hd;
                map.of(min(w0 + 8 * b, rows - 1), tk, hd);
                const T* src = static_cast<const T*>(a.q) + static_cast<int64_t>(first + tk) * a.q_stride + (h * G + hd) * D + quad * 8;
#pragma unroll
                for (int i = 0; i < NCH; ++i) v[b][i].load(src + 32 * i);
            }
            const float lscale = fabsf(a.scale) * 1.4426950408889634f;
#pragma unroll
            for (int b = 0; b < PASS; ++b) {
                const int rr = w0 + 8 * b;
                float x[NCH][8];
                uint32_t top = 0;
#pragma unroll
                for (int i = 0; i < NCH; ++i) {
                    v[b][i].values(x[i]);
#pragma unroll
                    for (int k = 0; k < 8; ++k) top = max(top, __float_as_uint(fabsf(x[i][k])));
                }
                top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
                top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
                float mul, back;
                row_scale(rr < rows ? top : 0, mul, back);
                if (quad == 0) rowf[rr] = back * lscale;
                if (a.scale < 0.0f) mul = -mul;
                if (rr >= rows) mul = 0.0f;
                uint8_t* dst = smem + W::OFF_Q + (rr >> 7) * W::QB;
#pragma unroll
                for (int i = 0; i < NCH; ++i) {
                    uint32_t hi[4], lo[4];
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const float y0 = x[i][2 * k] * mul, y1 = x[i][2 * k + 1] * mul;
                        const __half2 hh = __floats2half2_rn(y0, y1);
                        hi[k] = *reinterpret_cast<const uint32_t*>(&hh);
                        if constexpr (F32) {
                            const float2 f = __half22float2(hh);
                            const __half2 hl = __floats2half2_rn(y0 - f.x, y1 - f.y);
                            lo[k] = *reinterpret_cast<const uint32_t*>(&hl);
                        }
                    }
                    const int off = tc::tile_off_sw128(rr & 127, 8 * (quad + 4 * i), 128);
                    *reinterpret_cast<uint4*>(dst + off) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
                    if constexpr (F32) *reinterpret_cast<uint4*>(dst + W::QB + off) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
                }
            }
            fence_proxy_async_smem();
            tc::mbar_arrive(&bars[B_Q]);
        }
        if (!mbar_wait_bounded(&bars[B_Q], 0, WAIT_LIMIT_NS)) abort_flag.set(1);     // rowf is every warp's work
        const float rf = rowf[row];
        int from = 0, stop = 0;
        uint64_t mask = 0;
        if (row < rows) token_range<TREE>(a, n, kv, my_tok, from, stop);
        if (TREE && row < rows) mask = tree_mask(a, first, n, my_tok);
        const uint32_t s_col0 = tmem + lanes + W::S0 + KT * part;
        const uint32_t p_col = tmem + lanes + W::SP + 64 * mt + KT / 2 * part;         // 16-bit types
        const uint32_t p3_col = tmem + lanes + W::SP + KT / 2 * part;
        const uint32_t o_col = tmem + lanes + (mt == 0 ? W::O0 : W::O1) + OC * part;
        constexpr int CHUNKS = KT / 32;
        float M = -INFINITY, l = 0.0f;
        // The results before the last FLUSH steps, and their reference. fp32: a thread's first 32 columns, the others in tensor
        // memory; 16-bit types, which come here rarely and have no column left: in local memory.
        float total[!W::FLUSH ? 1 : F32 ? 32 : OC], total_M = -INFINITY;
        const uint32_t t_col = tmem + lanes + W::T0 + 32 * part;
        bool ok = true;
        // After a wait that ran out (ok false) the loop goes on without waiting: the meetings stay paired.
        auto wait = [&](int bar, int parity) {
            if (!ok || !__all_sync(0xffffffffu, mbar_try_wait(&bars[bar], parity))) {
                if (ok && !mbar_wait_bounded(&bars[bar], parity, WAIT_LIMIT_NS)) ok = false;
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) abort_flag.set(1);
            }
            tc::fence_after();
        };
        // The last steps' results to the totals, before step j, whose products begin them anew.
        auto factor = [&]() { return total_M == M ? 1.0f : exp2_approx(total_M - M); };      // 0 from -inf
        auto flush = [&](const int j) {
            wait(B_O + mt, (j - 1) & 1);
            const float f = factor();
            auto add = [&](float was, float now) { return (j > W::FLUSH ? was * f : 0.0f) + now; };
            if constexpr (F32) {
#pragma unroll
                for (int ch = 0; ch < 2; ++ch) {
                    uint32_t big[16], small[16];
                    tc::ld16(o_col + 16 * ch, big);
                    tc::ld16(o_col + 16 * ch + (W::O1 - W::O0), small);
                    tc::wait_ld();
#pragma unroll
                    for (int i = 0; i < 16; ++i)
                        total[16 * ch + i] = add(total[16 * ch + i], __uint_as_float(big[i]) + __uint_as_float(small[i]));
                }
#pragma unroll 1
                for (int ch = 2; ch < OC / 16; ++ch) {
                    uint32_t big[16], small[16], rest[16];
                    tc::ld16(o_col + 16 * ch, big);
                    tc::ld16(o_col + 16 * ch + (W::O1 - W::O0), small);
                    tc::ld16(t_col + 16 * (ch - 2), rest);
                    tc::wait_ld();
#pragma unroll
                    for (int i = 0; i < 16; ++i)
                        rest[i] = __float_as_uint(add(__uint_as_float(rest[i]), __uint_as_float(big[i]) + __uint_as_float(small[i])));
                    tc::st16(t_col + 16 * (ch - 2), rest);
                }
            } else {
#pragma unroll 1
                for (int col = 0; col < OC; col += 16) {
                    uint32_t x[16];
                    tc::ld16(o_col + col, x);
                    tc::wait_ld();
#pragma unroll
                    for (int i = 0; i < 16; ++i) total[col + i] = add(total[col + i], __uint_as_float(x[i]));
                }
            }
            total_M = M;
        };
        // A step; whole: every row sees all its keys.
        auto step = [&](const int j, auto whole_) {
            constexpr bool whole = decltype(whole_)::value;
            // The blocks' factors and offsets are there before the scores, and stay in registers: a
            // 16-byte read of one address by all lanes occupies shared memory for four cycles.
            wait(B_INFO + j % INFO, (j / INFO) & 1);
            float fk[KT / 16], lv[KT / 16];
            auto blocks = [&](int what, float (&x)[KT / 16]) {
#pragma unroll
                for (int b = 0; b < KT / 16; b += 4)
                    *reinterpret_cast<float4*>(x + b) = *reinterpret_cast<const float4*>(&info[j % INFO][what][KT / 16 * part + b]);
            };
            blocks(0, fk);
            blocks(1, lv);
#pragma unroll
            for (int b = 0; b < KT / 16; ++b) fk[b] *= rf;
            if constexpr (SBUF == 2) wait(B_S + (j & 1), (j >> 1) & 1);
            else wait(B_S + mt, j & 1);
            const uint32_t s_col = s_col0 + (SBUF == 2 ? (j & 1) * (W::S1 - W::S0) : 0);
            const int k0 = key0 + j * KEYS + KT * part;
            // The scores are read once and stay in registers: tensor memory is what a step would wait for.
            uint32_t v[CHUNKS][32];
#pragma unroll
            for (int ch = 0; ch < CHUNKS; ++ch) tc::ld32(s_col + 32 * ch, v[ch]);
            tc::wait_ld();
            if constexpr (MT == 2) {                        // the other tile's scores may come
                tc::fence_before();
                __syncwarp();
                if (lane == 0) tc::mbar_arrive(&bars[B_FREE + mt]);
            }
            if constexpr (!whole) {
                // x itself, hidden keys at -inf: factor 1 and no offset from here on
#pragma unroll
                for (int ch = 0; ch < CHUNKS; ++ch)
#pragma unroll
                    for (int b = 0; b < 2; ++b) {
                        const int key = k0 + 32 * ch + 16 * b;
                        uint32_t bits = 0;                  // of the mask, key by key
                        if constexpr (TREE) {
                            const int at = key - (kv - n);
                            if (at > -16 && at < CQ_TREE_MAX) bits = static_cast<uint32_t>(at >= 0 ? mask >> at : mask << -at);
                        }
#pragma unroll
                        for (int i = 0; i < 16; ++i) {
                            const float x = fmaf(__uint_as_float(v[ch][16 * b + i]), fk[2 * ch + b], lv[2 * ch + b]);
                            v[ch][16 * b + i] = __float_as_uint((key + i >= from && key + i < stop) || (TREE && (bits >> i & 1) != 0) ? x : -INFINITY);
                        }
                    }
            }
            // the largest x: a block's from its largest score, since its factor is not negative
            float top = -INFINITY;
#pragma unroll
            for (int ch = 0; ch < CHUNKS; ++ch)
#pragma unroll
                for (int b = 0; b < 2; ++b) {
                    float m = __uint_as_float(v[ch][16 * b]);
#pragma unroll
                    for (int i = 1; i < 15; i += 2) m = max3(m, __uint_as_float(v[ch][16 * b + i]), __uint_as_float(v[ch][16 * b + i + 1]));
                    m = fmaxf(m, __uint_as_float(v[ch][16 * b + 15]));
                    top = fmaxf(top, whole ? fmaf(m, fk[2 * ch + b], lv[2 * ch + b]) : m);
                }
            // the row's other parts (a slot is written again two steps on, after the next meeting)
            if constexpr (SPLIT > 1) {
                exch[j & 1][part][row] = top;
                meet();
#pragma unroll
                for (int i = 0; i < SPLIT; ++i) top = fmaxf(top, exch[j & 1][i][row]);
            }
            const bool raise = top > M + RAISE;
            bool o_known = j == 0;
            if (__any_sync(0xffffffffu, raise)) {
                const float old = M;
                if (raise) M = top;
                const float f = raise ? exp2_approx(old - M) : 1.0f;             // 0 from -inf
                l *= f;
                if (j > 0) {
                    wait(B_O + mt, (j - 1) & 1);
                    o_known = true;
#pragma unroll 1
                    for (int ch = 0; ch < (F32 ? 2 : 1) * (OC / 16); ++ch) {     // its share of the row's columns
                        uint32_t orr[16];
                        const uint32_t at = o_col + (ch % (OC / 16)) * 16 + (ch < OC / 16 ? 0 : W::O1 - W::O0);
                        tc::ld16(at, orr);
                        tc::wait_ld();
#pragma unroll
                        for (int i = 0; i < 16; ++i) orr[i] = __float_as_uint(__uint_as_float(orr[i]) * f);
                        tc::st16(at, orr);
                    }
                }
            }
            // P (fp32: its third part) has columns of its own, the product of the step before has to be done with them
            if (!o_known) wait(B_O + mt, (j - 1) & 1);
            const float base = M == -INFINITY ? 0.0f : M - OFF;
            // (fp32: each part's P overlays its own scores, which are in registers)
            // A chunk's exponentials all come before their sums and conversions, and no chunk's P is in
            // another's registers: a pair at a time takes a warp half as long again.
            uint32_t pr[CHUNKS][16];
            float weight[KT / 16];
            blocks(2, weight);
#pragma unroll
            for (int ch = 0; ch < CHUNKS; ++ch) {
#pragma unroll
                for (int b = 0; b < 2; ++b) {
                    const float f = whole ? fk[2 * ch + b] : 1.0f, lb = (whole ? lv[2 * ch + b] : 0.0f) - base;
                    const uint64_t f2 = tc::pk(f, f), lb2 = tc::pk(lb, lb);
#pragma unroll
                    for (int i = 0; i < 16; i += 2) {
                        uint32_t &v0 = v[ch][16 * b + i], &v1 = v[ch][16 * b + i + 1];
                        float x0, x1;
                        tc::upk(tc::fma2(tc::pk(__uint_as_float(v0), __uint_as_float(v1)), f2, lb2), x0, x1);
                        v0 = __float_as_uint(exp2_approx(x0));
                        v1 = __float_as_uint(exp2_approx(x1));
                    }
                }
#pragma unroll
                for (int b = 0; b < 2; ++b) {
                    uint64_t sums[2] = {0, 0};
#pragma unroll
                    for (int i = 0; i < 16; i += 2) {
                        const float p0 = __uint_as_float(v[ch][16 * b + i]), p1 = __uint_as_float(v[ch][16 * b + i + 1]);
                        sums[(i >> 1) & 1] = tc::add2(sums[(i >> 1) & 1], tc::pk(p0, p1));
                        if constexpr (W::PARTS == 1) {       // 11 bits (two tiles: the columns of a second part are in use)
                            const __half2 x = __floats2half2_rn(p0, p1);
                            pr[ch][8 * b + i / 2] = *reinterpret_cast<const uint32_t*>(&x);
                        }
                    }
                    float s0, s1;
                    tc::upk(tc::add2(sums[0], sums[1]), s0, s1);
                    l = fmaf(s0 + s1, weight[2 * ch + b], l);        // (a weight is finite, or the sum is not)
                }
                if constexpr (W::PAIR) {
                    // The first part is cut off to 11 bits, which takes no conversion back; what is left is exact.
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        uint32_t &v0 = v[ch][2 * i], &v1 = v[ch][2 * i + 1];
                        const float h0 = __uint_as_float(v0 & 0xffffe000u), h1 = __uint_as_float(v1 & 0xffffe000u);
                        const __half2 x = __floats2half2_rn(h0, h1);
                        pr[ch][i] = *reinterpret_cast<const uint32_t*>(&x);
                        float l0, l1;
                        tc::upk(tc::fma2(tc::pk(h0, h1), tc::pk(-1.0f, -1.0f), tc::pk(__uint_as_float(v0), __uint_as_float(v1))), l0, l1);
                        v0 = __float_as_uint(l0);
                        v1 = __float_as_uint(l1);
                    }
                    tc::st16(p_col + 16 * ch, pr[ch]);
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        const __half2 x = __floats2half2_rn(__uint_as_float(v[ch][2 * i]), __uint_as_float(v[ch][2 * i + 1]));
                        pr[ch][i] = *reinterpret_cast<const uint32_t*>(&x);
                    }
                    tc::st16(p_col + (W::P2 - W::SP) + 16 * ch, pr[ch]);
                } else if constexpr (F32) {
#pragma unroll
                    for (int p3 = 0; p3 < 3; ++p3) {
#pragma unroll
                        for (int i = 0; i < 16; ++i) {
                            const float p0 = __uint_as_float(v[ch][2 * i]), p1 = __uint_as_float(v[ch][2 * i + 1]);
                            const __nv_bfloat162 x = __floats2bfloat162_rn(p0, p1);
                            pr[ch][i] = *reinterpret_cast<const uint32_t*>(&x);
                            v[ch][2 * i] = __float_as_uint(p0 - __uint_as_float(pr[ch][i] << 16));
                            v[ch][2 * i + 1] = __float_as_uint(p1 - __uint_as_float(pr[ch][i] & 0xffff0000u));
                        }
                        tc::st16(p3 < 2 ? s_col + KT / 2 * p3 + 16 * ch : p3_col + 16 * ch, pr[ch]);
                    }
                } else {
                    tc::st16(p_col + 16 * ch, pr[ch]);
                }
            }
            tc::wait_st();
            tc::fence_before();
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(&bars[B_P + mt]);
        };
        // (One tile: a loop in a loop, 128 us for 130 at binary16's 64 contexts. Elsewhere that spills: 197 us for 193, bfloat16,
        // 4 contexts of 30k-60k.)
        if constexpr (NARROW) {
            for (int j = 0; j < steps;) {
                if (j > 0) flush(j);
                for (const int until = min(j + W::FLUSH, steps); j < until; ++j) {
                    const int k0 = key0 + j * KEYS + KT * part;
                    if (k0 >= all_from && k0 <= all_stop - KT) step(j, std::true_type{});
                    else step(j, std::false_type{});
                }
            }
        } else {
            for (int j = 0; j < steps; ++j) {
                const int k0 = key0 + j * KEYS + KT * part;
                if constexpr (W::FLUSH > 0) {
                    if (j > 0 && j % W::FLUSH == 0) flush(j);
                }
                if (k0 >= all_from && k0 <= all_stop - KT) step(j, std::true_type{});
                else step(j, std::false_type{});
            }
        }
        // ---- the rows
        if (steps > 0) wait(B_O + mt, (steps - 1) & 1);
        if constexpr (W::FLUSH > 0 && !F32) {               // the totals to the results (fp32: as the rows are written)
            if (steps > W::FLUSH) {
                const float f = factor();
#pragma unroll 1
                for (int col = 0; col < OC; col += 16) {
                    uint32_t x[16];
                    tc::ld16(o_col + col, x);
                    tc::wait_ld();
#pragma unroll
                    for (int i = 0; i < 16; ++i) x[i] = __float_as_uint(fmaf(total[col + i], f, __uint_as_float(x[i])));
                    tc::st16(o_col + col, x);
                }
                tc::wait_st();
            }
        }
        if constexpr (SPLIT > 1) {
            exch[steps & 1][part][row] = l;
            meet();
            l = 0.0f;
#pragma unroll
            for (int i = 0; i < SPLIT; ++i) l += exch[steps & 1][i][row];
        }
        const float total_f = factor();
        auto load_o = [&](int col, uint32_t (&orr)[32]) {       // of the thread's columns
            const uint32_t at = o_col + col;
            if (steps == 0) {
#pragma unroll
                for (int i = 0; i < 32; ++i) orr[i] = 0;
                return;
            }
            tc::ld32(at, orr);
            tc::wait_ld();
            if constexpr (F32) {
                uint32_t os[32];
                tc::ld32(at + (W::O1 - W::O0), os);
                tc::wait_ld();
#pragma unroll
                for (int i = 0; i < 32; ++i) orr[i] = __float_as_uint(__uint_as_float(orr[i]) + __uint_as_float(os[i]));
                if constexpr (W::FLUSH > 0) {
                    if (steps > W::FLUSH) {
                        if (col > 0) {
                            tc::ld32(t_col, os);
                            tc::wait_ld();
                        }
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            orr[i] = __float_as_uint(fmaf(col > 0 ? __uint_as_float(os[i]) : total[i], total_f, __uint_as_float(orr[i])));
                    }
                }
            }
        };
        if (ok && parts > 1) {
            // Sums as they are, fp32, to the workspace: half the columns at a time through the query operand's place.
            constexpr int PC = D / 2, NC = PC / 4, SW = (NC < 8 ? NC : 8) - 1, ROWF = D + 4;
            float* mine_ = reinterpret_cast<float*>(smem + W::OFF_Q + warp * (32 * PC * 4));
            float* dst = pl.tile_part + static_cast<int64_t>(blockIdx.x) * (256 * ROWF) + (128 * mt + (warp & 3) * 32) * ROWF;
#pragma unroll
            for (int ps = 0; ps < OC / PC; ++ps) {
#pragma unroll
                for (int ch = 0; ch < PC / 32; ++ch) {
                    uint32_t orr[32];
                    load_o(ps * PC + 32 * ch, orr);
#pragma unroll
                    for (int i = 0; i < 32; i += 4)
                        *reinterpret_cast<uint4*>(mine_ + lane * PC + (((32 * ch + i) / 4) ^ (lane & SW)) * 4) =
                            make_uint4(orr[i], orr[i + 1], orr[i + 2], orr[i + 3]);
                }
                __syncwarp();
#pragma unroll 4
                for (int x = lane; x < 32 * NC; x += 32) {
                    const int lr = x / NC, cc = x % NC;
                    if (128 * mt + (warp & 3) * 32 + lr < rows)
                        *reinterpret_cast<uint4*>(dst + lr * ROWF + OC * part + ps * PC + cc * 4) =
                            *reinterpret_cast<const uint4*>(mine_ + lr * PC + (cc ^ (lr & SW)) * 4);
                }
                __syncwarp();
            }
            if (row < rows && part == 0) { dst[lane * ROWF + D] = M; dst[lane * ROWF + D + 1] = l; }
        } else if (ok) {
            // A row a thread in tensor memory, but a row a few lanes in global memory: the
            // warp's rows change hands in the query operand's place, which no MMA reads any more.
            constexpr int CH = 16 / sizeof(T), NC = OC / CH;                 // values of a 16-byte chunk, chunks of the warp's columns
            constexpr int SW = (NC < 8 ? NC : 8) - 1;
            uint8_t* mine = smem + W::OFF_Q + warp * (32 * OC * sizeof(T));
            float inv, down;
            row_factors(l, inv, down);
            static_assert(OC % 32 == 0, "columns in chunks of 32");
#pragma unroll
            for (int ch = 0; ch < OC / 32; ++ch) {
                uint32_t orr[32];
                load_o(32 * ch, orr);
#pragma unroll
                for (int i = 0; i < 32; i += CH) {
                    T* dst = reinterpret_cast<T*>(mine + lane * (OC * sizeof(T)) + (((32 * ch + i) / CH) ^ (lane & SW)) * 16);
#pragma unroll
                    for (int k = 0; k < CH; k += 4)
                        store4(dst + k, make_float4(__uint_as_float(orr[i + k]) * inv * down, __uint_as_float(orr[i + k + 1]) * inv * down,
                                                    __uint_as_float(orr[i + k + 2]) * inv * down, __uint_as_float(orr[i + k + 3]) * inv * down));
                }
            }
            if (a.lse != nullptr && row < rows && part == 0)
                a.lse[static_cast<int64_t>(first + my_tok) * a.heads + h * G + my_head] =
                    l == 0.0f ? -INFINITY : 0.6931471805599453f * (M - OFF + SUM_LOG + log2f(l));
            __syncwarp();
            const int cc = lane % NC;
#pragma unroll 4
            for (int lr = lane / NC; lr < 32; lr += 32 / NC) {
                const int rr = 128 * mt + (warp & 3) * 32 + lr;
                int tk, hd;
                map.of(rr, tk, hd);
                const uint4 x = *reinterpret_cast<const uint4*>(mine + lr * (OC * sizeof(T)) + ((cc ^ (lr & SW)) * 16));
                if (rr < rows)
                    *reinterpret_cast<uint4*>(static_cast<T*>(a.out) + static_cast<int64_t>(first + tk) * a.out_stride +
                                              (h * G + hd) * D + OC * part + cc * CH) = x;
            }
        } else if (lane == 0) {
            atomicOr(a.status, CQ_DEV_WAIT_TIMEOUT);
        }
    } else if (warp < (SOFT + CONV) / 32) {
        // ---------------------------------------------------------- converters
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(W::REGS_CONV));
        // A load takes 16 dimensions a lane of 8 keys. Eight lanes (a phase of a 16-byte
        // access) hold four pieces of an even key and four of the odd one after it; at D = 128
        // the other half of the row: the bytes then come from different banks of the lines,
        // and the chunks go to different banks of the swizzled rows (8-way conflicts on both
        // sides otherwise).
        const int cw = warp - SOFT / 32;
        const int odd = (lane >> 2) & 1, ck = 2 * (lane >> 3) + odd;
        auto piece = [&](int i) { return (lane & 3) + (D == 128 ? 4 * (odd ^ i) : 0); };
        constexpr int NL = D / 64;                          // loads a lane and 8 keys
        constexpr int KW = W::KW, NBK = W::NBK;
        constexpr int GROUPS = KW / 8;                      // groups of 8 keys of a warp: keys KW cw ..
        const int32_t* table = a.table + static_cast<int64_t>(r) * a.max_blocks;
        const int64_t head_off = static_cast<int64_t>(h) * c.page_size * D;
        // The warp's blocks of 16 keys of a step, two (one where there are eight warps): a lane each looks them up. A step's
        // table entries are fetched two steps ahead, its scales and bytes one: no lookup
        // is waited for in the loop, and a step's loads run behind the one before's stores.
        auto block_at = [&](int j) { return key0 + j * KEYS + KW * cw + 16 * lane; };
        auto has_keys = [&](int j) { return lane < NBK && j < steps && block_at(j) < tstop; };
        auto entry = [&](int j) { return has_keys(j) ? table[block_at(j) >> c.page_shift] : -1; };
        auto checked = [&](int e, int j) {
            if (e >= 0 && e < c.num_pages) return e;
            if (has_keys(j)) atomicOr(a.status, CQ_DEV_KV_PAGE);
            return -1;
        };
        int64_t at[NBK];
        auto place = [&](int page, int j) {
            const int k = block_at(j);
            const int64_t mine = page >= 0 ? page * c.page_stride + head_off + static_cast<int64_t>(k & (c.page_size - 1)) * D : -1;
#pragma unroll
            for (int b = 0; b < NBK; ++b) at[b] = __shfl_sync(0xffffffffu, mine, b);
        };
        float p_ks = 0.0f, p_vs = 0.0f;
        auto scales = [&](int page) {
            if (page < 0) return;
            p_ks = c.k_scale[page * c.scale_stride + h];
            p_vs = c.v_scale[page * c.scale_stride + h];
        };
        // (NARROW: bytes by asynchronous copies instead, see below)
        uint4 kr[GROUPS][NL] = {}, vr[GROUPS][NL] = {};
        auto load = [&](const int8_t* src, uint4 (&x)[GROUPS][NL]) {
#pragma unroll
            for (int g = 0; g < GROUPS; ++g)
#pragma unroll
                for (int i = 0; i < NL; ++i) {
                    if (at[g >> 1] >= 0)                    // else what it held: integers that meet a P of zero
                        x[g][i] = ldg_stream16(src + at[g >> 1] + (8 * (g & 1) + ck) * D + 16 * piece(i));
                }
        };
        int put[NL][2];                                     // a piece's places in the operand; 8 keys on are 8 rows
#pragma unroll
        for (int i = 0; i < NL; ++i) {
            put[i][0] = tc::tile_off_sw128(KW * cw + ck, 16 * piece(i), KEYS);
            put[i][1] = tc::tile_off_sw128(KW * cw + ck, 16 * piece(i) + 8, KEYS);
        }
        auto store = [&](uint8_t* dst, const uint4 (&x)[GROUPS][NL], bool bf) {      // bf: bfloat16
#pragma unroll
            for (int g = 0; g < GROUPS; ++g)
#pragma unroll
                for (int i = 0; i < NL; ++i) {
                    const uint32_t w[4] = {x[g][i].x, x[g][i].y, x[g][i].z, x[g][i].w};
                    uint32_t o[8];
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        if (bf) s8x4_bf16(w[k], o[2 * k], o[2 * k + 1]);
                        else tc::s8x4_half(w[k], o[2 * k], o[2 * k + 1]);
                    }
                    *reinterpret_cast<uint4*>(dst + put[i][0] + 8 * g * 128) = make_uint4(o[0], o[1], o[2], o[3]);
                    *reinterpret_cast<uint4*>(dst + put[i][1] + 8 * g * 128) = make_uint4(o[4], o[5], o[6], o[7]);
                }
        };
        if constexpr (NARROW) {
            // A step is shorter than a load takes, and loads into registers are waited for together: whoever takes the keys
            // waits for the values' loads behind them as well. The bytes come by asynchronous copies instead, three halves
            // of a step in front; a thread takes what it has copied itself. The lookups of sixteen steps are made at once,
            // a lane a step: one step's alone are 900 cycles of one instruction behind another.
            static_assert(!NARROW || NBK == 1, "one block a warp and step");
            constexpr int BATCH = 16;
            uint8_t* const raw = smem + W::OFF_RAW + cw * (GROUPS * NL * 512) + lane * 16;
            auto copy = [&](const int8_t* src, int64_t from, int slot) {
                if (from >= 0) {                            // else what lies there: integers that meet a P of zero
#pragma unroll
                    for (int g = 0; g < GROUPS; ++g)
#pragma unroll
                        for (int i = 0; i < NL; ++i)
                            cp_async16(raw + slot * W::SLOT + (g * NL + i) * 512, src + from + (8 * g + ck) * D + 16 * piece(i));
                }
                cp_async_commit();
            };
            auto take = [&](uint4 (&x)[GROUPS][NL], int slot) {
                cp_async_wait<2>();
#pragma unroll
                for (int g = 0; g < GROUPS; ++g)
#pragma unroll
                    for (int i = 0; i < NL; ++i) x[g][i] = *reinterpret_cast<const uint4*>(raw + slot * W::SLOT + (g * NL + i) * 512);
            };
            // the lane's step of a batch that begins at step j0
            auto key_of = [&](int j0) { return key0 + (j0 + lane) * KEYS + KW * cw; };
            auto has = [&](int j0) { return lane < BATCH && j0 + lane < steps && key_of(j0) < tstop; };
            auto entry_of = [&](int j0) { return has(j0) ? table[key_of(j0) >> c.page_shift] : -1; };
            int n_entry = -1, n_page = -1;
            int64_t b_at = -1, n_at = -1;                   // the blocks' bytes, this batch's and the next one's
            float n_ks = 0.0f, n_vs = 0.0f;
            float3 b_in = make_float3(0.0f, -INFINITY, 1.0f);
            auto look = [&](int j0) {                       // entries to places; the scales on their way
                n_page = n_entry >= 0 && n_entry < c.num_pages ? n_entry : -1;
                if (n_page < 0 && has(j0)) atomicOr(a.status, CQ_DEV_KV_PAGE);
                n_at = -1;
                if (n_page >= 0) {
                    n_at = n_page * c.page_stride + head_off + static_cast<int64_t>(key_of(j0) & (c.page_size - 1)) * D;
                    n_ks = c.k_scale[n_page * c.scale_stride + h];
                    n_vs = c.v_scale[n_page * c.scale_stride + h];
                }
            };
            auto open = [&]() {                             // the next batch is this one
                b_at = n_at;
                b_in = make_float3(0.0f, -INFINITY, 1.0f);
                if (n_page >= 0) {
                    b_in.x = n_ks;
                    value_factors<F32>(n_vs, b_in.y, b_in.z);
                }
            };
            n_entry = entry_of(0);
            look(0);
            copy(c.k, __shfl_sync(0xffffffffu, n_at, 0), 0);
            copy(c.v, __shfl_sync(0xffffffffu, n_at, 0), 1);
            copy(c.k, __shfl_sync(0xffffffffu, n_at, 1), 2);
            int slot = 0;
            for (int j = 0; j < steps; ++j) {
                const int st = j & 1, p = j % BATCH;
                if (j % 8 == 0 && __any_sync(0xffffffffu, abort_flag.get())) break;
                if (p == 0) open();
                if (p == 2) n_entry = entry_of(j - p + BATCH);
                if (p == 7) look(j - p + BATCH);
                // the step that used this entry before is past its softmax: the scores of two steps ago were its next
                take(kr, slot);
                // (the whole warp leaves or none of it: it shuffles)
                if (!__all_sync(0xffffffffu, tc::wait_or_abort_sleep(&bars[B_K_EMPTY + st], ((j >> 1) & 1) ^ 1, abort_flag, a.status))) break;
                if (lane == p) {
                    info[j % INFO][0][cw] = b_in.x;
                    info[j % INFO][1][cw] = b_in.y;
                    info[j % INFO][2][cw] = b_in.z;
                    tc::mbar_arrive(&bars[B_INFO + j % INFO]);
                }
                store(smem + W::OFF_K + st * W::KB, kr, false);
                fence_proxy_async_smem();
                tc::mbar_arrive(&bars[B_K_FULL + st]);
                copy(c.v, __shfl_sync(0xffffffffu, p + 1 < BATCH ? b_at : n_at, (j + 1) % BATCH), slot);
                slot = slot == 2 ? 0 : slot + 1;
                take(vr, slot);
                if (!__all_sync(0xffffffffu, tc::wait_or_abort_sleep(&bars[B_V_EMPTY + st], ((j >> 1) & 1) ^ 1, abort_flag, a.status))) break;
                store(smem + W::OFF_V + st * W::KB, vr, F32);
                fence_proxy_async_smem();
                tc::mbar_arrive(&bars[B_V_FULL + st]);
                copy(c.k, __shfl_sync(0xffffffffu, p + 2 < BATCH ? b_at : n_at, (j + 2) % BATCH), slot);
                slot = slot == 2 ? 0 : slot + 1;
            }
            cp_async_wait_all();                            // none is in flight when the CTA leaves
        } else {
            int page = checked(entry(0), 0), ahead = entry(1);
            scales(page);
            place(page, 0);
            load(c.k, kr);
            load(c.v, vr);
            for (int j = 0; j < steps; ++j) {
                const int st = j & 1;
                if (j % 8 == 0 && __any_sync(0xffffffffu, abort_flag.get())) break;
                // (the whole warp leaves or none of it: it shuffles)
                if (!__all_sync(0xffffffffu, tc::wait_or_abort_sleep(&bars[B_K_EMPTY + st], ((j >> 1) & 1) ^ 1, abort_flag, a.status))) break;
                store(smem + W::OFF_K + st * W::KB, kr, false);
                fence_proxy_async_smem();
                tc::mbar_arrive(&bars[B_K_FULL + st]);
                // What was looked up for this step and the next is taken before any load is issued: right
                // behind the values' loads, this waits for them, half a step.
                float3 in = make_float3(0.0f, -INFINITY, 1.0f);
                if (page >= 0) {
                    in.x = p_ks;
                    // (exact here for the 16-bit types too: 443 us for 437 at the 8192-token prompt)
                    value_factors<F32>(p_vs, in.y, in.z);
                }
                // the step that used this entry before is past its softmax: the scores of two steps ago were its next
                if (lane < NBK) {
                    info[j % INFO][0][NBK * cw + lane] = in.x;
                    info[j % INFO][1][NBK * cw + lane] = in.y;
                    info[j % INFO][2][NBK * cw + lane] = in.z;
                }
                __syncwarp();
                if (lane == 0) tc::mbar_arrive(&bars[B_INFO + j % INFO]);
                page = checked(ahead, j + 1);
                ahead = entry(j + 2);
                scales(page);
                place(page, j + 1);
                load(c.k, kr);
                if (!__all_sync(0xffffffffu, tc::wait_or_abort_sleep(&bars[B_V_EMPTY + st], ((j >> 1) & 1) ^ 1, abort_flag, a.status))) break;
                store(smem + W::OFF_V + st * W::KB, vr, F32);
                fence_proxy_async_smem();
                tc::mbar_arrive(&bars[B_V_FULL + st]);
                load(c.v, vr);
            }
        }
    } else {
        // --------------------------------------------------------- MMA issuer
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(W::REGS_MMA));
        if (warp == (SOFT + CONV) / 32 && steps > 0) {
        const uint32_t lead = tc::elect_one();
        const uint32_t q0 = smem_u32(smem + W::OFF_Q), k0 = smem_u32(smem + W::OFF_K), v0 = smem_u32(smem + W::OFF_V);
        constexpr uint32_t ID_S = tc::idesc_f16_f32(128, KEYS);
        constexpr uint32_t ID_O = tc::idesc_f16_f32(128, D) | tc::IDESC_B_MN | (F32 ? tc::IDESC_BF16 : 0u);
        // One warp issues all MMAs between busy ones, so an MMA is to cost it few
        // instructions: the warp runs as one, one lane issues, descriptors are a base and a constant. A k-step of 16 values adds 32
        // bytes inside a 128-byte row, 64 values on is the next block of rows; 16 keys of
        // values are 16 rows of 128 bytes.
        const uint64_t qd = tc::smem_desc_sw128(q0, 1024), kd = tc::smem_desc_sw128(k0, 1024),
                       vd = tc::smem_desc_sw128_mn(v0, KEYS * 128, 1024);
        auto scores = [&](int m, int st) {                  // one tile: m is the buffer
            const uint32_t d = tmem + (MT == 2 || m == 0 ? W::S0 : W::S1);
            const uint64_t bd = kd + st * (W::KB >> 4);
#pragma unroll
            for (int part = 0; part < (F32 ? 2 : 1); ++part) {
                const uint64_t ad = qd + (F32 ? 1 - part : MT == 2 ? m : 0) * (W::QB >> 4);      // fp32: the lower parts first, while the sums are small
#pragma unroll
                for (int k = 0; k < D / 16; ++k) {
                    const uint32_t off = ((k >> 2) * (128 * 128) + (k & 3) * 32) >> 4, off_k = ((k >> 2) * (KEYS * 128) + (k & 3) * 32) >> 4;
                    tc::mma_f16_lead(d, ad + off, bd + off_k, ID_S, part > 0 || k > 0, lead);
                }
            }
        };
        auto product = [&](int m, int st, bool add) {       // m: the tile; one tile: the scores' buffer
            const uint64_t bd = vd + st * (W::KB >> 4);
            const uint32_t p0 = tmem + (MT == 2 ? W::SP + 64 * m : NARROW ? W::SP : m == 0 ? W::S0 : W::S1);
#pragma unroll
            for (int part = 0; part < W::PARTS; ++part)
#pragma unroll
                for (int k = 0; k < KEYS / 16; ++k) {
                    const uint32_t own = NARROW ? k * 8 : k / (KT / 16) * KT + k % (KT / 16) * 8;      // P in its thread's scores
                    const uint32_t d = F32 ? (part == 0 ? W::O0 : W::O1) : MT == 1 || m == 0 ? W::O0 : W::O1;
                    tc::mma_f16_ts_lead(tmem + d, part < 2 ? p0 + (NARROW ? W::P2 - W::SP : KT / 2) * part + own : tmem + W::SP + 8 * k,
                                        bd + k * (2048 >> 4), ID_O, part > (F32 ? 1 : 0) || k > 0 ? 1u : add, lead);
                }
        };
        auto wait = [&](int bar, int parity) {
            const bool got = tc::wait_or_abort(&bars[bar], parity, abort_flag, a.status);
            tc::fence_after();
            return __all_sync(0xffffffffu, got) != 0;
        };
        bool ok = wait(B_Q, 0) && wait(B_K_FULL, 0);
#pragma unroll
        for (int m = 0; m < MT && ok; ++m) {
            if (m == 1) ok = wait(B_FREE, 0);
            if (!ok) break;
            scores(m, 0);
            tc::commit_lead(&bars[B_S + m], lead);
            if (m == MT - 1) tc::commit_lead(&bars[B_K_EMPTY], lead);
        }
        for (int j = 0; j < steps && ok && !(j % 8 == 0 && __any_sync(0xffffffffu, abort_flag.get())); ++j) {
            const int st = j & 1, nst = st ^ 1;
            const bool next = j + 1 < steps;
#pragma unroll
            for (int m = 0; m < MT && ok; ++m) {
                if (MT == 2 && next) {
                    // the tile's next scores, once the other tile's last are in registers
                    if (m == 0) ok = wait(B_K_FULL + nst, ((j + 1) >> 1) & 1);
                    ok = ok && wait(B_FREE + (m ^ 1), (j + m) & 1);
                    if (!ok) break;
                    scores(m, nst);
                    tc::commit_lead(&bars[B_S + m], lead);
                    if (m == 1) tc::commit_lead(&bars[B_K_EMPTY + nst], lead);
                }
                if (SBUF == 2 && next) {
                    // the other buffer's scores: its softmax was waited for a step ago
                    ok = wait(B_K_FULL + nst, ((j + 1) >> 1) & 1);
                    if (!ok) break;
                    scores(nst, nst);
                    tc::commit_lead(&bars[B_S + nst], lead);
                    tc::commit_lead(&bars[B_K_EMPTY + nst], lead);
                }
                ok = wait(B_P + m, j & 1);
                if (!ok) break;
                if (m == 0) ok = wait(B_V_FULL + st, (j >> 1) & 1);
                if (!ok) break;
                product(SBUF == 2 ? st : m, st, W::FLUSH > 0 ? j % (W::FLUSH > 0 ? W::FLUSH : 1) != 0 : j > 0);
                tc::commit_lead(&bars[B_O + m], lead);
                if (m == MT - 1) tc::commit_lead(&bars[B_V_EMPTY + st], lead);
                if (MT == 1 && SBUF == 1 && next) {
                    // P's columns are the scores': the MMAs run in the order they were issued in
                    ok = wait(B_K_FULL + nst, ((j + 1) >> 1) & 1);
                    if (!ok) break;
                    scores(0, nst);
                    tc::commit_lead(&bars[B_S], lead);
                    tc::commit_lead(&bars[B_K_EMPTY + nst], lead);
                }
            }
        }
        // Wherever the loop was left: all MMAs issued, and their arrivals at the other barriers, are
        // over before the tensor memory goes and the CTA's shared memory with it.
        tc::commit_lead(&bars[B_DRAINED], lead);
        (void)tc::wait_or_abort_sleep(&bars[B_DRAINED], 0, abort_flag, a.status);
        }
    }
    // ---- every role has left its loop, and no MMA is in flight
    tc::fence_before();
    __syncthreads();
    tc::fence_after();
    if (warp == (SOFT + CONV) / 32) tc::tmem_dealloc(tmem, 512);
}

template <typename T, int D, bool TREE, bool NARROW>
cudaError_t launch_tiles_n(const DeviceInfo& dev, const KvView& c, const AttnArgs& a, const RowsPlan& pl, cudaStream_t s) {
    using W = Tiles<T, D, TREE, NARROW>;
    if (W::SMEM > dev.smem_optin) return cudaErrorInvalidConfiguration;
    cudaError_t e = raise_smem_limit(reinterpret_cast<const void*>(attn_tiles_kernel<T, D, TREE, NARROW>), W::SMEM);
    if (e != cudaSuccess) return e;
    const int64_t G = a.heads / c.heads;
    // Each request that this kernel takes has at most one part-filled item more than its rows make
    int64_t items = (a.T * G / W::ROWS + std::min<int64_t>(a.R, a.T * G / pl.tile_rows + 1)) * c.heads;
    if (items > 0x7fffffff) return cudaErrorInvalidConfiguration;
    items = std::max<int64_t>(items, pl.sms);              // parts of items
    return launch_kernel(attn_tiles_kernel<T, D, TREE, NARROW>, dim3(static_cast<unsigned>(items)), dim3(W::THREADS), W::SMEM, s, c, a, pl);
}

template <typename T, int D, bool TREE>
cudaError_t launch_tiles_t(const DeviceInfo& dev, const KvView& c, const AttnArgs& a, const RowsPlan& pl, cudaStream_t s) {
    if constexpr (TREE && !std::is_same<T, float>::value) {
        if (pl.one_tile) return launch_tiles_n<T, D, TREE, true>(dev, c, a, pl, s);
    }
    return launch_tiles_n<T, D, TREE, false>(dev, c, a, pl, s);
}

template <bool TREE>
cudaError_t launch_tiles(const DeviceInfo& dev, const KvView& c, int dtype, const AttnArgs& a, const RowsPlan& pl,
                         cudaStream_t s) {
    const bool d64 = c.dim == 64;
    switch (dtype) {
    case CQ_F32: return d64 ? launch_tiles_t<float, 64, TREE>(dev, c, a, pl, s) : launch_tiles_t<float, 128, TREE>(dev, c, a, pl, s);
    case CQ_F16: return d64 ? launch_tiles_t<__half, 64, TREE>(dev, c, a, pl, s) : launch_tiles_t<__half, 128, TREE>(dev, c, a, pl, s);
    case CQ_BF16:
        return d64 ? launch_tiles_t<__nv_bfloat16, 64, TREE>(dev, c, a, pl, s)
                   : launch_tiles_t<__nv_bfloat16, 128, TREE>(dev, c, a, pl, s);
    default: return cudaErrorInvalidValue;
    }
}

}  // namespace

cudaError_t launch_attn_tiles(const DeviceInfo& dev, const KvView& c, int dtype, const AttnArgs& a, const RowsPlan& pl,
                              cudaStream_t s) {
    return a.tree != nullptr ? launch_tiles<true>(dev, c, dtype, a, pl, s) : launch_tiles<false>(dev, c, dtype, a, pl, s);
}

}  // namespace cq
