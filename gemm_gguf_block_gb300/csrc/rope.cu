// Norm and rotation of queries and keys (cq_qk_rope in include/cq_tree.h).
//
// D / 8 lanes hold a head, each two groups of four neighbouring values that are turned into one
// another (halves), or within themselves (adjacent pairs): a rotation moves nothing between
// lanes, and a head's sum of squares is three or four shuffles for two or four heads. The angles are
// the same for all heads of a token: a CTA goes through the tokens a few at a time and works out the
// next ones' sines and cosines while these ones' rows are on their way. An angle is held as a 64-bit
// fraction of a turn: the frequency's fraction times the position, modulo 2^64, is exact, where fp32
// would lose it (a position of 10^5 at one radian is known to 2^-8 of a radian) and fp64 runs at
// a sixty-fourth of fp32's rate; a thread keeps one frequency's fraction for all its tokens.
#include <algorithm>

#include "tree.cuh"

namespace cq {
namespace {

constexpr int THREADS = 256;
constexpr int WARPS = THREADS / 32;
constexpr int CTAS = 4;                     // of an SM
constexpr int MOST_TOKENS = 4;              // of a round
constexpr int BATCH = 4;                    // heads of a lane in flight

template <typename TI, typename TO, int D>
__global__ void __launch_bounds__(THREADS) qk_rope_kernel(const RopeArgs a, const int tokens) {
    pdl_trigger();
    pdl_wait();
    constexpr int LPH = D / 8, HPW = 32 / LPH;          // lanes of a head, heads of a warp
    // angles in the order of the lanes that use them: lane l its 4 l .. 4 l + 3
    __shared__ __align__(16) float cs[2][MOST_TOKENS][D / 2], sn[2][MOST_TOKENS][D / 2];
    __shared__ int where[2][MOST_TOKENS];               // the tokens' positions
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int half = a.rot / 2, H = a.heads[0] + a.heads[1];
    const int l = lane % LPH, turned = a.rot / 8;       // lanes of a head that turn
    // the lane's two groups of four: (l, l + turned) of the turned ones, then the others two by two
    const int g0 = l < turned ? l : 2 * turned + 2 * (l - turned), g1 = l < turned ? l + turned : g0 + 1;

    // thread: one frequency, every per-th token of a round
    const int mine = half > 0 && tid < THREADS / half * half ? tid % half : -1, per = half > 0 ? THREADS / half : 1;
    uint64_t turn = 0;
    if (mine >= 0) {
        const int e = mine & 3, ml = mine >> 2;
        const int i = !a.adjacent ? mine : e < 2 ? 2 * ml + e : 2 * (ml + turned) + e - 2;
        constexpr double INV = 0.15915494309189535, INV_LO = -9.839338337591243e-18;   // 1 / 2 pi in two parts
        // a negative frequency's is the positive one's, negated: exact, where the fraction of a small negative number is not
        const double f = a.freqs[i], size = fabs(f);
        double hi = size * INV;
        const double lo = fma(size, INV, -hi) + size * INV_LO;
        hi -= floor(hi);                                 // exact
        turn = static_cast<uint64_t>(hi * 18446744073709551616.0) +
               static_cast<uint64_t>(static_cast<int64_t>(lo * 18446744073709551616.0));
        if (f < 0.0) turn = 0 - turn;
    }
    auto angles = [&](int64_t t0, int buf) {
        if (tid < tokens && t0 + tid < a.T) where[buf][tid] = a.positions[t0 + tid];
        if (mine < 0) return;
        for (int t = tid / half; t < tokens && t0 + t < a.T; t += per) {
            const int64_t phase = static_cast<int64_t>(turn * static_cast<uint64_t>(static_cast<int64_t>(a.positions[t0 + t])));
            float s, c;
            sincospif(static_cast<float>(phase) * 1.0842021724855044e-19f, &s, &c);       // 2^-63: half turns
            cs[buf][t][mine] = c;
            sn[buf][t][mine] = s;
        }
    };

    const int64_t stride = static_cast<int64_t>(gridDim.x) * tokens;
    int buf = 0;
    int64_t t0 = static_cast<int64_t>(blockIdx.x) * tokens;
    if (t0 < a.T) angles(t0, 0);
    for (; t0 < a.T; t0 += stride, buf ^= 1) {
        __syncthreads();
        const int nt = static_cast<int>(min(static_cast<int64_t>(tokens), a.T - t0));
        // (token, head) of the lane, heads of a token in order
        int t = 0, h = warp * HPW + lane / LPH;
        while (h >= H) { h -= H; ++t; }
        bool first = true;
        do {
            Raw4<TI> v[BATCH][2];
            int at_t[BATCH], at_h[BATCH];
#pragma unroll
            for (int b = 0; b < BATCH; ++b) {
                at_t[b] = t < nt && where[buf][t] >= 0 ? t : -1;
                at_h[b] = h;
                v[b][0].zero();
                v[b][1].zero();
                if (at_t[b] >= 0) {
                    const int which = h >= a.heads[0];
                    const TI* p = static_cast<const TI*>(which ? a.x[1] : a.x[0]) + (t0 + t) * (which ? a.x_stride[1] : a.x_stride[0]) +
                                  (which ? h - a.heads[0] : h) * D;
                    v[b][0].load(p + 4 * g0);
                    v[b][1].load(p + 4 * g1);
                }
                h += WARPS * HPW;
                while (h >= H) { h -= H; ++t; }
            }
            if (first && t0 + stride < a.T) angles(t0 + stride, buf ^ 1);
            first = false;
#pragma unroll
            for (int b = 0; b < BATCH; ++b) {
                const int which = at_h[b] >= a.heads[0];
                float4 x = v[b][0].value(), y = v[b][1].value();
                auto squares = [&]() {
                    float s = fmaf(x.x, x.x, x.y * x.y) + fmaf(x.z, x.z, x.w * x.w) + (fmaf(y.x, y.x, y.y * y.y) + fmaf(y.z, y.z, y.w * y.w));
#pragma unroll
                    for (int o = LPH / 2; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
                    return s;
                };
                float ss = squares(), eps = a.eps;
                const float* norm = which ? a.w[1] : a.w[0];
                // Squares of tiny values fall below fp32's normal numbers, where eps does not hide them: a head whose mean is
                // below 2^-90 is taken 2^100 times as large, eps with its square, which the norm takes out again. (The test
                // of eps, the same for all, comes first: 82.9 us at 16003 tokens of fp32, without it 84.3.)
                constexpr float LEAST = 8.0779357e-28f;                                 // 2^-90
                if (eps < LEAST) {
                    const bool tiny = norm != nullptr && at_t[b] >= 0 && fmaf(ss, 1.0f / D, eps) < LEAST;
                    if (__any_sync(0xffffffffu, tiny)) {
                        const float up = tiny ? 1.2676506e30f : 1.0f;                   // 2^100
                        x = make_float4(x.x * up, x.y * up, x.z * up, x.w * up);
                        y = make_float4(y.x * up, y.y * up, y.z * up, y.w * up);
                        eps = eps * up * up;
                        ss = squares();
                    }
                }
                if (at_t[b] < 0) continue;
                if (norm != nullptr) {
                    const float4 w = *reinterpret_cast<const float4*>(norm + 4 * g0), z = *reinterpret_cast<const float4*>(norm + 4 * g1);
                    const float r = rsqrtf(fmaf(ss, 1.0f / D, eps));
                    x = make_float4(x.x * r * w.x, x.y * r * w.y, x.z * r * w.z, x.w * r * w.w);
                    y = make_float4(y.x * r * z.x, y.y * r * z.y, y.z * r * z.z, y.w * r * z.w);
                }
                if (l < turned) {
                    const float4 c = *reinterpret_cast<const float4*>(&cs[buf][at_t[b]][4 * l]), s = *reinterpret_cast<const float4*>(&sn[buf][at_t[b]][4 * l]);
                    const float4 p = x, q = y;
                    if (a.adjacent) {
                        x = make_float4(p.x * c.x - p.y * s.x, p.y * c.x + p.x * s.x, p.z * c.y - p.w * s.y, p.w * c.y + p.z * s.y);
                        y = make_float4(q.x * c.z - q.y * s.z, q.y * c.z + q.x * s.z, q.z * c.w - q.w * s.w, q.w * c.w + q.z * s.w);
                    } else {
                        x = make_float4(p.x * c.x - q.x * s.x, p.y * c.y - q.y * s.y, p.z * c.z - q.z * s.z, p.w * c.w - q.w * s.w);
                        y = make_float4(q.x * c.x + p.x * s.x, q.y * c.y + p.y * s.y, q.z * c.z + p.z * s.z, q.w * c.w + p.w * s.w);
                    }
                }
                TO* p = static_cast<TO*>(which ? a.y[1] : a.y[0]) + (t0 + at_t[b]) * (which ? a.y_stride[1] : a.y_stride[0]) +
                        (which ? at_h[b] - a.heads[0] : at_h[b]) * D;
                store4(p + 4 * g0, x);
                store4(p + 4 * g1, y);
            }
        } while (__any_sync(0xffffffffu, t < nt));       // (a warp stays together: it shuffles)
    }
}

constexpr int64_t rounds_of(int64_t T, int tokens) { return (T + tokens - 1) / tokens; }
static_assert(rounds_of(INT32_MAX, MOST_TOKENS) == INT32_MAX / MOST_TOKENS + 1, "the largest T is in range");

template <typename TI, typename TO, int D>
cudaError_t launch_d(const DeviceInfo& dev, const RopeArgs& a, cudaStream_t s) {
    // Tokens of a round: one where there are SMs for all of them, else four, so that a warp has several heads' loads
    // in flight between barriers. As many CTAs as run at once: each goes on to further tokens.
    int tokens = 1;
    while (tokens < MOST_TOKENS && a.T / (2 * tokens) >= CTAS * dev.sm_count) tokens *= 2;
    const int64_t ctas = std::min<int64_t>(rounds_of(a.T, tokens), static_cast<int64_t>(dev.sm_count) * CTAS);
    return launch_kernel(qk_rope_kernel<TI, TO, D>, dim3(static_cast<unsigned>(ctas)), dim3(THREADS), 0, s, a, tokens);
}

template <typename TI, typename TO>
cudaError_t launch_t(const DeviceInfo& dev, int64_t D, const RopeArgs& a, cudaStream_t s) {
    return D == 64 ? launch_d<TI, TO, 64>(dev, a, s) : launch_d<TI, TO, 128>(dev, a, s);
}

}  // namespace

cudaError_t launch_qk_rope(const DeviceInfo& dev, int in, int out, int64_t D, const RopeArgs& a, cudaStream_t s) {
    if (in == CQ_F32 && out == CQ_F32) return launch_t<float, float>(dev, D, a, s);
    if (in == CQ_F32 && out == CQ_F16) return launch_t<float, __half>(dev, D, a, s);
    if (in == CQ_F32 && out == CQ_BF16) return launch_t<float, __nv_bfloat16>(dev, D, a, s);
    if (in == CQ_F16 && out == CQ_F16) return launch_t<__half, __half>(dev, D, a, s);
    if (in == CQ_BF16 && out == CQ_BF16) return launch_t<__nv_bfloat16, __nv_bfloat16>(dev, D, a, s);
    return cudaErrorInvalidValue;
}

}  // namespace cq
