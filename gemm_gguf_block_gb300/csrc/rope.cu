// Norm and rotation of queries and keys (cq_qk_rope in include/cq_tree.h).
//
// A head of D values lies with D / 4 lanes, four values each; its sum of squares
// is a few shuffles, and the partner of a value is in the same lane (adjacent
// pairs) or rot / 8 lanes away. The angles are the same for all heads of a token:
// a CTA takes a few tokens, works out their sines and cosines once and goes over
// the heads. An angle is held as a 64-bit fraction of a turn: the frequency's
// fraction times the position, modulo 2^64, is exact, where fp32 would lose it
// (a position of 10^5 at one radian is known to 2^-8 of a radian) and fp64 runs at
// a sixty-fourth of fp32's rate.
#include <algorithm>

#include "tree.cuh"

namespace cq {
namespace {

constexpr int THREADS = 256;
constexpr int WARPS = THREADS / 32;
constexpr int MOST_TOKENS = 16;             // of a CTA
constexpr int BATCH = 4;                    // heads of a warp's lanes in flight

template <typename TI, typename TO, int D>
__global__ void __launch_bounds__(THREADS) qk_rope_kernel(const RopeArgs a, const int tokens) {
    pdl_trigger();
    pdl_wait();
    constexpr int LPH = D / 4, HPW = 32 / LPH;          // lanes of a head, heads of a warp
    __shared__ __align__(16) float cs[MOST_TOKENS][D / 2], sn[MOST_TOKENS][D / 2];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int half = a.rot / 2, H = a.heads[0] + a.heads[1];
    const int64_t t0 = static_cast<int64_t>(blockIdx.x) * tokens;
    const int nt = static_cast<int>(min(static_cast<int64_t>(tokens), a.T - t0));

    // item: (token, head), heads of a token in order
    struct Item { int t, h; };
    const int step = WARPS * HPW;
    auto forward = [&](Item& it) {
        it.h += step;
        while (it.h >= H) { it.h -= H; ++it.t; }
    };
    Item it{0, warp * HPW + lane / LPH};
    while (it.h >= H) { it.h -= H; ++it.t; }
    const int d0 = (lane % LPH) * 4;
    Raw4<TI> v[BATCH];
    Item at[BATCH];
    int pos[BATCH];
    auto load = [&]() {
#pragma unroll
        for (int b = 0; b < BATCH; ++b) {
            at[b] = it;
            pos[b] = -1;
            v[b].zero();
            if (it.t < nt) {
                const int which = it.h >= a.heads[0], h = it.h - (which ? a.heads[0] : 0);
                const int64_t t = t0 + it.t;
                pos[b] = a.positions[t];
                v[b].load(static_cast<const TI*>(a.x[which]) + t * a.x_stride[which] + h * D + d0);
            }
            forward(it);
        }
    };
    load();                                              // on its way while the angles are worked out

    // thread: one frequency, every (THREADS / half)-th token
    if (half > 0 && tid < THREADS / half * half) {
        const int i = tid % half;
        constexpr double INV = 0.15915494309189535, INV_LO = -9.839338337591243e-18;   // 1 / 2 pi in two parts
        const double f = a.freqs[i];
        double hi = f * INV;
        const double lo = fma(f, INV, -hi) + f * INV_LO;
        hi -= floor(hi);                                 // exact
        const uint64_t turn = static_cast<uint64_t>(hi * 18446744073709551616.0) +
                              static_cast<uint64_t>(static_cast<int64_t>(lo * 18446744073709551616.0));
        for (int t = tid / half; t < nt; t += THREADS / half) {
            const int64_t phase = static_cast<int64_t>(turn * static_cast<uint64_t>(static_cast<int64_t>(a.positions[t0 + t])));
            float s, c;
            sincospif(static_cast<float>(phase) * 1.0842021724855044e-19f, &s, &c);       // 2^-63: half turns
            cs[t][i] = c;
            sn[t][i] = s;
        }
    }
    __syncthreads();

    // the lane's angles and its partner's lane
    const bool turned = d0 < a.rot;
    const int i0 = a.adjacent ? d0 / 2 : d0 < half ? d0 : d0 - half;
    const int other = a.adjacent || !turned ? lane : d0 < half ? lane + half / 4 : lane - half / 4;
    const float side = d0 < half ? -1.0f : 1.0f;
    for (;;) {
#pragma unroll
        for (int b = 0; b < BATCH; ++b) {
            const Item x = at[b];
            const int which = x.h >= a.heads[0], h = x.h - (which ? a.heads[0] : 0);
            const bool on = x.t < nt && pos[b] >= 0;
            float4 f = v[b].value();
            float ss = fmaf(f.x, f.x, f.y * f.y) + fmaf(f.z, f.z, f.w * f.w);
#pragma unroll
            for (int o = LPH / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
            if (on && a.w[which] != nullptr) {
                const float4 w = *reinterpret_cast<const float4*>(a.w[which] + d0);
                const float r = __frsqrt_rn(fmaf(ss, 1.0f / D, a.eps));
                f = make_float4(f.x * r * w.x, f.y * r * w.y, f.z * r * w.z, f.w * r * w.w);
            }
            float4 g;
            g.x = __shfl_sync(0xffffffffu, f.x, other);
            g.y = __shfl_sync(0xffffffffu, f.y, other);
            g.z = __shfl_sync(0xffffffffu, f.z, other);
            g.w = __shfl_sync(0xffffffffu, f.w, other);
            if (!on) continue;
            if (turned) {
                if (a.adjacent) {
                    const float2 c = *reinterpret_cast<const float2*>(&cs[x.t][i0]), s = *reinterpret_cast<const float2*>(&sn[x.t][i0]);
                    f = make_float4(f.x * c.x - f.y * s.x, f.y * c.x + f.x * s.x, f.z * c.y - f.w * s.y, f.w * c.y + f.z * s.y);
                } else {
                    const float4 c = *reinterpret_cast<const float4*>(&cs[x.t][i0]), s = *reinterpret_cast<const float4*>(&sn[x.t][i0]);
                    f = make_float4(fmaf(side * g.x, s.x, f.x * c.x), fmaf(side * g.y, s.y, f.y * c.y),
                                    fmaf(side * g.z, s.z, f.z * c.z), fmaf(side * g.w, s.w, f.w * c.w));
                }
            }
            store4(static_cast<TO*>(a.y[which]) + (t0 + x.t) * a.y_stride[which] + h * D + d0, f);
        }
        // (the first item of a batch is the earliest of its lanes; a warp leaves as one)
        if (!__any_sync(0xffffffffu, it.t < nt)) break;
        load();
    }
}

template <typename TI, typename TO>
cudaError_t launch_t(const DeviceInfo& dev, int64_t D, const RopeArgs& a, cudaStream_t s) {
    // Tokens of a CTA: enough heads for its warps' loads in flight, as long as there are CTAs for every SM.
    const int H = a.heads[0] + a.heads[1];
    int tokens = 1;
    while (tokens < MOST_TOKENS && (tokens * H < 8 * WARPS || tokens < 4) && a.T / (2 * tokens) >= 2 * dev.sm_count) tokens *= 2;
    const dim3 grid(static_cast<unsigned>((a.T + tokens - 1) / tokens));
    return D == 64 ? launch_kernel(qk_rope_kernel<TI, TO, 64>, grid, dim3(THREADS), 0, s, a, tokens)
                   : launch_kernel(qk_rope_kernel<TI, TO, 128>, grid, dim3(THREADS), 0, s, a, tokens);
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
