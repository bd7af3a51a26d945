// Norm of each q and k head and the rotation of its first R elements by
// position, and its backward pass.
//
// A wave takes a token: first the token's R/2 angles, one or two to a lane,
// into LDS, then its heads, 64 / LPR rows at a time with LPR lanes of 8
// elements to a row (16-byte loads and stores).  The cosines, sines and
// weights of a lane's 8 elements stay in registers for all heads of the
// token, so the angle's 64-bit arithmetic is paid once for q_heads + k_heads
// rows.  Few tokens (decode) split their heads over several waves.
//
// Measured (bf16): 4 x 4096 tokens of 16 + 16 heads of 128, 51 us, 5.3 TB/s
// with part of it in the cache; 16411 tokens of 32 + 8 heads, 67 us forward
// (5.0 TB/s, a large copy's rate) and 122 us backward with the sums for the weights (4.1
// TB/s); 64 tokens of 16 + 2 heads of 256, 5.0 us.
//
// The element that a half-split rotation pairs with sits R/16 lanes away and
// comes by a lane shuffle; interleaved pairs are in the lane itself.
#include <algorithm>

#include "gdn_rope.hpp"

namespace gdn {

template <typename T, int LPR, bool INTER>
__global__ __launch_bounds__(256) void qk_fwd_kernel(QkLaunch p) {
    __shared__ float2 s_cs[4][128];
    constexpr int RPW = 64 / LPR;
    const int lane = threadIdx.x & 63, w = wave_id();
    const int64_t task = (int64_t)blockIdx.x * 4 + w, all = p.tokens * p.split;
    const bool live = task < all;
    const int64_t t = live ? task : all - 1, token = t / p.split, part = t - token * p.split;
    Spin<INTER> spin;
    spin_of<INTER>(p, token, s_cs[w], lane, lane % LPR, &spin);
    // this wave's share of the token's row groups, q's before k's
    const int64_t gq = (p.Hq + RPW - 1) / RPW, gk = (p.Hk + RPW - 1) / RPW, per = (gq + gk + p.split - 1) / p.split;
    const int64_t a = part * per, b = min(a + per, gq + gk);
    if (a < gq)
        heads_fwd<T, LPR, INTER>(p, spin, static_cast<const T*>(p.q) + token * p.qs,
                                 static_cast<T*>(p.qo) + token * p.Hq * p.D, p.qw, p.qhs, p.D, a * RPW,
                                 min(b * RPW, p.Hq), lane, live);
    if (b > gq)
        heads_fwd<T, LPR, INTER>(p, spin, static_cast<const T*>(p.k) + token * p.ks,
                                 static_cast<T*>(p.ko) + token * p.Hk * p.D, p.kw, p.khs, p.D, (max(a, gq) - gq) * RPW,
                                 min((b - gq) * RPW, p.Hk), lane, live);
}

// dn = rotation back of dy; with dw_i = dn_i w_i:
// dx = r (dw - x r^2/n sum x dw), and the weight's gradient sums dn x r
template <typename T, int LPR, bool INTER>
__device__ __forceinline__ void heads_bwd(const QkLaunch& p, const Spin<INTER>& spin, const T* x, const T* dy, T* dx,
                                          const float* w, int64_t hs, int64_t H, int lane, float* acc) {
    constexpr int RPW = 64 / LPR;
    const int sub = lane % LPR, e0 = 8 * sub;
    const bool in = e0 < p.D;
    const float inv_n = p.norm == GDN_NORM_RMS ? 1.f / (float)p.D : 1.f;
    float gain[8];
    gain_of(p, w, e0, in, gain);
    // the next group's rows are loaded before this one's are worked on
    Oct<T> nx, nd;
    const auto fetch = [&](int64_t h) {
        if (in && h < H) {
            nx.load(x + h * hs + e0);
            nd.load(dy + h * p.D + e0);
        } else {
            nx.zero();
            nd.zero();
        }
    };
    fetch(lane / LPR);
    for (int64_t h0 = 0; h0 < H; h0 += RPW) {
        const int64_t h = h0 + lane / LPR;
        const bool row = in && h < H;
        const Oct<T> rx = nx, rd = nd;
        if (h0 + RPW < H) fetch(h + RPW);
        float v[8], d[8], ss = 0.f, dot = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            v[e] = rx.get(e);
            d[e] = rd.get(e);
            ss += v[e] * v[e];
        }
        spin.template apply<true>(d);
#pragma unroll
        for (int e = 0; e < 8; ++e) dot += v[e] * (d[e] * gain[e]);
        float r = 1.f, k = 0.f;
        if (p.norm != GDN_NORM_NONE) {
            r = norm_of(p, row_sum<LPR>(ss), inv_n);
            k = r * r * inv_n * row_sum<LPR>(dot);
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            if (row) acc[e] += d[e] * (v[e] * r);
            d[e] = r * (d[e] * gain[e] - v[e] * k);
        }
        if (row) Oct<T>::store(dx + h * p.D + e0, d);
    }
}

// Waves walk the tokens by the grid's number of waves, for q and then for k:
// only one of the two keeps its sums for the weights in registers at a time.
// They stay there until the lane's last token, then meet over the workgroup's rows in LDS.
template <typename T, int LPR, bool INTER>
__global__ __launch_bounds__(256, 4) void qk_bwd_kernel(QkLaunch p) {
    __shared__ float2 s_cs[4][128];
    __shared__ float s_acc[4 * (64 / LPR)][8 * LPR];
    constexpr int RPW = 64 / LPR;
    const int lane = threadIdx.x & 63, w = wave_id(), sub = lane % LPR;
#pragma unroll 1
    for (int which = 0; which < 2; ++which) {
        const int64_t H = which ? p.Hk : p.Hq, ts = which ? p.ks : p.qs, hs = which ? p.khs : p.qhs;
        const T* x = static_cast<const T*>(which ? p.k : p.q);
        const T* dy = static_cast<const T*>(which ? p.dko : p.dqo);
        T* dx = static_cast<T*>(which ? p.ko : p.qo);
        float acc[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) acc[e] = 0.f;
        for (int64_t token = (int64_t)blockIdx.x * 4 + w; token < p.tokens; token += (int64_t)gridDim.x * 4) {
            Spin<INTER> spin;
            spin_of<INTER>(p, token, s_cs[w], lane, sub, &spin);
            heads_bwd<T, LPR, INTER>(p, spin, x + token * ts, dy + token * H * p.D, dx + token * H * p.D,
                                     which ? p.kw : p.qw, hs, H, lane, acc);
        }
        if (!(which ? p.dkw : p.dqw)) continue;
        __syncthreads();
#pragma unroll
        for (int e = 0; e < 8; ++e) s_acc[w * RPW + lane / LPR][8 * sub + e] = acc[e];
        __syncthreads();
        const int e = threadIdx.x;
        if (e < p.D) {
            float s = 0.f;
            for (int i = 0; i < 4 * RPW; ++i) s += s_acc[i][e];
            p.part[((int64_t)blockIdx.x * 2 + which) * p.D + e] = s;
        }
    }
}

template <typename T, int LPR, bool INTER>
static hipError_t go2(const QkLaunch& p, bool bwd) {
    if (bwd) {
        hipLaunchKernelGGL((qk_bwd_kernel<T, LPR, INTER>), dim3((unsigned)qk_bwd_blocks(p.tokens)), dim3(256), 0,
                           p.stream, p);
    } else {
        // Waves for at least half of the chip's slots: decode's few tokens share their row
        // groups out, one to a wave at most.
        QkLaunch a = p;
        const int64_t rpw = 64 / LPR, groups = (p.Hq + rpw - 1) / rpw + (p.Hk + rpw - 1) / rpw;
        a.split = std::min(groups, std::max((int64_t)1, 4096 / p.tokens));
        hipLaunchKernelGGL((qk_fwd_kernel<T, LPR, INTER>), dim3((unsigned)((p.tokens * a.split + 3) / 4)), dim3(256),
                           0, p.stream, a);
    }
    return hipGetLastError();
}
template <typename T, bool INTER>
static hipError_t go1(const QkLaunch& p, bool bwd) {
    if (p.D <= 32) return go2<T, 4, INTER>(p, bwd);
    if (p.D <= 64) return go2<T, 8, INTER>(p, bwd);
    if (p.D <= 128) return go2<T, 16, INTER>(p, bwd);
    return go2<T, 32, INTER>(p, bwd);
}
static hipError_t go(const QkLaunch& p, bool bwd) {
    if (p.bf16) return p.interleaved ? go1<bf16, true>(p, bwd) : go1<bf16, false>(p, bwd);
    return p.interleaved ? go1<float, true>(p, bwd) : go1<float, false>(p, bwd);
}

// Workgroups of the backward: a token to a wave, more only to bound the partial
// rows (16411 tokens of 40 heads: 119 us with one, 127 with two).
int64_t qk_bwd_blocks(int64_t tokens) {
    const int64_t per = std::max((int64_t)1, tokens / 16384);
    return (tokens + 4 * per - 1) / (4 * per);
}

hipError_t launch_qk(const QkLaunch& p) { return go(p, false); }

hipError_t launch_qk_bwd(const QkLaunch& p) {
    if (p.tokens > 0) {
        hipError_t e = go(p, true);
        if (e != hipSuccess) return e;
    }
    if (!p.dqw && !p.dkw) return hipSuccess;
    return launch_row_sum(RowSumLaunch{p.part, qk_bwd_blocks(p.tokens), p.D, 1, 2, p.dqw, p.dkw, p.sums, p.stream});
}

}  // namespace gdn
