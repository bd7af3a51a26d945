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

#include "gdn_layer.hpp"

namespace gdn {

// cos and sin of pos * f: the angle in turns is formed and reduced to
// [-1/2, 1/2] in 64 bits, so that far positions keep every bit that 32 hold
__device__ __forceinline__ float2 turn(int64_t pos, double f) {
    double t = (double)pos * (f * 0.15915494309189533577);
    t -= rint(t);
    float s, c;
    sincospif((float)(2.0 * t), &s, &c);
    return make_float2(c, s);
}

// 8 consecutive elements as loaded
template <typename T> struct Oct;
template <> struct Oct<bf16> {
    uint4 r;
    __device__ __forceinline__ void load(const bf16* p) { r = *reinterpret_cast<const uint4*>(p); }
    __device__ __forceinline__ void zero() { r = make_uint4(0, 0, 0, 0); }
    __device__ __forceinline__ float get(int e) const { return Vec16<bf16>::get(r, e); }
    __device__ __forceinline__ static void store(bf16* p, const float* f) {
        *reinterpret_cast<uint4*>(p) = Vec16<bf16>::pack(f);
    }
};
template <> struct Oct<float> {
    float4 a, b;
    __device__ __forceinline__ void load(const float* p) {
        a = reinterpret_cast<const float4*>(p)[0];
        b = reinterpret_cast<const float4*>(p)[1];
    }
    __device__ __forceinline__ void zero() { a = b = make_float4(0.f, 0.f, 0.f, 0.f); }
    __device__ __forceinline__ float get(int e) const {
        const float4 v = e < 4 ? a : b;
        return (e & 3) == 0 ? v.x : (e & 3) == 1 ? v.y : (e & 3) == 2 ? v.z : v.w;
    }
    __device__ __forceinline__ static void store(float* p, const float* f) {
        reinterpret_cast<float4*>(p)[0] = make_float4(f[0], f[1], f[2], f[3]);
        reinterpret_cast<float4*>(p)[1] = make_float4(f[4], f[5], f[6], f[7]);
    }
};

template <int LPR>
__device__ __forceinline__ float row_sum(float v) {
#pragma unroll
    for (int off = 1; off < LPR; off <<= 1) v += __shfl_xor(v, off, 64);
    return v;
}

// What a lane needs of its token: the cosines of its 8 elements (4 pairs when
// interleaved) and the sines with the sign that its half takes.
template <bool INTER> struct Spin {
    float c[8], s[8];
    int partner;     // lane that holds the other half
    bool on;         // the lane's elements are rotated (R is a multiple of 16: all or none)
    // v rotated by the angle (back: by its negative), v as held by the row's lanes
    template <bool BACK>
    __device__ __forceinline__ void apply(float* v) const {
        if (INTER) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float a = v[2 * j], b = v[2 * j + 1], sj = BACK ? -s[j] : s[j];
                v[2 * j] = on ? a * c[j] - b * sj : a;
                v[2 * j + 1] = on ? b * c[j] + a * sj : b;
            }
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float o = __shfl(v[e], partner, 64), se = BACK ? -s[e] : s[e];
                v[e] = on ? v[e] * c[e] + o * se : v[e];
            }
        }
    }
};

template <bool INTER>
__device__ __forceinline__ void spin_of(const QkLaunch& p, int64_t token, float2* s_cs, int lane, int sub,
                                        Spin<INTER>* r) {
    const int half = p.R / 2, e0 = 8 * sub;
    __builtin_amdgcn_wave_barrier();   // the wave's LDS accesses stay in order
    if (half > 0) {
        const int64_t pos = p.positions ? p.positions[token] : (int64_t)((unsigned)token % (unsigned)p.T);
        for (int i = lane; i < half; i += 64) s_cs[i] = turn(pos, p.inv_freq[i]);
    }
    __builtin_amdgcn_wave_barrier();
    r->on = e0 < p.R;
    const bool up = e0 >= half;        // second half of a half-split pair
    r->partner = INTER || !r->on ? lane : up ? lane - half / 8 : lane + half / 8;
    const int i0 = !r->on ? 0 : INTER ? e0 / 2 : up ? e0 - half : e0;
#pragma unroll
    for (int e = 0; e < (INTER ? 4 : 8); ++e) {
        const float2 cs = half > 0 ? s_cs[i0 + e] : make_float2(1.f, 0.f);
        r->c[e] = cs.x;
        r->s[e] = INTER || up ? cs.y : -cs.y;
    }
}

__device__ __forceinline__ void gain_of(const QkLaunch& p, const float* w, int e0, bool live, float* g) {
#pragma unroll
    for (int e = 0; e < 8; ++e) g[e] = w && live ? w[e0 + e] + p.offset : 1.f;
}

__device__ __forceinline__ float norm_of(const QkLaunch& p, float ss, float inv_n) {
    return p.norm == GDN_NORM_NONE ? 1.f : 1.f / sqrtf(ss * inv_n + p.eps);
}

// rows [first, last) of one token, a group of 64 / LPR rows after another
template <typename T, int LPR, bool INTER>
__device__ __forceinline__ void heads_fwd(const QkLaunch& p, const Spin<INTER>& spin, const T* x, T* out,
                                          const float* w, int64_t hs, int64_t first, int64_t last, int lane,
                                          bool live) {
    constexpr int RPW = 64 / LPR, U = 2;
    const int sub = lane % LPR, e0 = 8 * sub;
    const bool in = e0 < p.D;
    const float inv_n = p.norm == GDN_NORM_RMS ? 1.f / (float)p.D : 1.f;
    float gain[8];
    gain_of(p, w, e0, in, gain);
    for (int64_t h0 = first; h0 < last; h0 += U * RPW) {
        Oct<T> raw[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t h = h0 + u * RPW + lane / LPR;
            if (in && h < last) raw[u].load(x + h * hs + e0);
            else raw[u].zero();
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t h = h0 + u * RPW + lane / LPR;
            float v[8], ss = 0.f;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                v[e] = raw[u].get(e);
                ss += v[e] * v[e];
            }
            const float r = norm_of(p, p.norm == GDN_NORM_NONE ? 0.f : row_sum<LPR>(ss), inv_n);
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] *= r * gain[e];
            spin.template apply<false>(v);
            if (in && live && h < last) Oct<T>::store(out + h * p.D + e0, v);
        }
    }
}

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
                                 static_cast<T*>(p.qo) + token * p.Hq * p.D, p.qw, p.qhs, a * RPW,
                                 min(b * RPW, p.Hq), lane, live);
    if (b > gq)
        heads_fwd<T, LPR, INTER>(p, spin, static_cast<const T*>(p.k) + token * p.ks,
                                 static_cast<T*>(p.ko) + token * p.Hk * p.D, p.kw, p.khs, (max(a, gq) - gq) * RPW,
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
