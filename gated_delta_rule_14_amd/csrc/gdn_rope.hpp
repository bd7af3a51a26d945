// The norm of a head and its rotation by position, as the kernels that write q
// and k share them: a token's angles in LDS, a lane's 8 elements of a row, and
// the rows of a token by one wave (the layout is described in k_qknorm.hip).
#pragma once

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
__device__ __forceinline__ void spin_at(const QkLaunch& p, int64_t pos, float2* s_cs, int lane, int sub,
                                        Spin<INTER>* r) {
    const int half = p.R / 2, e0 = 8 * sub;
    __builtin_amdgcn_wave_barrier();   // the wave's LDS accesses stay in order
    if (half > 0) {
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

template <bool INTER>
__device__ __forceinline__ void spin_of(const QkLaunch& p, int64_t token, float2* s_cs, int lane, int sub,
                                        Spin<INTER>* r) {
    int64_t pos = 0;
    if (p.R > 0) pos = p.positions ? p.positions[token] : (int64_t)((unsigned)token % (unsigned)p.T);
    spin_at<INTER>(p, pos, s_cs, lane, sub, r);
}

__device__ __forceinline__ void gain_of(const QkLaunch& p, const float* w, int e0, bool live, float* g) {
#pragma unroll
    for (int e = 0; e < 8; ++e) g[e] = w && live ? w[e0 + e] + p.offset : 1.f;
}

__device__ __forceinline__ float norm_of(const QkLaunch& p, float ss, float inv_n) {
    return p.norm == GDN_NORM_NONE ? 1.f : 1.f / sqrtf(ss * inv_n + p.eps);
}

// rows [first, last) of one token, a group of 64 / LPR rows after another; the outputs' rows ohs apart
template <typename T, int LPR, bool INTER>
__device__ __forceinline__ void heads_fwd(const QkLaunch& p, const Spin<INTER>& spin, const T* x, T* out,
                                          const float* w, int64_t hs, int64_t ohs, int64_t first, int64_t last,
                                          int lane, bool live) {
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
            if (in && live && h < last) Oct<T>::store(out + h * ohs + e0, v);
        }
    }
}

}  // namespace gdn
