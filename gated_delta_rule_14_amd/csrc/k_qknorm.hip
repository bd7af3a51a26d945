// Norm of each q and k head and the rotation of its first R elements by
// position, and its backward pass.
//
// One wave per (token, head) row; lane l holds elements l, l + 64, ... so any
// pair of a rotation is reached through the row in LDS.
#include "gdn_layer.hpp"

namespace gdn {

// cos and sin of pos * f: the angle in turns is formed and reduced to
// [-1/2, 1/2] in 64 bits, so that far positions keep every bit that 32 hold.
__device__ __forceinline__ void turn(int64_t pos, double f, float* c, float* s) {
    double t = (double)pos * (f * 0.15915494309189533577);
    t -= rint(t);
    sincospif((float)(2.0 * t), s, c);
}

struct Row {
    bool is_q;
    int64_t token, head;
};
__device__ __forceinline__ Row row_of(const QkLaunch& p, int64_t i) {
    const int64_t H = p.Hq + p.Hk, h = i % H;
    return Row{h < p.Hq, i / H, h < p.Hq ? h : h - p.Hq};
}

template <typename T, bool BWD>
__global__ __launch_bounds__(64) void qk_kernel(QkLaunch p) {
    __shared__ float s_row[256];
    const int lane = threadIdx.x;
    const Row r = row_of(p, blockIdx.x);
    const T* x = r.is_q ? static_cast<const T*>(p.q) + r.token * p.qs + r.head * p.qhs
                        : static_cast<const T*>(p.k) + r.token * p.ks + r.head * p.khs;
    const int64_t dense = (r.token * (r.is_q ? p.Hq : p.Hk) + r.head) * p.D;
    T* out = static_cast<T*>(r.is_q ? p.qo : p.ko) + dense;
    const float* w = r.is_q ? p.qw : p.kw;
    const int64_t pos = p.positions ? p.positions[r.token] : r.token % p.T;
    const int half = p.R / 2;
    float v[4], d[4], ss = 0.f;
    for (int i = 0; i < 4; ++i) {
        const int e = lane + 64 * i;
        v[i] = e < p.D ? Elem<T>::load(x + e) : 0.f;
        ss += v[i] * v[i];
    }
    ss = wave_sum(ss);
    const float nn = p.norm == GDN_NORM_RMS ? (float)p.D : 1.f;
    const float rr = p.norm == GDN_NORM_NONE ? 1.f : 1.f / sqrtf(ss / nn + p.eps);
    const T* dy = nullptr;
    if (BWD) dy = static_cast<const T*>(r.is_q ? p.dqo : p.dko) + dense;
    for (int i = 0; i < 4; ++i) {
        const int e = lane + 64 * i;
        d[i] = 0.f;
        if (e < p.D) {
            if (BWD) d[i] = Elem<T>::load(dy + e);
            s_row[e] = BWD ? d[i] : v[i] * rr * (w ? w[e] + p.offset : 1.f);
        }
    }
    __syncthreads();
    float dot = 0.f;
    for (int i = 0; i < 4; ++i) {
        const int e = lane + 64 * i;
        float y = e < p.D ? s_row[e] : 0.f;
        if (e < p.R) {
            const int f = p.interleaved ? e >> 1 : (e < half ? e : e - half);
            const bool first = p.interleaved ? !(e & 1) : e < half;
            const float other = s_row[p.interleaved ? e ^ 1 : (first ? e + half : e - half)];
            float c, s;
            turn(pos, p.inv_freq[f], &c, &s);
            if (BWD) s = -s;
            y = first ? y * c - other * s : y * c + other * s;
        }
        if (BWD) {
            d[i] = y;    // gradient of the normalised, weighted row
            dot += v[i] * y * (w && e < p.D ? w[e] + p.offset : 1.f);
        } else if (e < p.D) {
            Elem<T>::store(out + e, y);
        }
    }
    if (BWD) {
        dot = p.norm == GDN_NORM_NONE ? 0.f : wave_sum(dot);
        float* part = r.is_q ? (p.dqw ? p.part : nullptr) : (p.dkw ? p.part : nullptr);
        for (int i = 0; i < 4; ++i) {
            const int e = lane + 64 * i;
            if (e >= p.D) continue;
            const float dn = d[i] * (w ? w[e] + p.offset : 1.f);
            Elem<T>::store(out + e, rr * (dn - v[i] * (rr * rr / nn) * dot));
            if (part) part[(int64_t)blockIdx.x * p.D + e] = d[i] * v[i] * rr;
        }
    }
}

__global__ __launch_bounds__(64) void qk_sum_kernel(QkLaunch p) {
    const int e = blockIdx.x * 64 + threadIdx.x;
    const bool is_q = blockIdx.y == 0;
    float* out = is_q ? p.dqw : p.dkw;
    if (e >= p.D || !out) return;
    double s = 0;
    const int64_t H = p.Hq + p.Hk;
    for (int64_t t = 0; t < p.tokens; ++t)
        for (int64_t h = is_q ? 0 : p.Hq; h < (is_q ? p.Hq : H); ++h) s += p.part[(t * H + h) * p.D + e];
    out[e] = (float)s;
}

hipError_t launch_qk(const QkLaunch& p) {
    const dim3 grid((unsigned)(p.tokens * (p.Hq + p.Hk)));
    if (p.bf16)
        hipLaunchKernelGGL((qk_kernel<bf16, false>), grid, dim3(64), 0, p.stream, p);
    else
        hipLaunchKernelGGL((qk_kernel<float, false>), grid, dim3(64), 0, p.stream, p);
    return hipGetLastError();
}

hipError_t launch_qk_bwd(const QkLaunch& p) {
    const dim3 grid((unsigned)(p.tokens * (p.Hq + p.Hk)));
    if (p.tokens > 0) {
        if (p.bf16)
            hipLaunchKernelGGL((qk_kernel<bf16, true>), grid, dim3(64), 0, p.stream, p);
        else
            hipLaunchKernelGGL((qk_kernel<float, true>), grid, dim3(64), 0, p.stream, p);
        hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    if (!p.dqw && !p.dkw) return hipSuccess;
    hipLaunchKernelGGL(qk_sum_kernel, dim3((unsigned)((p.D + 63) / 64), 2), dim3(64), 0, p.stream, p);
    return hipGetLastError();
}

}  // namespace gdn
