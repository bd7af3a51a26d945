// Gated linear recurrence over channels: h_t = a_t h_{t-1} + u_t, a = exp(g),
// u = x or sqrt(1 - a^2) x, and its backward pass.
//
// One thread per (sequence, channel) walks the tokens; the backward first
// leaves every h_t in a workspace, then walks back.
#include "gdn_layer.hpp"

namespace gdn {

// log a, and with it a, the factor m of x, and d log a / d g.  1 - a^2 is
// -expm1(2 log a), which keeps its leading bits for gates near 1.
struct Gate {
    float la, a, m, slope;
};
template <bool ACT, bool NORM>
__device__ __forceinline__ Gate gate_of(float g, float rate, float bias) {
    Gate r;
    if (ACT) {
        const float z = g + bias;
        r.la = rate * softplus_f(z);
        r.slope = rate / (1.f + expf(-z));
    } else {
        r.la = g;
        r.slope = 1.f;
    }
    r.a = expf(r.la);
    r.m = NORM ? sqrtf(-expm1f(2.f * r.la)) : 1.f;
    return r;
}

__device__ __forceinline__ void seq_of(const SeqMap& m, int64_t n, int64_t* row0, int64_t* len) {
    if (m.seqs) {
        const int4 s = m.seqs[n];
        *row0 = s.x;
        *len = s.y;
    } else {
        *row0 = n * m.T;
        *len = m.T;
    }
}

template <typename X, typename G, bool ACT, bool NORM>
__global__ __launch_bounds__(64) void linrec_fwd_kernel(LinrecLaunch p) {
    const int64_t nb = (p.D + 63) / 64, n = blockIdx.x / nb, c = (blockIdx.x - n * nb) * 64 + threadIdx.x;
    if (c >= p.D) return;
    const X* x = static_cast<const X*>(p.x);
    const G* g = static_cast<const G*>(p.g);
    X* y = static_cast<X*>(p.y);
    int64_t row0, len;
    seq_of(p.map, n, &row0, &len);
    const float rate = ACT ? -expf(p.act.A_log[c]) : 0.f, bias = ACT ? p.act.dt_bias[c] : 0.f;
    float h = p.h0 ? p.h0[n * p.D + c] : 0.f;
    for (int64_t t = 0; t < len; ++t) {
        const int64_t r = row0 + t;
        const Gate q = gate_of<ACT, NORM>(Elem<G>::load(g + r * p.gs + c), rate, bias);
        h = q.a * h + q.m * Elem<X>::load(x + r * p.xs + c);
        if (y) Elem<X>::store(y + r * p.ys + c, h);
        if (p.hbuf) p.hbuf[r * p.D + c] = h;
    }
    if (p.ht) p.ht[n * p.D + c] = h;
}

template <typename X, typename G, bool ACT, bool NORM>
__global__ __launch_bounds__(64) void linrec_bwd_kernel(LinrecLaunch p) {
    const int64_t nb = (p.D + 63) / 64, n = blockIdx.x / nb, c = (blockIdx.x - n * nb) * 64 + threadIdx.x;
    if (c >= p.D) return;
    const X *x = static_cast<const X*>(p.x), *dy = static_cast<const X*>(p.dy);
    const G* g = static_cast<const G*>(p.g);
    X* dx = static_cast<X*>(p.dx);
    G* dg = static_cast<G*>(p.dg);
    int64_t row0, len;
    seq_of(p.map, n, &row0, &len);
    const float rate = ACT ? -expf(p.act.A_log[c]) : 0.f, bias = ACT ? p.act.dt_bias[c] : 0.f;
    const float h0 = p.h0 ? p.h0[n * p.D + c] : 0.f;
    float e = p.dht ? p.dht[n * p.D + c] : 0.f, sA = 0.f, sb = 0.f;
    for (int64_t t = len - 1; t >= 0; --t) {
        const int64_t r = row0 + t;
        const Gate q = gate_of<ACT, NORM>(Elem<G>::load(g + r * p.gs + c), rate, bias);
        const float xv = Elem<X>::load(x + r * p.xs + c);
        const float before = t > 0 ? p.hbuf[(r - 1) * p.D + c] : h0;
        const float dh = Elem<X>::load(dy + r * p.ys + c) + e;
        e = q.a * dh;
        float dla = e * before;
        if (NORM && q.m > 0.f) dla -= e * xv * (q.a / q.m);
        Elem<X>::store(dx + r * p.D + c, q.m * dh);
        Elem<G>::store(dg + r * p.D + c, dla * q.slope);
        sA += dla * q.la;
        sb += dla * q.slope;
    }
    if (p.dh0) p.dh0[n * p.D + c] = e;
    if (ACT) {
        p.part[(2 * n) * p.D + c] = sA;
        p.part[(2 * n + 1) * p.D + c] = sb;
    }
}

__global__ __launch_bounds__(64) void linrec_sum_kernel(LinrecLaunch p) {
    const int64_t c = blockIdx.x * (int64_t)64 + threadIdx.x;
    if (c >= p.D) return;
    double sA = 0, sb = 0;
    for (int64_t n = 0; n < p.map.N; ++n) {
        sA += p.part[(2 * n) * p.D + c];
        sb += p.part[(2 * n + 1) * p.D + c];
    }
    p.dA_log[c] = (float)sA;
    p.ddt_bias[c] = (float)sb;
}

#define LINREC_CASES(KERNEL)                                                              \
    if (p.x_bf16)                                                                         \
        e = p.g_bf16 ? go<KERNEL, bf16, bf16>(p) : go<KERNEL, bf16, float>(p);            \
    else                                                                                  \
        e = p.g_bf16 ? go<KERNEL, float, bf16>(p) : go<KERNEL, float, float>(p);

enum { FWD, BWD };
template <int WHICH, typename X, typename G, bool ACT, bool NORM>
static hipError_t go1(const LinrecLaunch& p) {
    const dim3 grid((unsigned)((p.D + 63) / 64 * p.map.N));
    if (WHICH == FWD)
        hipLaunchKernelGGL((linrec_fwd_kernel<X, G, ACT, NORM>), grid, dim3(64), 0, p.stream, p);
    else
        hipLaunchKernelGGL((linrec_bwd_kernel<X, G, ACT, NORM>), grid, dim3(64), 0, p.stream, p);
    return hipGetLastError();
}
template <int WHICH, typename X, typename G>
static hipError_t go(const LinrecLaunch& p) {
    if (p.act.flags & ACT_GATE)
        return p.normalize ? go1<WHICH, X, G, true, true>(p) : go1<WHICH, X, G, true, false>(p);
    return p.normalize ? go1<WHICH, X, G, false, true>(p) : go1<WHICH, X, G, false, false>(p);
}

hipError_t launch_linrec_fwd(const LinrecLaunch& p) {
    hipError_t e;
    LINREC_CASES(FWD)
    return e;
}

hipError_t launch_linrec_bwd(const LinrecLaunch& p) {
    LinrecLaunch f = p;
    f.y = nullptr;
    f.ht = nullptr;
    hipError_t e = launch_linrec_fwd(f);
    if (e != hipSuccess) return e;
    LINREC_CASES(BWD)
    if (e != hipSuccess || !(p.act.flags & ACT_GATE)) return e;
    hipLaunchKernelGGL(linrec_sum_kernel, dim3((unsigned)((p.D + 63) / 64)), dim3(64), 0, p.stream, p);
    return hipGetLastError();
}

// The single token: sequences of one token whose state is both h0 and ht.
hipError_t launch_linrec_step(const LinrecLaunch& p) { return launch_linrec_fwd(p); }

}  // namespace gdn
