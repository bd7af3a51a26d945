// Short causal depthwise convolution (width W in 2..4) with an optional SiLU,
// and its backward pass.
//
// One workgroup per (tile of tokens, 64 channels); a thread walks a tile's
// tokens with the last W - 1 inputs in registers.  The carried window is row
// 0..W-2 before a sequence's first token.
#include "gdn_layer.hpp"

namespace gdn {

// input at position p of a sequence (p >= -(W-1)); s0 may be null
template <typename T>
__device__ __forceinline__ float input_at(const ConvLaunch& a, const T* x, const T* s0, int64_t row0,
                                          int64_t seq, int64_t p, int64_t c) {
    if (p >= 0) return Elem<T>::load(x + (row0 + p) * a.xs + c);
    if (!s0) return 0.f;
    return Elem<T>::load(s0 + (seq * (a.W - 1) + a.W - 1 + p) * a.D + c);
}

__device__ __forceinline__ float sigmoid_f(float z) { return 1.f / (1.f + expf(-z)); }

// z and silu'(z) (or 1) at position p
template <typename T>
__device__ __forceinline__ float preact(const ConvLaunch& a, const T* x, const T* s0, int64_t row0,
                                        int64_t seq, int64_t p, int64_t c) {
    float z = a.b ? a.b[c] : 0.f;
    for (int j = 0; j < a.W; ++j)
        z += a.w[c * a.W + j] * input_at(a, x, s0, row0, seq, p - (a.W - 1) + j, c);
    return z;
}

__device__ __forceinline__ float slope_of(bool silu, float z) {
    if (!silu) return 1.f;
    const float s = sigmoid_f(z);
    return s * (1.f + z * (1.f - s));
}

template <typename T>
__global__ __launch_bounds__(64) void conv_fwd_kernel(ConvLaunch a) {
    const int64_t nb = (a.D + 63) / 64, tile = blockIdx.x / nb, c = (blockIdx.x - tile * nb) * 64 + threadIdx.x;
    if (c >= a.D) return;
    const Tile t = tile_of(a.map, tile);
    const T *x = static_cast<const T*>(a.x), *s0 = static_cast<const T*>(a.s0);
    T* y = static_cast<T*>(a.y);
    const int64_t p0 = (int64_t)t.j * a.map.tile, seq0 = t.row0 - p0;
    for (int i = 0; i < t.n; ++i) {
        const float z = preact(a, x, s0, seq0, t.seq, p0 + i, c);
        Elem<T>::store(y + (t.row0 + i) * a.ys + c, a.silu ? z * sigmoid_f(z) : z);
    }
}

__device__ __forceinline__ void conv_seq(const SeqMap& m, int64_t n, int64_t* row0, int64_t* len) {
    if (m.seqs) {
        const int4 s = m.seqs[n];
        *row0 = s.x;
        *len = s.y;
    } else {
        *row0 = n * m.T;
        *len = m.T;
    }
}

// st: the last W - 1 inputs of each sequence
template <typename T>
__global__ __launch_bounds__(64) void conv_window_kernel(ConvLaunch a) {
    const int64_t nb = (a.D + 63) / 64, n = blockIdx.x / nb, c = (blockIdx.x - n * nb) * 64 + threadIdx.x;
    if (c >= a.D) return;
    const T *x = static_cast<const T*>(a.x), *s0 = static_cast<const T*>(a.s0);
    int64_t row0, len;
    conv_seq(a.map, n, &row0, &len);
    for (int r = 0; r < a.W - 1; ++r)
        Elem<T>::store(static_cast<T*>(a.st) + (n * (a.W - 1) + r) * a.D + c,
                       input_at(a, x, s0, row0, n, len - (a.W - 1) + r, c));
}

template <typename T>
__global__ __launch_bounds__(64) void conv_bwd_kernel(ConvLaunch a) {
    const int64_t nb = (a.D + 63) / 64, tile = blockIdx.x / nb, c = (blockIdx.x - tile * nb) * 64 + threadIdx.x;
    if (c >= a.D) return;
    const Tile t = tile_of(a.map, tile);
    const T *x = static_cast<const T*>(a.x), *s0 = static_cast<const T*>(a.s0);
    const T *dy = static_cast<const T*>(a.dy), *dst = static_cast<const T*>(a.dst);
    const int64_t p0 = (int64_t)t.j * a.map.tile, seq0 = t.row0 - p0;
    int64_t row0, len = 0;
    if (t.n > 0) conv_seq(a.map, t.seq, &row0, &len);
    float sw[4] = {0.f, 0.f, 0.f, 0.f}, sb = 0.f;
    for (int i = 0; i < t.n; ++i) {
        const int64_t p = p0 + i;
        float dx = 0.f;
        for (int k = 0; k < a.W && p + k < len; ++k) {
            const float z = preact(a, x, s0, seq0, t.seq, p + k, c);
            const float dz = Elem<T>::load(dy + (seq0 + p + k) * a.ys + c) * slope_of(a.silu, z);
            dx += dz * a.w[c * a.W + a.W - 1 - k];
            if (k == 0) {
                sb += dz;
                for (int j = 0; j < a.W; ++j)
                    sw[j] += dz * input_at(a, x, s0, seq0, t.seq, p - (a.W - 1) + j, c);
            }
        }
        const int64_t kept = p - len + a.W - 1;
        if (dst && kept >= 0) dx += Elem<T>::load(dst + (t.seq * (int64_t)(a.W - 1) + kept) * a.D + c);
        Elem<T>::store(static_cast<T*>(a.dx) + (seq0 + p) * a.D + c, dx);
    }
    float* part = a.part + tile * (a.W + 1) * a.D + c;
    for (int j = 0; j < a.W; ++j) part[j * a.D] = sw[j];
    part[a.W * a.D] = sb;
}

// ds0: positions -(W-1) .. -1 of each sequence
template <typename T>
__global__ __launch_bounds__(64) void conv_ds0_kernel(ConvLaunch a) {
    const int64_t nb = (a.D + 63) / 64, n = blockIdx.x / nb, c = (blockIdx.x - n * nb) * 64 + threadIdx.x;
    if (c >= a.D) return;
    const T *x = static_cast<const T*>(a.x), *s0 = static_cast<const T*>(a.s0);
    const T *dy = static_cast<const T*>(a.dy), *dst = static_cast<const T*>(a.dst);
    int64_t row0, len;
    conv_seq(a.map, n, &row0, &len);
    for (int r = 0; r < a.W - 1; ++r) {
        const int64_t p = r - (a.W - 1);
        float d = 0.f;
        for (int k = 1; k < a.W; ++k)
            if (p + k >= 0 && p + k < len)
                d += a.w[c * a.W + a.W - 1 - k] * Elem<T>::load(dy + (row0 + p + k) * a.ys + c) *
                     slope_of(a.silu, preact(a, x, s0, row0, n, p + k, c));
        if (dst && r - len >= 0) d += Elem<T>::load(dst + (n * (a.W - 1) + r - len) * a.D + c);
        Elem<T>::store(static_cast<T*>(a.ds0) + (n * (a.W - 1) + r) * a.D + c, d);
    }
}

__global__ __launch_bounds__(64) void conv_sum_kernel(ConvLaunch a) {
    const int64_t c = blockIdx.x * (int64_t)64 + threadIdx.x;
    const int j = blockIdx.y;
    if (c >= a.D) return;
    double s = 0;
    for (int64_t t = 0; t < a.map.max_tiles; ++t) s += a.part[(t * (a.W + 1) + j) * a.D + c];
    if (j < a.W)
        a.dw[c * a.W + j] = (float)s;
    else if (a.db)
        a.db[c] = (float)s;
}

template <typename T>
__global__ __launch_bounds__(64) void conv_step_kernel(ConvLaunch a) {
    const int64_t nb = (a.D + 63) / 64, n = blockIdx.x / nb, c = (blockIdx.x - n * nb) * 64 + threadIdx.x;
    if (c >= a.D) return;
    const int W = a.W;
    T* st = static_cast<T*>(a.st) + n * (W - 1) * a.D + c;
    const T xv = static_cast<const T*>(a.x)[n * a.xs + c];
    float z = a.b ? a.b[c] : 0.f;
    for (int j = 0; j < W - 1; ++j) z += a.w[c * W + j] * Elem<T>::load(st + j * a.D);
    z += a.w[c * W + W - 1] * Elem<T>::load(&xv);
    for (int j = 0; j + 1 < W - 1; ++j) st[j * a.D] = st[(j + 1) * a.D];
    st[(W - 2) * a.D] = xv;
    Elem<T>::store(static_cast<T*>(a.y) + n * a.ys + c, a.silu ? z * sigmoid_f(z) : z);
}

#define CONV_LAUNCH(KERNEL, GY)                                                                     \
    do {                                                                                            \
        const dim3 grid((unsigned)((a.D + 63) / 64 * (GY)));                             \
        if (a.bf16)                                                                                 \
            hipLaunchKernelGGL((KERNEL<bf16>), grid, dim3(64), 0, a.stream, a);                     \
        else                                                                                        \
            hipLaunchKernelGGL((KERNEL<float>), grid, dim3(64), 0, a.stream, a);                    \
        hipError_t e = hipGetLastError();                                                           \
        if (e != hipSuccess) return e;                                                              \
    } while (0)

hipError_t launch_conv_fwd(const ConvLaunch& a) {
    if (a.map.max_tiles > 0) CONV_LAUNCH(conv_fwd_kernel, a.map.max_tiles);
    if (a.st) CONV_LAUNCH(conv_window_kernel, a.map.N);
    return hipSuccess;
}

hipError_t launch_conv_bwd(const ConvLaunch& a) {
    if (a.map.max_tiles > 0) CONV_LAUNCH(conv_bwd_kernel, a.map.max_tiles);
    if (a.ds0) CONV_LAUNCH(conv_ds0_kernel, a.map.N);
    hipLaunchKernelGGL(conv_sum_kernel, dim3((unsigned)((a.D + 63) / 64), (unsigned)(a.W + 1)), dim3(64), 0,
                       a.stream, a);
    return hipGetLastError();
}

hipError_t launch_conv_step(const ConvLaunch& a) {
    CONV_LAUNCH(conv_step_kernel, a.map.N);
    return hipSuccess;
}

}  // namespace gdn
