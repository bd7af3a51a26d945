// Short causal depthwise convolution (width W in 2..4) with an optional SiLU,
// and its backward pass.
//
// A wave takes a tile of tokens and 64 V channels and walks the tokens with
// the last W - 1 inputs in registers; rows come in batches of U, the next
// batch's loads issued before the present one is worked on.  At a tile's
// start those inputs are read again (W - 1 rows more a tile, out of the
// cache), or come from the carried window at a sequence's start; at a
// sequence's end what the registers hold is the window to carry on.
//
// The backward walks the same way, W - 1 tokens past its tile: once dz of
// token p is known, dx of token p - W + 1 is complete.  A tile's sums for the
// weights stay in registers and are added up over the tiles afterwards, in a fixed order.
#include "gdn_layer.hpp"

namespace gdn {

// V consecutive elements as loaded
template <typename T, int V> struct Few;
template <> struct Few<bf16, 4> {
    uint2 r;
    __device__ __forceinline__ void load(const bf16* p) { r = *reinterpret_cast<const uint2*>(p); }
    __device__ __forceinline__ void zero() { r = make_uint2(0, 0); }
    __device__ __forceinline__ float get(int e) const {
        const uint32_t w = e < 2 ? r.x : r.y;
        return __uint_as_float(e & 1 ? w & 0xffff0000u : w << 16);
    }
    __device__ __forceinline__ static void store(bf16* p, const float* f) {
        *reinterpret_cast<uint2*>(p) = make_uint2(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]));
    }
};
template <> struct Few<float, 4> {
    float4 r;
    __device__ __forceinline__ void load(const float* p) { r = *reinterpret_cast<const float4*>(p); }
    __device__ __forceinline__ void zero() { r = make_float4(0.f, 0.f, 0.f, 0.f); }
    __device__ __forceinline__ float get(int e) const { return e == 0 ? r.x : e == 1 ? r.y : e == 2 ? r.z : r.w; }
    __device__ __forceinline__ static void store(float* p, const float* f) {
        *reinterpret_cast<float4*>(p) = make_float4(f[0], f[1], f[2], f[3]);
    }
};
template <typename T> struct Few<T, 1> {
    typename Elem<T>::Raw r;
    __device__ __forceinline__ void load(const T* p) { r = Elem<T>::load_raw(p); }
    __device__ __forceinline__ void zero() { r = 0; }
    __device__ __forceinline__ float get(int) const { return Elem<T>::from_raw(r); }
    __device__ __forceinline__ static void store(T* p, const float* f) { Elem<T>::store(p, f[0]); }
};

// 1 / (1 + exp(-z)) by the hardware's exp2 and reciprocal (1 unit in the last place each)
__device__ __forceinline__ float sigmoid_hw(float z) {
    return __builtin_amdgcn_rcpf(1.f + exp2_hw(-LOG2E * z));
}

// W, V: the taps and channels of a lane
template <int W, int V> struct Taps {
    float w[W][V], b[V];
    __device__ __forceinline__ void load(const ConvLaunch& a, int64_t c) {
#pragma unroll
        for (int e = 0; e < V; ++e) {
#pragma unroll
            for (int j = 0; j < W; ++j) w[j][e] = a.w[(c + e) * W + j];
            b[e] = a.b ? a.b[c + e] : 0.f;
        }
    }
};

// the W - 1 inputs before position p0 of sequence t.seq, oldest first
template <typename T, int W, int V>
__device__ __forceinline__ void history(const ConvLaunch& a, const Tile& t, int64_t c, float (*h)[V]) {
    const T *x = static_cast<const T*>(a.x), *s0 = static_cast<const T*>(a.s0);
    const int64_t p0 = (int64_t)t.j * a.map.tile;
#pragma unroll
    for (int j = 0; j < W - 1; ++j) {
        Few<T, V> f;
        const int64_t back = W - 1 - j;
        if (p0 >= back) f.load(x + (t.row0 - back) * a.xs + c);
        else if (s0) f.load(s0 + (t.seq * (W - 1) + p0 + j) * a.D + c);
        else f.zero();
#pragma unroll
        for (int e = 0; e < V; ++e) h[j][e] = f.get(e);
    }
}

template <int W, int V>
__device__ __forceinline__ void push(float (*h)[V], const float* v) {
#pragma unroll
    for (int j = 0; j + 1 < W - 1; ++j)
#pragma unroll
        for (int e = 0; e < V; ++e) h[j][e] = h[j + 1][e];
#pragma unroll
    for (int e = 0; e < V; ++e) h[W - 2][e] = v[e];
}

// z of the token whose input is v
template <int W, int V>
__device__ __forceinline__ void preact(const Taps<W, V>& k, float (*h)[V], const float* v, float* z) {
#pragma unroll
    for (int e = 0; e < V; ++e) {
        z[e] = k.b[e];
#pragma unroll
        for (int j = 0; j < W - 1; ++j) z[e] += k.w[j][e] * h[j][e];
        z[e] += k.w[W - 1][e] * v[e];
    }
}

// tile and first channel of this wave; false where it has none
template <int V>
__device__ __forceinline__ bool place(const ConvLaunch& a, Tile* t, int64_t* tile, int64_t* cl) {
    const unsigned nb = (unsigned)((a.D + 64 * V - 1) / (64 * V)), k = blockIdx.x * 4 + wave_id(), i = k / nb;
    if (i >= a.map.max_tiles) return false;
    *t = tile_of(a.map, i);
    *tile = i;
    *cl = ((int64_t)(k - i * nb) * 64 + (threadIdx.x & 63)) * V;
    return true;
}

template <typename T, int W, int V, bool SILU>
__global__ __launch_bounds__(256) void conv_fwd_kernel(ConvLaunch a) {
    constexpr int U = 8;
    Tile t;
    int64_t tile, c;
    if (!place<V>(a, &t, &tile, &c) || t.n <= 0 || c >= a.D) return;
    const T* x = static_cast<const T*>(a.x) + t.row0 * a.xs + c;
    T* y = static_cast<T*>(a.y) + t.row0 * a.ys + c;
    Few<T, V> next[U];
#pragma unroll
    for (int u = 0; u < U; ++u) next[u].load(x + (int64_t)min(u, t.n - 1) * a.xs);
    Taps<W, V> k;
    k.load(a, c);
    float h[W - 1][V];
    history<T, W, V>(a, t, c, h);
    for (int i0 = 0; i0 < t.n; i0 += U) {
        Few<T, V> now[U];
#pragma unroll
        for (int u = 0; u < U; ++u) now[u] = next[u];
        if (i0 + U < t.n) {
#pragma unroll
            for (int u = 0; u < U; ++u) next[u].load(x + (int64_t)min(i0 + U + u, t.n - 1) * a.xs);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (i0 + u >= t.n) break;
            float v[V], z[V];
#pragma unroll
            for (int e = 0; e < V; ++e) v[e] = now[u].get(e);
            preact<W, V>(k, h, v, z);
            push<W, V>(h, v);
            if (SILU)
#pragma unroll
                for (int e = 0; e < V; ++e) z[e] *= sigmoid_hw(z[e]);
            Few<T, V>::store(y + (i0 + u) * a.ys, z);
        }
    }
    if (a.st && t.j + 1 == t.nt)
#pragma unroll
        for (int j = 0; j < W - 1; ++j)
            Few<T, V>::store(static_cast<T*>(a.st) + (t.seq * (int64_t)(W - 1) + j) * a.D + c, h[j]);
}

template <typename T, int W, int V, bool SILU>
__global__ __launch_bounds__(256) void conv_bwd_kernel(ConvLaunch a) {
    constexpr int U = 8;
    Tile t;
    int64_t tile, c;
    if (!place<V>(a, &t, &tile, &c) || c >= a.D) return;
    float sw[W][V], sb[V];
#pragma unroll
    for (int e = 0; e < V; ++e) {
        sb[e] = 0.f;
#pragma unroll
        for (int j = 0; j < W; ++j) sw[j][e] = 0.f;
    }
    if (t.n > 0) {
        // tokens of the sequence from this tile's first on; of them the tile and W - 1 more
        const int64_t len = t.len, p0 = (int64_t)t.j * a.map.tile;
        const int left = (int)min(len - p0, (int64_t)t.n + W - 1), all = t.n + W - 1;
        const T* x = static_cast<const T*>(a.x) + t.row0 * a.xs + c;
        const T* dy = static_cast<const T*>(a.dy) + t.row0 * a.ys + c;
        const T* dst = static_cast<const T*>(a.dst);
        T* dx = static_cast<T*>(a.dx) + t.row0 * a.D + c;
        Few<T, V> nx[U], nd[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            nx[u].load(x + (int64_t)min(u, left - 1) * a.xs);
            nd[u].load(dy + (int64_t)min(u, left - 1) * a.ys);
        }
        Taps<W, V> k;
        k.load(a, c);
        float h[W - 1][V], dz[W][V];      // dz of the last W tokens, oldest first
        history<T, W, V>(a, t, c, h);
#pragma unroll
        for (int j = 0; j < W; ++j)
#pragma unroll
            for (int e = 0; e < V; ++e) dz[j][e] = 0.f;
        for (int i0 = 0; i0 < all; i0 += U) {
            Few<T, V> cx[U], cd[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                cx[u] = nx[u];
                cd[u] = nd[u];
            }
            if (i0 + U < left) {
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    nx[u].load(x + (int64_t)min(i0 + U + u, left - 1) * a.xs);
                    nd[u].load(dy + (int64_t)min(i0 + U + u, left - 1) * a.ys);
                }
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int i = i0 + u;
                if (i >= all) break;
#pragma unroll
                for (int j = 0; j + 1 < W; ++j)
#pragma unroll
                    for (int e = 0; e < V; ++e) dz[j][e] = dz[j + 1][e];
                if (i < left) {
                    float v[V], z[V];
#pragma unroll
                    for (int e = 0; e < V; ++e) v[e] = cx[u].get(e);
                    preact<W, V>(k, h, v, z);
#pragma unroll
                    for (int e = 0; e < V; ++e) {
                        float d = cd[u].get(e);
                        if (SILU) {
                            const float s = sigmoid_hw(z[e]);
                            d *= s * (1.f + z[e] * (1.f - s));
                        }
                        dz[W - 1][e] = d;
                        if (i < t.n) {     // the tile's own token
                            sb[e] += d;
#pragma unroll
                            for (int j = 0; j < W - 1; ++j) sw[j][e] += d * h[j][e];
                            sw[W - 1][e] += d * v[e];
                        }
                    }
                    push<W, V>(h, v);
                } else {
#pragma unroll
                    for (int e = 0; e < V; ++e) dz[W - 1][e] = 0.f;
                }
                // dx of token q = i - (W - 1) of the tile; before a sequence's start: of its window
                const int q = i - (W - 1);
                if (q < 0 && (t.j > 0 || !a.ds0)) continue;
                float o[V];
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    o[e] = 0.f;
#pragma unroll
                    for (int j = 0; j < W; ++j) o[e] += k.w[W - 1 - j][e] * dz[j][e];
                }
                const int64_t kept = p0 + q - len + W - 1;     // row of the final window that is this input
                if (dst && kept >= 0) {
                    Few<T, V> f;
                    f.load(dst + (t.seq * (int64_t)(W - 1) + kept) * a.D + c);
#pragma unroll
                    for (int e = 0; e < V; ++e) o[e] += f.get(e);
                }
                if (q >= 0) Few<T, V>::store(dx + q * a.D, o);
                else Few<T, V>::store(static_cast<T*>(a.ds0) + (t.seq * (int64_t)(W - 1) + i) * a.D + c, o);
            }
        }
    }
    float* part = a.part + tile * (W + 1) * a.D + c;
#pragma unroll
    for (int j = 0; j < W; ++j) Few<float, V>::store(part + j * a.D, sw[j]);
    Few<float, V>::store(part + W * a.D, sb);
}

// dweight and dbias: the tiles' sums, 16 strands of tiles per channel, in 64 bits
__global__ __launch_bounds__(1024) void conv_sum_kernel(ConvLaunch a) {
    __shared__ double s[16][64];
    const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
    const int64_t nb = (a.D + 63) / 64, j = blockIdx.x / nb, c = (blockIdx.x - j * nb) * 64 + lane;
    double v = 0;
    if (c < a.D)
        for (int64_t i = w; i < a.map.max_tiles; i += 16) v += a.part[(i * (a.W + 1) + j) * a.D + c];
    s[w][lane] = v;
    __syncthreads();
    if (w != 0 || c >= a.D) return;
    for (int i = 1; i < 16; ++i) v += s[i][lane];
    if (j < a.W) a.dw[c * a.W + j] = (float)v;
    else a.db[c] = (float)v;
}

// sequences without a token hand their window through: fwd st = s0, bwd ds0 = dst
template <typename T>
__global__ __launch_bounds__(256) void conv_empty_kernel(ConvLaunch a, const T* from, T* to) {
    const int64_t row = (a.W - 1) * a.D, nb = (row + 255) / 256, n = blockIdx.x / nb;
    const int64_t i = (blockIdx.x - n * nb) * 256 + threadIdx.x;
    if (i >= row || (a.map.seqs ? a.map.seqs[n].y : a.map.T) > 0) return;
    if (from) to[n * row + i] = from[n * row + i];
    else Elem<T>::store(to + n * row + i, 0.f);
}

template <typename T, int W, int V, bool SILU>
__global__ __launch_bounds__(64) void conv_step_kernel(ConvLaunch a) {
    const int64_t nb = (a.D + 64 * V - 1) / (64 * V), n = blockIdx.x / nb;
    const int64_t c = ((blockIdx.x - n * nb) * 64 + threadIdx.x) * V;
    if (c >= a.D) return;
    T* st = static_cast<T*>(a.st) + n * (W - 1) * a.D + c;
    Few<T, V> in, win[W - 1];
    in.load(static_cast<const T*>(a.x) + n * a.xs + c);
#pragma unroll
    for (int j = 0; j < W - 1; ++j) win[j].load(st + j * a.D);
    Taps<W, V> k;
    k.load(a, c);
    float h[W - 1][V], v[V], z[V];
#pragma unroll
    for (int e = 0; e < V; ++e) {
        v[e] = in.get(e);
#pragma unroll
        for (int j = 0; j < W - 1; ++j) h[j][e] = win[j].get(e);
    }
    preact<W, V>(k, h, v, z);
    push<W, V>(h, v);
    if (SILU)
#pragma unroll
        for (int e = 0; e < V; ++e) z[e] *= sigmoid_hw(z[e]);
#pragma unroll
    for (int j = 0; j < W - 1; ++j) Few<T, V>::store(st + j * a.D, h[j]);
    Few<T, V>::store(static_cast<T*>(a.y) + n * a.ys + c, z);
}

// ---- launches
enum { FWD, BWD, STEP };
template <int WHICH, typename T, int W, int V, bool SILU>
static hipError_t go3(const ConvLaunch& a) {
    const int64_t nb = (a.D + 64 * V - 1) / (64 * V);
    const dim3 grid((unsigned)((nb * a.map.max_tiles + 3) / 4));
    if constexpr (WHICH == FWD)
        hipLaunchKernelGGL((conv_fwd_kernel<T, W, V, SILU>), grid, dim3(256), 0, a.stream, a);
    else if constexpr (WHICH == BWD)
        hipLaunchKernelGGL((conv_bwd_kernel<T, W, V, SILU>), grid, dim3(256), 0, a.stream, a);
    else
        hipLaunchKernelGGL((conv_step_kernel<T, W, V, SILU>), dim3((unsigned)(nb * a.map.N)), dim3(64), 0, a.stream, a);
    return hipGetLastError();
}
template <int WHICH, typename T, int V, bool SILU>
static hipError_t go2(const ConvLaunch& a) {
    return a.W == 2 ? go3<WHICH, T, 2, V, SILU>(a)
                    : a.W == 3 ? go3<WHICH, T, 3, V, SILU>(a) : go3<WHICH, T, 4, V, SILU>(a);
}
template <int WHICH, typename T>
static hipError_t go1(const ConvLaunch& a, bool four) {
    if (four) return a.silu ? go2<WHICH, T, 4, true>(a) : go2<WHICH, T, 4, false>(a);
    return a.silu ? go2<WHICH, T, 1, true>(a) : go2<WHICH, T, 1, false>(a);
}
// Four channels to a lane where every row and pointer allows them.
template <int WHICH>
static hipError_t go(const ConvLaunch& a) {
    const uintptr_t p = (uintptr_t)a.x | (uintptr_t)a.y | (uintptr_t)a.dy | (uintptr_t)a.dx | (uintptr_t)a.s0 |
                        (uintptr_t)a.st | (uintptr_t)a.dst | (uintptr_t)a.ds0;
    const bool four = ((a.D | a.xs | a.ys) & 3) == 0 && p % (a.bf16 ? 8 : 16) == 0;
    return a.bf16 ? go1<WHICH, bf16>(a, four) : go1<WHICH, float>(a, four);
}

static hipError_t empty(const ConvLaunch& a, const void* from, void* to) {
    if (!to || (!a.map.seqs && a.map.T > 0)) return hipSuccess;
    const dim3 grid((unsigned)(((a.W - 1) * a.D + 255) / 256 * a.map.N));
    if (a.bf16)
        hipLaunchKernelGGL((conv_empty_kernel<bf16>), grid, dim3(256), 0, a.stream, a, static_cast<const bf16*>(from),
                           static_cast<bf16*>(to));
    else
        hipLaunchKernelGGL((conv_empty_kernel<float>), grid, dim3(256), 0, a.stream, a,
                           static_cast<const float*>(from), static_cast<float*>(to));
    return hipGetLastError();
}

hipError_t launch_conv_fwd(const ConvLaunch& a) {
    hipError_t e = empty(a, a.s0, a.st);
    if (e != hipSuccess || a.map.max_tiles == 0) return e;
    return go<FWD>(a);
}

hipError_t launch_conv_bwd(const ConvLaunch& a) {
    hipError_t e = empty(a, a.dst, a.ds0);
    if (e != hipSuccess) return e;
    if (a.map.max_tiles > 0 && (e = go<BWD>(a)) != hipSuccess) return e;
    hipLaunchKernelGGL(conv_sum_kernel, dim3((unsigned)((a.D + 63) / 64 * (a.W + (a.db ? 1 : 0)))), dim3(1024), 0,
                       a.stream, a);
    return hipGetLastError();
}

hipError_t launch_conv_step(const ConvLaunch& a) { return go<STEP>(a); }

}  // namespace gdn
