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
//
// Measured (bf16, W = 4, SiLU): 4 x 4096 tokens of 6144 channels forward 81 us,
// 4.9 TB/s; 38 thousand packed tokens of 4096 channels forward 122 us (5.1
// TB/s, a large copy's rate), backward 228 us (4.1 TB/s: 183 us of bytes next to
// 172 us of ALU slots); one token of 256 sequences and 8192 channels 8 us (4.2 TB/s).
#include "gdn_layer.hpp"

namespace gdn {

// V consecutive elements of a row as loaded, at a byte offset
template <typename T, int V> struct Few;
template <> struct Few<bf16, 4> {
    u32x2 r;
    __device__ __forceinline__ void load(const bf16* row, unsigned off) { r = peek_row<u32x2>(row, off); }
    __device__ __forceinline__ void zero() { r = u32x2{0, 0}; }
    __device__ __forceinline__ float get(int e) const {
        const uint32_t w = e < 2 ? r.x : r.y;
        return __uint_as_float(e & 1 ? w & 0xffff0000u : w << 16);
    }
    __device__ __forceinline__ static void store(bf16* row, unsigned off, const float* f) {
        poke_row<u32x2>(row, off, u32x2{pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3])});
    }
};
template <> struct Few<float, 4> {
    f32x4 r;
    __device__ __forceinline__ void load(const float* row, unsigned off) { r = peek_row<f32x4>(row, off); }
    __device__ __forceinline__ void zero() { r = zero4(); }
    __device__ __forceinline__ float get(int e) const { return r[e]; }
    __device__ __forceinline__ static void store(float* row, unsigned off, const float* f) {
        poke_row<f32x4>(row, off, f32x4{f[0], f[1], f[2], f[3]});
    }
};
template <> struct Few<bf16, 1> {
    uint32_t r;
    __device__ __forceinline__ void load(const bf16* row, unsigned off) { r = peek_row<uint16_t>(row, off); }
    __device__ __forceinline__ void zero() { r = 0; }
    __device__ __forceinline__ float get(int) const { return __uint_as_float(r << 16); }
    __device__ __forceinline__ static void store(bf16* row, unsigned off, const float* f) {
        poke_row<uint16_t>(row, off, f32_to_bf16(f[0]));
    }
};
template <> struct Few<float, 1> {
    float r;
    __device__ __forceinline__ void load(const float* row, unsigned off) { r = peek_row<float>(row, off); }
    __device__ __forceinline__ void zero() { r = 0.f; }
    __device__ __forceinline__ float get(int) const { return r; }
    __device__ __forceinline__ static void store(float* row, unsigned off, const float* f) {
        poke_row<float>(row, off, f[0]);
    }
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
__device__ __forceinline__ void history(const ConvLaunch& a, const Tile& t, unsigned off, float (*h)[V]) {
    const T *x = static_cast<const T*>(a.x), *s0 = static_cast<const T*>(a.s0);
    const int64_t p0 = (int64_t)t.j * a.map.tile;
#pragma unroll
    for (int j = 0; j < W - 1; ++j) {
        Few<T, V> f;
        const int64_t back = W - 1 - j;
        if (p0 >= back) f.load(in_scalar(x + (t.row0 - back) * a.xs), off);
        else if (s0) f.load(in_scalar(s0 + (t.seq * (int64_t)(W - 1) + p0 + j) * a.D), off);
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

// The waves past the tiles' take a sequence each: one without a token hands its
// window through (forward st = s0, backward ds0 = dst).
template <typename T, int W, int V>
__device__ __forceinline__ void hand_through(const ConvLaunch& a, int64_t n, const T* from, T* to, unsigned off) {
    if (!to || n >= a.map.N) return;
    const int len = a.map.seqs ? __builtin_amdgcn_readfirstlane(a.map.seqs[n].y) : (int)a.map.T;
    if (len > 0) return;
#pragma unroll
    for (int j = 0; j < W - 1; ++j) {
        const int64_t row = (n * (W - 1) + j) * a.D;
        Few<T, V> f;
        if (from) f.load(in_scalar(from + row), off);
        else f.zero();
        float v[V];
#pragma unroll
        for (int e = 0; e < V; ++e) v[e] = f.get(e);
        Few<T, V>::store(in_scalar(to + row), off, v);
    }
}

template <typename T, int W, int V, bool SILU>
__device__ __forceinline__ void fwd_token(const ConvLaunch& a, const Taps<W, V>& k, float (*h)[V], const Few<T, V>& in,
                                          T* y, unsigned off) {
    float v[V], z[V];
#pragma unroll
    for (int e = 0; e < V; ++e) v[e] = in.get(e);
    preact<W, V>(k, h, v, z);
    push<W, V>(h, v);
    if (SILU)
#pragma unroll
        for (int e = 0; e < V; ++e) z[e] *= sigmoid_hw(z[e]);
    Few<T, V>::store(in_scalar(y), off, z);
}

template <typename T, int W, int V, bool SILU>
__global__ __launch_bounds__(256) void conv_fwd_kernel(ConvLaunch a) {
    constexpr int U = 8;
    // four neighbouring channel blocks of a tile to a workgroup: whole rows of 2 KB
    const unsigned nb = (unsigned)((a.D + 64 * V - 1) / (64 * V)), k0 = blockIdx.x * 4 + wave_id(), tile = k0 / nb;
    const int64_t c = ((int64_t)(k0 - tile * nb) * 64 + (threadIdx.x & 63)) * V;
    if (c >= a.D) return;
    const unsigned off = (unsigned)c * sizeof(T);
    if (tile >= a.map.max_tiles) {
        hand_through<T, W, V>(a, tile - a.map.max_tiles, static_cast<const T*>(a.s0), static_cast<T*>(a.st), off);
        return;
    }
    const Tile t = tile_of(a.map, tile);
    if (t.n <= 0) return;
    const T* x = static_cast<const T*>(a.x) + t.row0 * a.xs;
    T* y = static_cast<T*>(a.y) + t.row0 * a.ys;
    Few<T, V> next[U];
#pragma unroll
    for (int u = 0; u < U; ++u) next[u].load(in_scalar(x + (int64_t)min(u, t.n - 1) * a.xs), off);
    Taps<W, V> k;
    k.load(a, c);
    float h[W - 1][V];
    history<T, W, V>(a, t, off, h);
    for (int i0 = 0; i0 < t.n; i0 += U) {
        Few<T, V> now[U];
#pragma unroll
        for (int u = 0; u < U; ++u) now[u] = next[u];
        if (i0 + U < t.n) {
#pragma unroll
            for (int u = 0; u < U; ++u) next[u].load(in_scalar(x + (int64_t)min(i0 + U + u, t.n - 1) * a.xs), off);
        }
        // whole batches without a condition inside: the window then moves on by renaming
        // registers, where a branch in between costs a move for each of them
        if (i0 + U <= t.n) {
#pragma unroll
            for (int u = 0; u < U; ++u) fwd_token<T, W, V, SILU>(a, k, h, now[u], y + (i0 + u) * a.ys, off);
        } else {
            for (int u = 0; u < t.n - i0; ++u) {
                Few<T, V> one;
                one.load(in_scalar(x + (int64_t)(i0 + u) * a.xs), off);
                fwd_token<T, W, V, SILU>(a, k, h, one, y + (i0 + u) * a.ys, off);
            }
        }
    }
    if (a.st && t.j + 1 == t.nt)
#pragma unroll
        for (int j = 0; j < W - 1; ++j)
            Few<T, V>::store(in_scalar(static_cast<T*>(a.st) + (t.seq * (int64_t)(W - 1) + j) * a.D), off, h[j]);
}

// One token of the backward's walk: dz of it (LIVE: it is a token of the
// sequence), its terms of the weights' sums (OWN: of the tile).
template <typename T, int W, int V, bool SILU>
__device__ __forceinline__ void bwd_token(const Taps<W, V>& k, float (*h)[V], float (*dz)[V], const Few<T, V>& in,
                                          const Few<T, V>& din, bool live, bool own, float (*sw)[V], float* sb) {
#pragma unroll
    for (int j = 0; j + 1 < W; ++j)
#pragma unroll
        for (int e = 0; e < V; ++e) dz[j][e] = dz[j + 1][e];
    if (!live) {
#pragma unroll
        for (int e = 0; e < V; ++e) dz[W - 1][e] = 0.f;
        return;
    }
    float v[V], z[V];
#pragma unroll
    for (int e = 0; e < V; ++e) v[e] = in.get(e);
    preact<W, V>(k, h, v, z);
#pragma unroll
    for (int e = 0; e < V; ++e) {
        float d = din.get(e);
        if (SILU) {
            const float s = sigmoid_hw(z[e]);
            d *= s * (1.f + z[e] * (1.f - s));
        }
        dz[W - 1][e] = d;
    }
    if (own)
#pragma unroll
        for (int e = 0; e < V; ++e) {
            const float d = dz[W - 1][e];
            sb[e] += d;
#pragma unroll
            for (int j = 0; j < W - 1; ++j) sw[j][e] += d * h[j][e];
            sw[W - 1][e] += d * v[e];
        }
    push<W, V>(h, v);
}
template <int W, int V> __device__ __forceinline__ void dx_of(const Taps<W, V>& k, float (*dz)[V], float* o) {
#pragma unroll
    for (int e = 0; e < V; ++e) {
        o[e] = 0.f;
#pragma unroll
        for (int j = 0; j < W; ++j) o[e] += k.w[W - 1 - j][e] * dz[j][e];
    }
}

// the tile's tokens; sw, sb: its sums for the weights and the bias
template <typename T, int W, int V, bool SILU>
__device__ __forceinline__ void bwd_tile(const ConvLaunch& a, const Tile& t, int64_t c, float (*sw)[V], float* sb) {
    constexpr int U = 4;            // batches of 8 take it past three waves to a SIMD: 228 -> 244 us
    // tokens of the sequence from this tile's first on; of them the tile and W - 1 more
    const int64_t len = t.len, p0 = (int64_t)t.j * a.map.tile;
    const int left = (int)min(len - p0, (int64_t)t.n + W - 1), all = t.n + W - 1;
    // tokens whose dx takes nothing from the final window's gradient
    const int plain = a.dst ? (int)min(len - p0, (int64_t)t.n + W - 1) : all;
    const unsigned off = (unsigned)c * sizeof(T);
    const T* x = static_cast<const T*>(a.x) + t.row0 * a.xs;
    const T* dy = static_cast<const T*>(a.dy) + t.row0 * a.ys;
    const T* dst = static_cast<const T*>(a.dst);
    T* dx = static_cast<T*>(a.dx) + t.row0 * a.D;
    Few<T, V> nx[U], nd[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        nx[u].load(in_scalar(x + (int64_t)min(u, left - 1) * a.xs), off);
        nd[u].load(in_scalar(dy + (int64_t)min(u, left - 1) * a.ys), off);
    }
    Taps<W, V> k;
    k.load(a, c);
    float h[W - 1][V], dz[W][V];      // dz of the last W tokens, oldest first
    history<T, W, V>(a, t, off, h);
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
                nx[u].load(in_scalar(x + (int64_t)min(i0 + U + u, left - 1) * a.xs), off);
                nd[u].load(in_scalar(dy + (int64_t)min(i0 + U + u, left - 1) * a.ys), off);
            }
        }
        // a batch inside the tile, away from its ends: no condition inside (see the forward)
        if (i0 >= U && i0 + U <= t.n && i0 + U <= plain) {
#pragma unroll
            for (int u = 0; u < U; ++u) {
                float o[V];
                bwd_token<T, W, V, SILU>(k, h, dz, cx[u], cd[u], true, true, sw, sb);
                dx_of<W, V>(k, dz, o);
                Few<T, V>::store(in_scalar(dx + (i0 + u - (W - 1)) * a.D), off, o);
            }
            continue;
        }
        for (int u = 0; u < min(U, all - i0); ++u) {
            const int i = i0 + u, q = i - (W - 1);   // dx of token q is complete; before a sequence's start: of its window
            Few<T, V> one, done;
            one.load(in_scalar(x + (int64_t)min(i, left - 1) * a.xs), off);
            done.load(in_scalar(dy + (int64_t)min(i, left - 1) * a.ys), off);
            bwd_token<T, W, V, SILU>(k, h, dz, one, done, i < left, i < t.n, sw, sb);
            if (q < 0 && (t.j > 0 || !a.ds0)) continue;
            float o[V];
            dx_of<W, V>(k, dz, o);
            const int64_t kept = p0 + q - len + W - 1;     // row of the final window that is this input
            if (dst && kept >= 0) {
                Few<T, V> f;
                f.load(in_scalar(dst + (t.seq * (int64_t)(W - 1) + kept) * a.D), off);
#pragma unroll
                for (int e = 0; e < V; ++e) o[e] += f.get(e);
            }
            if (q >= 0) Few<T, V>::store(in_scalar(dx + q * a.D), off, o);
            else Few<T, V>::store(in_scalar(static_cast<T*>(a.ds0) + (t.seq * (int64_t)(W - 1) + i) * a.D), off, o);
        }
    }
}

template <typename T, int W, int V, bool SILU>
__global__ __launch_bounds__(256) void conv_bwd_kernel(ConvLaunch a) {
    // four neighbouring tiles to a workgroup: their sums for the weights meet in LDS, a quarter
    // of the partial rows that a row to a tile would be
    __shared__ float s_sum[4][W + 1][64 * V];
    const unsigned nb = (unsigned)((a.D + 64 * V - 1) / (64 * V)), group = blockIdx.x / nb;
    const int64_t c0 = (int64_t)(blockIdx.x - group * nb) * 64 * V;
    const int w = wave_id(), lane = threadIdx.x & 63;
    const int64_t tile = (int64_t)group * 4 + w, c = c0 + lane * V;
    float sw[W][V], sb[V];
#pragma unroll
    for (int e = 0; e < V; ++e) {
        sb[e] = 0.f;
#pragma unroll
        for (int j = 0; j < W; ++j) sw[j][e] = 0.f;
    }
    const int64_t groups = (a.map.max_tiles + 3) / 4;
    if (group >= groups) {
        if (c < a.D)
            hand_through<T, W, V>(a, (group - groups) * 4 + w, static_cast<const T*>(a.dst), static_cast<T*>(a.ds0),
                                  (unsigned)c * sizeof(T));
        return;
    }
    if (tile < a.map.max_tiles && c < a.D) {
        const Tile t = tile_of(a.map, tile);
        if (t.n > 0) bwd_tile<T, W, V, SILU>(a, t, c, sw, sb);
    }
#pragma unroll
    for (int e = 0; e < V; ++e) {
#pragma unroll
        for (int j = 0; j < W; ++j) s_sum[w][j][lane * V + e] = sw[j][e];
        s_sum[w][W][lane * V + e] = sb[e];
    }
    __syncthreads();
    for (int i = threadIdx.x; i < (W + 1) * 64 * V; i += 256) {
        const int j = i / (64 * V), k = i - j * 64 * V;
        if (c0 + k < a.D)
            a.part[((int64_t)group * (W + 1) + j) * a.D + c0 + k] =
                (s_sum[0][j][k] + s_sum[1][j][k]) + (s_sum[2][j][k] + s_sum[3][j][k]);
    }
}

template <typename T, int W, int V, bool SILU>
__global__ __launch_bounds__(64) void conv_step_kernel(ConvLaunch a) {
    const int64_t nb = (a.D + 64 * V - 1) / (64 * V), n = blockIdx.x / nb;
    const int64_t c = ((blockIdx.x - n * nb) * 64 + threadIdx.x) * V;
    if (c >= a.D) return;
    const unsigned off = (unsigned)c * sizeof(T);
    T* st = static_cast<T*>(a.st) + n * (W - 1) * a.D;
    Few<T, V> in, win[W - 1];
    in.load(static_cast<const T*>(a.x) + n * a.xs, off);
#pragma unroll
    for (int j = 0; j < W - 1; ++j) win[j].load(st + j * a.D, off);
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
    for (int j = 0; j < W - 1; ++j) Few<T, V>::store(st + j * a.D, off, h[j]);
    Few<T, V>::store(static_cast<T*>(a.y) + n * a.ys, off, z);
}

// ---- launches
enum { FWD, BWD, STEP };
template <int WHICH, typename T, int W, int V, bool SILU>
static hipError_t go3(const ConvLaunch& a) {
    const int64_t nb = (a.D + 64 * V - 1) / (64 * V), tiles = a.map.max_tiles;
    const bool empties = a.map.seqs || a.map.T == 0;     // sequences without a token are possible
    if constexpr (WHICH == FWD)
        hipLaunchKernelGGL((conv_fwd_kernel<T, W, V, SILU>), 
                           dim3((unsigned)((nb * (tiles + (empties && a.st ? a.map.N : 0)) + 3) / 4)), dim3(256),
                           0, a.stream, a);
    else if constexpr (WHICH == BWD)
        hipLaunchKernelGGL((conv_bwd_kernel<T, W, V, SILU>), 
                           dim3((unsigned)(nb * ((tiles + 3) / 4 + (empties && a.ds0 ? (a.map.N + 3) / 4 : 0)))), dim3(256),
                           0, a.stream, a);
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

hipError_t launch_conv_fwd(const ConvLaunch& a) {
    if (a.map.max_tiles == 0 && !a.st) return hipSuccess;
    return go<FWD>(a);
}

hipError_t launch_conv_bwd(const ConvLaunch& a) {
    if (a.map.max_tiles > 0 || a.ds0) {
        hipError_t e = go<BWD>(a);
        if (e != hipSuccess) return e;
    }
    return launch_row_sum(RowSumLaunch{a.part, (a.map.max_tiles + 3) / 4, a.D, a.W, a.W + 1, a.dw, a.db, a.sums, a.stream});
}

hipError_t launch_conv_step(const ConvLaunch& a) { return go<STEP>(a); }

}  // namespace gdn
