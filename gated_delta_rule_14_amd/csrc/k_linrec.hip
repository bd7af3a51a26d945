// Gated linear recurrence over channels: h_t = a_t h_{t-1} + u_t, a = exp(g),
// u = x or sqrt(1 - a^2) x, and its backward pass.
//
// The recurrence is a composition of affine maps, so a stretch of tokens is a
// pair (A, H): h_out = A h_in + H.  One workgroup takes a tile of tokens and
// CB channels: each wave holds S consecutive tokens of the tile in registers
// and reduces them to a pair; the pairs of the waves meet in LDS, the pair of
// the tile is published in the workspace, and the state entering the tile is
// put together from the pairs of the sequence's earlier tiles.  x and g are
// read once and y is written once.
//
// The pairs are published without waiting for anything, so a tile waits for
// one hand-off only, not for a chain of them.  Sixteen tiles form a group whose last
// tile publishes the group's pair too (after reading the other fifteen): a
// tile reads at most 15 pairs of its own group and one of every group before.  They are
// composed in the order of the tokens, whatever order they arrive in, so
// equal calls give equal bits.  A pair is one 64-bit word, stored and loaded
// by relaxed agent-scope atomics: it is there whole or not at all, so no
// fence and no flag is needed; "not there" is a NaN pattern of A that is
// never published, set by a kernel in front.
//
// Workgroups take their tile from a ticket counter, tiles in the order they
// wait for each other: every tile that one waits for belongs to a workgroup
// that is already running and that publishes without a wait (a group's pair:
// after waits of that kind), so every wait ends.  Each is bounded all the
// same and reports in words[1].
#include "gdn_layer.hpp"

namespace gdn {

constexpr int GROUP = 16;
constexpr unsigned ABSENT = 0xffffffffu;     // never the bits of a published A
constexpr int POLLS = 1 << 20;               // about a second; a hand-off takes microseconds

// ---- gates
// All of the gate's functions come from the hardware's exp2, reciprocal and
// square root (1 unit in the last place each) and series that hold the
// leading bits where the direct formula cancels.
__device__ __forceinline__ float rcp_hw(float x) { return __builtin_amdgcn_rcpf(x); }
__device__ __forceinline__ float sqrt_hw(float x) { return __builtin_amdgcn_sqrtf(x); }

// log1p(e), 0 <= e <= 1: 2 artanh(s), s = e / (2 + e) <= 1/3; the first term
// left out is s^16/17 < 2e-9 of the sum
__device__ __forceinline__ float log1p_unit(float e) {
    const float s = e * rcp_hw(2.f + e), q = s * s;
    float p = 1.f / 15.f;
    p = p * q + 1.f / 13.f;
    p = p * q + 1.f / 11.f;
    p = p * q + 1.f / 9.f;
    p = p * q + 1.f / 7.f;
    p = p * q + 1.f / 5.f;
    p = p * q + 1.f / 3.f;
    return 2.f * s + 2.f * s * (q * p);
}

// 1 - exp(t) for t <= 0, et = exp(t): the series of -expm1 above -0.35, where
// 1 - et would cancel (first term left out: t^7/8! < 2e-8 of the sum)
__device__ __forceinline__ float one_minus_exp(float t, float et) {
    float p = 1.f / 5040.f;
    p = p * t + 1.f / 720.f;
    p = p * t + 1.f / 120.f;
    p = p * t + 1.f / 24.f;
    p = p * t + 1.f / 6.f;
    p = p * t + 0.5f;
    p = p * t + 1.f;
    return t > -0.35f ? -t * p : 1.f - et;
}

constexpr float LN2 = 0.6931471805599453f;

struct Gate {
    float la;      // log a
    float a;
    float m;       // factor of x
    float sg;      // sigmoid(g + bias): d log a / d g = rate sg
};
// rate2 = -exp(A_log) log2(e)
template <bool ACT, bool NORM, bool BWD>
__device__ __forceinline__ Gate gate_of(float g, float rate2, float bias) {
    Gate r;
    float l2;
    r.sg = 0.f;
    if (ACT) {
        const float z = g + bias, e = exp2_hw(-LOG2E * fabsf(z));
        l2 = rate2 * (fmaxf(z, 0.f) + log1p_unit(e));
        if (BWD) r.sg = (z >= 0.f ? 1.f : e) * rcp_hw(1.f + e);
        r.la = LN2 * l2;
    } else {
        l2 = g * LOG2E;
        r.la = g;
    }
    r.a = exp2_hw(l2);
    r.m = NORM ? sqrt_hw(fmaxf(one_minus_exp(2.f * r.la, r.a * r.a), 0.f)) : 1.f;
    return r;
}

// ---- V consecutive elements as loaded, and their floats
template <typename T, int V> struct Raw;
template <> struct Raw<bf16, 1> {
    uint32_t r;
    __device__ __forceinline__ void load(const bf16* p) { r = p->bits; }
    __device__ __forceinline__ float get(int) const { return __uint_as_float(r << 16); }
    __device__ __forceinline__ static void store(bf16* p, const float* f) { p->bits = f32_to_bf16(f[0]); }
};
template <> struct Raw<bf16, 2> {
    uint32_t r;
    __device__ __forceinline__ void load(const bf16* p) { r = *reinterpret_cast<const uint32_t*>(p); }
    __device__ __forceinline__ float get(int e) const {
        return __uint_as_float(e ? r & 0xffff0000u : r << 16);
    }
    __device__ __forceinline__ static void store(bf16* p, const float* f) {
        *reinterpret_cast<uint32_t*>(p) = pack_bf16x2(f[0], f[1]);
    }
};
template <> struct Raw<float, 1> {
    float r;
    __device__ __forceinline__ void load(const float* p) { r = *p; }
    __device__ __forceinline__ float get(int) const { return r; }
    __device__ __forceinline__ static void store(float* p, const float* f) { *p = f[0]; }
};
template <> struct Raw<float, 2> {
    float2 r;
    __device__ __forceinline__ void load(const float* p) { r = *reinterpret_cast<const float2*>(p); }
    __device__ __forceinline__ float get(int e) const { return e ? r.y : r.x; }
    __device__ __forceinline__ static void store(float* p, const float* f) {
        *reinterpret_cast<float2*>(p) = make_float2(f[0], f[1]);
    }
};

// ---- the published pairs
__device__ __forceinline__ void publish(uint64_t* p, float A, float H) {
    const unsigned a = A != A ? 0x7fc00000u : __float_as_uint(A);
    __hip_atomic_store(p, (uint64_t)__float_as_uint(H) << 32 | a, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ uint64_t peek(const uint64_t* p) {
    return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

// Compose the pairs at p, p + step, ... (n of them) in that order onto (A, H).
// `polls`: what is left of this thread's patience; 0 once a wait gave up.
__device__ __forceinline__ void compose(const uint64_t* p, int64_t step, int n, float* A, float* H, int* polls) {
    for (int i = 0; i < n; i += 8) {
        uint64_t v[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) v[k] = i + k < n ? peek(p + (i + k) * step) : 0;
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            if (i + k >= n) break;
            while ((unsigned)v[k] == ABSENT && *polls > 0) {
                --*polls;
                __builtin_amdgcn_s_sleep(1);
                v[k] = peek(p + (i + k) * step);
            }
            const float a = __uint_as_float((unsigned)v[k]);
            *H = a * *H + __uint_as_float((unsigned)(v[k] >> 32));
            *A *= a;
        }
    }
}

// The value entering tile j (of nt) of a sequence, for channel c, out of what
// the tiles before it publish; `tile` its row in the workspace, dir = 1 for
// tiles in the order of the tokens, -1 against it (j then counts from the
// sequence's end).  (A, H): the tile's own pair, published here.  The first
// tile's pair is published with the value `start` that enters the sequence
// worked in, as is its group's: those are values, and replace what is composed so far.
__device__ __forceinline__ float enter(const LinrecLaunch& p, int64_t tile, int j, int nt, int dir, int64_t c,
                                       float A, float H, float start) {
    uint64_t* const one = p.pairs + tile * p.D + c;
    const bool followed = j + 1 < nt;
    if (j == 0) {
        if (followed) publish(one, 0.f, A * start + H);
        return start;
    }
    if (followed) publish(one, A, H);
    int polls = POLLS;
    const int ng = j / GROUP, in = j - ng * GROUP;
    float v = 0.f, gA = 1.f, gH = 0.f;
    if (ng > 0) {
        // rows of the groups' last tiles: 16 tiles apart, so a sixteenth of the row is their own
        const int64_t last0 = tile + (int64_t)dir * (GROUP - 1 - j);
        for (int g = 0; g < ng; ++g) {
            const uint64_t* q = p.groups + ((last0 + (int64_t)dir * g * GROUP) / GROUP) * p.D + c;
            float a = 1.f, h = 0.f;
            compose(q, 0, 1, &a, &h, &polls);
            v = g == 0 ? h : a * v + h;
        }
    }
    compose(one - (int64_t)dir * in * p.D, (int64_t)dir * p.D, in, &gA, &gH, &polls);
    if (in == GROUP - 1 && followed)
        publish(p.groups + (tile / GROUP) * p.D + c, ng == 0 ? 0.f : gA * A, A * gH + H);
    if (polls == 0) atomicExch(p.words + 1, 1);
    // without a group before, the first of the pairs above was the first tile's value (A = 0)
    return ng == 0 ? gH : gA * v + gH;
}

// Every pair that some tile reads is marked absent, the ticket and the words cleared.
__global__ __launch_bounds__(256) void linrec_clear_kernel(LinrecLaunch p) {
    const int64_t nb = (p.D + 255) / 256, tile = blockIdx.x / nb, c = (blockIdx.x - tile * nb) * 256 + threadIdx.x;
    if (blockIdx.x == 0 && threadIdx.x == 0) {
        if (!p.map.table) p.words[0] = 0;
        p.words[1] = 0;
        p.words[2] = 0;
    }
    if (c >= p.D) return;
    const Tile t = tile_of(p.map, tile);
    if (t.n > 0 && t.nt > 1) {
        p.pairs[tile * p.D + c] = ABSENT;
        if (t.nt > GROUP) p.groups[(tile / GROUP) * p.D + c] = ABSENT;
    }
}

// tile and channel block of this workgroup: by ticket where tiles wait for each other
__device__ __forceinline__ unsigned ticket_of(const LinrecLaunch& p, unsigned* s) {
    if (!p.pairs) return blockIdx.x;
    if (threadIdx.x == 0) *s = atomicAdd(reinterpret_cast<unsigned*>(p.words) + 2, 1u);
    __syncthreads();
    return __builtin_amdgcn_readfirstlane(*s);
}

template <typename X, typename G, bool ACT, bool NORM, int V, int S, int NW>
__global__ __launch_bounds__(64 * NW) void linrec_fwd_kernel(LinrecLaunch p) {
    constexpr int CB = 64 * V;
    static_assert(CB <= 64 * NW, "one thread per channel of the block");
    __shared__ float s_A[NW][CB], s_H[NW][CB], s_in[CB];
    __shared__ unsigned s_ticket;
    const unsigned k = ticket_of(p, &s_ticket), nb = (unsigned)((p.D + CB - 1) / CB);
    const unsigned tile = k / nb;
    const int64_t c0 = (int64_t)(k - tile * nb) * CB;
    const Tile t = tile_of(p.map, tile);
    if (t.n <= 0) return;
    const int w = wave_id(), lane = threadIdx.x & 63;
    const int64_t cl = c0 + lane * V, c = min(cl, p.D - V);   // idle lanes repeat the last channels
    const int first = w * S, nv = min(S, t.n - first);        // this wave's tokens (may be none)

    Raw<X, V> rx[S];
    Raw<G, V> rg[S];
    const X* x = static_cast<const X*>(p.x) + t.row0 * p.xs;
    const G* g = static_cast<const G*>(p.g) + t.row0 * p.gs;
#pragma unroll
    for (int i = 0; i < S; ++i) {
        const int64_t r = min(first + i, t.n - 1);            // rows past the tile: loaded, not used
        rx[i].load(x + r * p.xs + c);
        rg[i].load(g + r * p.gs + c);
    }
    float rate2[V], bias[V], A[V], H[V], a[S][V], u[S][V];
#pragma unroll
    for (int e = 0; e < V; ++e) {
        rate2[e] = ACT ? -LOG2E * expf(p.act.A_log[c + e]) : 0.f;
        bias[e] = ACT ? p.act.dt_bias[c + e] : 0.f;
        A[e] = 1.f;
        H[e] = 0.f;
    }
#pragma unroll
    for (int i = 0; i < S; ++i) {
#pragma unroll
        for (int e = 0; e < V; ++e) {
            const Gate q = gate_of<ACT, NORM, false>(rg[i].get(e), rate2[e], bias[e]);
            a[i][e] = i < nv ? q.a : 1.f;
            u[i][e] = i < nv ? q.m * rx[i].get(e) : 0.f;
            H[e] = a[i][e] * H[e] + u[i][e];
            A[e] *= a[i][e];
        }
    }
#pragma unroll
    for (int e = 0; e < V; ++e) {
        s_A[w][lane * V + e] = A[e];
        s_H[w][lane * V + e] = H[e];
    }
    __syncthreads();
    const int tid = threadIdx.x;
    if (tid < CB && c0 + tid < p.D) {
        const int64_t cc = c0 + tid;
        float tA = 1.f, tH = 0.f;
#pragma unroll
        for (int i = 0; i < NW; ++i) {
            tH = s_A[i][tid] * tH + s_H[i][tid];
            tA *= s_A[i][tid];
        }
        const float h0 = t.j == 0 && p.h0 ? p.h0[t.seq * p.D + cc] : 0.f;
        const float in = t.nt > 1 ? enter(p, tile, t.j, t.nt, 1, cc, tA, tH, h0) : h0;
        s_in[tid] = in;
        if (p.states) p.states[tile * p.D + cc] = in;
        if (p.ht && t.j + 1 == t.nt) p.ht[t.seq * p.D + cc] = tA * in + tH;
    }
    if (!p.y) return;
    __syncthreads();
    if (cl >= p.D) return;
    X* y = static_cast<X*>(p.y) + (t.row0 + first) * p.ys + c;
    float h[V];
#pragma unroll
    for (int e = 0; e < V; ++e) {
        h[e] = s_in[lane * V + e];
        for (int i = 0; i < w; ++i) h[e] = s_A[i][lane * V + e] * h[e] + s_H[i][lane * V + e];
    }
#pragma unroll
    for (int i = 0; i < S; ++i) {
#pragma unroll
        for (int e = 0; e < V; ++e) h[e] = a[i][e] * h[e] + u[i][e];
        if (i < nv) Raw<X, V>::store(y + i * p.ys, h);
    }
}

// The same tiles taken from the last token: e = a (dy + e') is what a token
// hands to the one before it, again a composition of affine maps, with the
// same A.  The states before each token come from the state entering the
// tile, kept by the forward.
template <typename X, typename G, bool ACT, bool NORM, int V, int S, int NW>
__global__ __launch_bounds__(64 * NW) void linrec_bwd_kernel(LinrecLaunch p) {
    constexpr int CB = 64 * V;
    static_assert(CB <= 64 * NW, "one thread per channel of the block");
    __shared__ float s_A[NW][CB], s_H[NW][CB], s_E[NW][CB], s_in[CB], s_e[CB];
    __shared__ unsigned s_ticket;
    const unsigned k = ticket_of(p, &s_ticket), nb = (unsigned)((p.D + CB - 1) / CB);
    const unsigned tile = (unsigned)p.map.max_tiles - 1 - k / nb;
    const int64_t c0 = (int64_t)(k % nb) * CB;
    const Tile t = tile_of(p.map, tile);
    const int w = wave_id(), lane = threadIdx.x & 63, tid = threadIdx.x;
    if (t.n <= 0) {
        if (ACT && tid < CB && c0 + tid < p.D) {
            p.part[(int64_t)(2 * tile) * p.D + c0 + tid] = 0.f;
            p.part[(int64_t)(2 * tile + 1) * p.D + c0 + tid] = 0.f;
        }
        return;
    }
    const int64_t cl = c0 + lane * V, c = min(cl, p.D - V);
    const int first = w * S, nv = min(S, t.n - first);

    Raw<X, V> rx[S], rd[S];
    Raw<G, V> rg[S];
    const X* x = static_cast<const X*>(p.x) + t.row0 * p.xs;
    const G* g = static_cast<const G*>(p.g) + t.row0 * p.gs;
    const X* dy = static_cast<const X*>(p.dy) + t.row0 * p.ys;
#pragma unroll
    for (int i = 0; i < S; ++i) {
        const int64_t r = min(first + i, t.n - 1);
        rg[i].load(g + r * p.gs + c);
        rx[i].load(x + r * p.xs + c);
        rd[i].load(dy + r * p.ys + c);
    }
    float rate2[V], bias[V], A[V], H[V], E[V], a[S][V], la[S][V], m[S][V], sg[S][V];
#pragma unroll
    for (int e = 0; e < V; ++e) {
        rate2[e] = ACT ? -LOG2E * expf(p.act.A_log[c + e]) : 0.f;
        bias[e] = ACT ? p.act.dt_bias[c + e] : 0.f;
        A[e] = 1.f;
        H[e] = 0.f;
        E[e] = 0.f;
    }
#pragma unroll
    for (int i = 0; i < S; ++i) {
#pragma unroll
        for (int e = 0; e < V; ++e) {
            const Gate q = gate_of<ACT, NORM, true>(rg[i].get(e), rate2[e], bias[e]);
            a[i][e] = i < nv ? q.a : 1.f;
            m[i][e] = q.m;
            la[i][e] = q.la;
            sg[i][e] = q.sg;
            H[e] = a[i][e] * H[e] + (i < nv ? q.m * rx[i].get(e) : 0.f);
            A[e] *= a[i][e];
        }
    }
#pragma unroll
    for (int i = S - 1; i >= 0; --i)
#pragma unroll
        for (int e = 0; e < V; ++e) E[e] = a[i][e] * ((i < nv ? rd[i].get(e) : 0.f) + E[e]);
#pragma unroll
    for (int e = 0; e < V; ++e) {
        s_A[w][lane * V + e] = A[e];
        s_H[w][lane * V + e] = H[e];
        s_E[w][lane * V + e] = E[e];
    }
    __syncthreads();
    if (tid < CB && c0 + tid < p.D) {
        const int64_t cc = c0 + tid;
        float tA = 1.f, tE = 0.f;
#pragma unroll
        for (int i = NW - 1; i >= 0; --i) {
            tE = s_A[i][tid] * tE + s_E[i][tid];
            tA *= s_A[i][tid];
        }
        const bool end = t.j + 1 == t.nt;
        const float d0 = end && p.dht ? p.dht[t.seq * p.D + cc] : 0.f;
        const float in = t.nt > 1 ? enter(p, tile, t.nt - 1 - t.j, t.nt, -1, cc, tA, tE, d0) : d0;
        s_e[tid] = in;
        s_in[tid] = p.states[tile * p.D + cc];
        if (p.dh0 && t.j == 0) p.dh0[t.seq * p.D + cc] = tA * in + tE;
    }
    __syncthreads();
    float h[V], d[V], sA[V], sb[V];
    float before[S][V];
#pragma unroll
    for (int e = 0; e < V; ++e) {
        h[e] = s_in[lane * V + e];
        d[e] = s_e[lane * V + e];
        for (int i = 0; i < w; ++i) h[e] = s_A[i][lane * V + e] * h[e] + s_H[i][lane * V + e];
        for (int i = NW - 1; i > w; --i) d[e] = s_A[i][lane * V + e] * d[e] + s_E[i][lane * V + e];
        sA[e] = 0.f;
        sb[e] = 0.f;
    }
#pragma unroll
    for (int i = 0; i < S; ++i)
#pragma unroll
        for (int e = 0; e < V; ++e) {
            before[i][e] = h[e];
            h[e] = a[i][e] * h[e] + m[i][e] * rx[i].get(e);
        }
    X* dx = static_cast<X*>(p.dx) + (t.row0 + first) * p.D + c;
    G* dg = static_cast<G*>(p.dg) + (t.row0 + first) * p.D + c;
#pragma unroll
    for (int i = S - 1; i >= 0; --i) {
        if (i >= nv) continue;
        float ox[V], og[V];
#pragma unroll
        for (int e = 0; e < V; ++e) {
            const float dh = rd[i].get(e) + d[e];
            d[e] = a[i][e] * dh;
            float dla = d[e] * before[i][e];
            if (NORM) dla -= m[i][e] > 0.f ? d[e] * rx[i].get(e) * (a[i][e] * rcp_hw(m[i][e])) : 0.f;
            ox[e] = m[i][e] * dh;
            og[e] = ACT ? dla * (LN2 * rate2[e]) * sg[i][e] : dla;
            if (ACT) {
                sA[e] += dla * la[i][e];
                sb[e] += og[e];
            }
        }
        if (cl < p.D) {
            Raw<X, V>::store(dx + i * p.D, ox);
            Raw<G, V>::store(dg + i * p.D, og);
        }
    }
    if (!ACT) return;
    __syncthreads();                                          // the waves have read the pairs
#pragma unroll
    for (int e = 0; e < V; ++e) {
        s_A[w][lane * V + e] = sA[e];
        s_H[w][lane * V + e] = sb[e];
    }
    __syncthreads();
    if (tid < CB && c0 + tid < p.D) {
        float tA = 0.f, tb = 0.f;
#pragma unroll
        for (int i = 0; i < NW; ++i) {
            tA += s_A[i][tid];
            tb += s_H[i][tid];
        }
        p.part[(int64_t)(2 * tile) * p.D + c0 + tid] = tA;
        p.part[(int64_t)(2 * tile + 1) * p.D + c0 + tid] = tb;
    }
}

// dA_log and ddt_bias: the tiles' sums, 16 strands of tiles per channel, in 64 bits
__global__ __launch_bounds__(1024) void linrec_sum_kernel(LinrecLaunch p) {
    __shared__ double s[16][64];
    const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
    const int64_t nb = (p.D + 63) / 64, which = blockIdx.x / nb, c = (blockIdx.x - which * nb) * 64 + lane;
    double v = 0;
    if (c < p.D)
        for (int64_t i = w; i < p.map.max_tiles; i += 16) v += p.part[(2 * i + which) * p.D + c];
    s[w][lane] = v;
    __syncthreads();
    if (w != 0 || c >= p.D) return;
    for (int i = 1; i < 16; ++i) v += s[i][lane];
    (which ? p.ddt_bias : p.dA_log)[c] = (float)v;
}

// sequences without a token hand their state through: fwd ht = h0, bwd dh0 = dht
__global__ __launch_bounds__(256) void linrec_empty_kernel(LinrecLaunch p, const float* from, float* to) {
    const int64_t nb = (p.D + 255) / 256, n = blockIdx.x / nb, c = (blockIdx.x - n * nb) * 256 + threadIdx.x;
    if (c >= p.D || (p.map.seqs ? p.map.seqs[n].y : p.map.T) > 0) return;
    to[n * p.D + c] = from ? from[n * p.D + c] : 0.f;
}

// One token: y and the state, in place.
template <typename X, typename G, bool ACT, bool NORM, int V>
__global__ __launch_bounds__(64) void linrec_step_kernel(LinrecLaunch p) {
    const int64_t nb = (p.D + 64 * V - 1) / (64 * V), n = blockIdx.x / nb;
    const int64_t c = ((blockIdx.x - n * nb) * 64 + threadIdx.x) * V;
    if (c >= p.D) return;
    Raw<X, V> x;
    Raw<G, V> g;
    Raw<float, V> h;
    x.load(static_cast<const X*>(p.x) + n * p.xs + c);
    g.load(static_cast<const G*>(p.g) + n * p.gs + c);
    h.load(p.ht + n * p.D + c);
    float o[V];
#pragma unroll
    for (int e = 0; e < V; ++e) {
        const float rate2 = ACT ? -LOG2E * expf(p.act.A_log[c + e]) : 0.f, bias = ACT ? p.act.dt_bias[c + e] : 0.f;
        const Gate q = gate_of<ACT, NORM, false>(g.get(e), rate2, bias);
        o[e] = q.a * h.get(e) + q.m * x.get(e);
    }
    Raw<float, V>::store(p.ht + n * p.D + c, o);
    Raw<X, V>::store(static_cast<X*>(p.y) + n * p.ys + c, o);
}

// ---- launches
enum { FWD, BWD, STEP };
template <int WHICH, typename X, typename G, bool ACT, bool NORM, int V>
static hipError_t go2(const LinrecLaunch& p) {
    const int64_t nb = (p.D + 64 * V - 1) / (64 * V);
    if constexpr (WHICH == FWD) {
        hipLaunchKernelGGL((linrec_fwd_kernel<X, G, ACT, NORM, V, 16, 8>), dim3((unsigned)(nb * p.map.max_tiles)),
                           dim3(512), 0, p.stream, p);
    } else if constexpr (WHICH == BWD) {
        hipLaunchKernelGGL((linrec_bwd_kernel<X, G, ACT, NORM, V, 8, 16>), dim3((unsigned)(nb * p.map.max_tiles)),
                           dim3(1024), 0, p.stream, p);
    } else {
        hipLaunchKernelGGL((linrec_step_kernel<X, G, ACT, NORM, V>), dim3((unsigned)(nb * p.map.N)), dim3(64), 0,
                           p.stream, p);
    }
    return hipGetLastError();
}
template <int WHICH, typename X, typename G, int V>
static hipError_t go1(const LinrecLaunch& p) {
    if (p.act.flags & ACT_GATE)
        return p.normalize ? go2<WHICH, X, G, true, true, V>(p) : go2<WHICH, X, G, true, false, V>(p);
    return p.normalize ? go2<WHICH, X, G, false, true, V>(p) : go2<WHICH, X, G, false, false, V>(p);
}
template <int WHICH, int V>
static hipError_t go0(const LinrecLaunch& p) {
    if (p.x_bf16) return p.g_bf16 ? go1<WHICH, bf16, bf16, V>(p) : go1<WHICH, bf16, float, V>(p);
    return p.g_bf16 ? go1<WHICH, float, bf16, V>(p) : go1<WHICH, float, float, V>(p);
}
// Pairs of channels where every row and pointer allows them: half the
// instructions a byte of the one-channel form.
template <int WHICH>
static hipError_t go(const LinrecLaunch& p) {
    const uintptr_t xa = (uintptr_t)p.x | (uintptr_t)p.y | (uintptr_t)p.dy | (uintptr_t)p.dx;
    const uintptr_t ga = (uintptr_t)p.g | (uintptr_t)p.dg;
    const uintptr_t sa = WHICH == STEP ? (uintptr_t)p.ht : 0;
    const bool two = ((p.D | p.xs | p.gs | p.ys) & 1) == 0 && xa % (p.x_bf16 ? 4 : 8) == 0 &&
                     ga % (p.g_bf16 ? 4 : 8) == 0 && sa % 8 == 0;
    return two ? go0<WHICH, 2>(p) : go0<WHICH, 1>(p);
}

static hipError_t empty(const LinrecLaunch& p, const float* from, float* to) {
    if (!to || (!p.map.seqs && p.map.T > 0)) return hipSuccess;
    hipLaunchKernelGGL(linrec_empty_kernel, dim3((unsigned)((p.D + 255) / 256 * p.map.N)), dim3(256), 0, p.stream, p,
                       from, to);
    return hipGetLastError();
}

static hipError_t clear(const LinrecLaunch& p) {
    if (!p.pairs) return hipSuccess;
    hipLaunchKernelGGL(linrec_clear_kernel, dim3((unsigned)((p.D + 255) / 256 * p.map.max_tiles)), dim3(256), 0,
                       p.stream, p);
    return hipGetLastError();
}

hipError_t launch_linrec_fwd(const LinrecLaunch& p) {
    hipError_t e = empty(p, p.h0, p.ht);
    if (e != hipSuccess || p.map.max_tiles == 0) return e;
    if ((e = clear(p)) != hipSuccess) return e;
    return go<FWD>(p);
}

hipError_t launch_linrec_bwd(const LinrecLaunch& p) {
    hipError_t e = empty(p, p.dht, p.dh0);
    if (e != hipSuccess) return e;
    if (p.map.max_tiles > 0) {
        if (p.own_states) {   // the states entering the tiles were not kept
            LinrecLaunch f = p;
            f.y = nullptr;
            f.ht = nullptr;
            if ((e = clear(f)) != hipSuccess || (e = go<FWD>(f)) != hipSuccess) return e;
        }
        if ((e = clear(p)) != hipSuccess || (e = go<BWD>(p)) != hipSuccess) return e;
    }
    if (!(p.act.flags & ACT_GATE)) return hipSuccess;
    hipLaunchKernelGGL(linrec_sum_kernel, dim3((unsigned)(2 * ((p.D + 63) / 64))), dim3(1024), 0, p.stream, p);
    return hipGetLastError();
}

hipError_t launch_linrec_step(const LinrecLaunch& p) { return go<STEP>(p); }

}  // namespace gdn
