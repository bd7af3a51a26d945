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
// tile publishes the group's pair too (after reading the other fifteen), and
// later, in its place, the state that leaves the group.  A tile reads at most
// 15 pairs of its own group, and the groups before from a late one on whose
// state is there, so that the reads do not grow with the sequence (1048576 tokens
// of 512 channels, bf16 with raw gates: forward 1.54 -> 0.85 ms next to reading
// all of them).  Groups are applied to a state, one after the other:
// products of a never span more than a group, 2048 tokens, and where a tile
// starts does not change what is computed, so equal calls give equal bits.  A pair is one
// 64-bit word, stored and loaded by relaxed agent-scope atomics: it is there
// whole or not at all, so no fence and no flag is needed; "not there" is a NaN
// pattern of A that is never published, set by a kernel in front.
//
// Workgroups take their tile from a ticket counter, tiles in the order they
// wait for each other, the channel blocks of a tile one after the other (a
// counter to each block lets them drift apart: 674 -> 752 us on the packed
// input): every tile that one waits for belongs to a workgroup
// that is already running and that publishes without a wait (a group's pair:
// after waits of that kind), so every wait ends.  Each is bounded all the
// same and reports in words[1], which ends the others' waits too.
//
// Measured (bf16 x and y): 4 x 4096 tokens of 2048 channels with fp32 gates 58 us,
// 4.6 TB/s; 137 thousand packed tokens of 4096 channels with raw gates and
// normalised inputs 0.69 ms, bound by the vector ALU (32 instructions and 3
// transcendentals a token and channel, 0.63 ms of issue slots).  A tile is 128
// tokens and 128 channels, 16 tokens to a wave: tiles of 64 tokens take 15 to
// 35 % longer (a hand-off for half the work), of 256 leave one workgroup to a
// CU, 8 % longer on the packed input.
#include <algorithm>

#include "gdn_layer.hpp"

namespace gdn {

constexpr int GROUP = 16;
constexpr unsigned ABSENT = 0xffffffffu;     // never the bits of a published A
constexpr unsigned STATE = 0x80000000u;      // -0, which no product of a is: H is the state itself
constexpr int POLLS = 1 << 20;               // about a second; a hand-off takes microseconds

// ---- gates
// Everything in the log2 domain: the hardware's exp2, reciprocal and reciprocal
// square root (1 unit in the last place each) and two polynomials where a
// direct formula would cancel. Their coefficients are least-squares fits to
// the function over the stated range, reweighted towards the least largest
// relative error; evaluated in 32 bits both are within 2.5 half units.

// log1p(e), 0 <= e <= 1: no reciprocal, as a quotient form would need
__device__ __forceinline__ float log1p_unit(float e) {
    float p = -0.0032440086360021803f;
    p = p * e + 0.019851388409733772f;
    p = p * e - 0.05695939436554909f;
    p = p * e + 0.10603640973567963f;
    p = p * e - 0.1530558466911316f;
    p = p * e + 0.19675935804843903f;
    p = p * e - 0.24954132735729218f;
    p = p * e + 0.3332996368408203f;
    p = p * e - 0.4999990165233612f;
    p = p * e + 1.f;
    return p * e;
}

// 1 - a^2 from l = log2 a: a polynomial times -l for a^2 > 0.7, where 1 - a^2 would cancel
__device__ __forceinline__ float one_minus_sq(float l, float a) {
    float p = 0.03694247081875801f;
    p = p * l + 0.15266050398349762f;
    p = p * l + 0.4439232647418976f;
    p = p * l + 0.9609025716781616f;
    p = p * l + 1.3862943649291992f;
    float near = -l * p, far = 1.f - a * a;
    asm("" : "+v"(near), "+v"(far));       // both, and a select: a branch per element costs more
    return l > -0.25f ? near : far;
}

constexpr float LN2 = 0.6931471805599453f;

struct Gate {
    float l2;      // log2 a
    float a;
    float m;       // factor of x
    float sg;      // sigmoid(g + bias): d log a / d g = rate sg
};
// rate2 = -exp(A_log) log2(e)
template <bool ACT, bool NORM, bool BWD>
__device__ __forceinline__ Gate gate_of(float g, float rate2, float bias) {
    Gate r;
    r.sg = 0.f;
    if (ACT) {
        const float z = g + bias, e = exp2_hw(-LOG2E * fabsf(z));
        r.l2 = rate2 * (fmaxf(z, 0.f) + log1p_unit(e));
        if (BWD) r.sg = (z >= 0.f ? 1.f : e) * __builtin_amdgcn_rcpf(1.f + e);
    } else {
        r.l2 = g * LOG2E;
    }
    r.a = exp2_hw(r.l2);
    r.m = NORM ? __builtin_amdgcn_sqrtf(one_minus_sq(r.l2, r.a)) : 1.f;
    return r;
}

// ---- V consecutive elements as loaded, and their floats
template <typename T, int V> struct Raw;
template <> struct Raw<bf16, 1> {
    uint32_t r;
    __device__ __forceinline__ void load(const bf16* row, unsigned off) { r = peek_row<uint16_t>(row, off); }
    __device__ __forceinline__ float get(int) const { return __uint_as_float(r << 16); }
    __device__ __forceinline__ static void store(bf16* row, unsigned off, const float* f) {
        poke_row<uint16_t>(row, off, f32_to_bf16(f[0]));
    }
};
template <> struct Raw<bf16, 2> {
    uint32_t r;
    __device__ __forceinline__ void load(const bf16* row, unsigned off) { r = peek_row<uint32_t>(row, off); }
    __device__ __forceinline__ float get(int e) const {
        return __uint_as_float(e ? r & 0xffff0000u : r << 16);
    }
    __device__ __forceinline__ static void store(bf16* row, unsigned off, const float* f) {
        poke_row<uint32_t>(row, off, pack_bf16x2(f[0], f[1]));
    }
};
template <> struct Raw<float, 1> {
    float r;
    __device__ __forceinline__ void load(const float* row, unsigned off) { r = peek_row<float>(row, off); }
    __device__ __forceinline__ float get(int) const { return r; }
    __device__ __forceinline__ static void store(float* row, unsigned off, const float* f) {
        poke_row<float>(row, off, f[0]);
    }
};
template <> struct Raw<float, 2> {
    float2 r;
    __device__ __forceinline__ void load(const float* row, unsigned off) { r = __builtin_bit_cast(float2, peek_row<f32x2v>(row, off)); }
    __device__ __forceinline__ float get(int e) const { return e ? r.y : r.x; }
    __device__ __forceinline__ static void store(float* row, unsigned off, const float* f) {
        poke_row<f32x2v>(row, off, f32x2v{f[0], f[1]});
    }
};

// ---- the published pairs
__device__ __forceinline__ void publish(uint64_t* p, float A, float H) {
    const unsigned a = A != A ? 0x7fc00000u : __float_as_uint(A);
    __hip_atomic_store(p, (uint64_t)__float_as_uint(H) << 32 | a, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ void publish_state(uint64_t* p, float H) { publish(p, __uint_as_float(STATE), H); }
__device__ __forceinline__ uint64_t peek(const uint64_t* row, unsigned off) {
    return __hip_atomic_load((const GDN_GLOBAL uint64_t*)((const GDN_GLOBAL char*)in_scalar(row) + off),
                             __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

constexpr int BATCH = 8;
// Compose the pairs of channel c in rows p, p + step, ... (n of them; p, step and n the same
// for the whole wave) in that order onto (A, H), 8 loads in flight at once.  `polls`: what
// is left of this thread's patience; 0 or less once a wait gave up.
__device__ __forceinline__ void compose(const uint64_t* p, int64_t step, int n, int64_t c, float* A, float* H,
                                        int* polls, const int* failed) {
    constexpr int U = BATCH;
    const unsigned off = (unsigned)c * 8;
    for (int i = 0; i < n; i += U) {
        uint64_t v[U];
        bool missing;
        do {
#pragma unroll
            for (int k = 0; k < U; ++k) v[k] = peek(p + min(i + k, n - 1) * step, off);
            missing = false;
#pragma unroll
            for (int k = 0; k < U; ++k) missing |= (unsigned)v[k] == ABSENT;
            if (missing) __builtin_amdgcn_s_sleep(1);
            // someone else's patience has run out: so has this thread's
            if (missing && *polls % 1024 == 1 && __hip_atomic_load(failed, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT))
                *polls = 1;
        } while (missing && --*polls > 0);
        // (a STATE by its sign, which no other word has by now: a comparison with the pattern is
        // moved into the loop above and costs 16 registers)
#pragma unroll
        for (int k = 0; k < U; ++k) {
            const bool past = i + k >= n;
            const float a = __uint_as_float((unsigned)v[k]), h = __uint_as_float((unsigned)(v[k] >> 32));
            *H = past ? *H : (int)(unsigned)v[k] < 0 ? h : __builtin_fmaf(a, *H, h);
            *A = past ? *A : *A * a;
        }
    }
}

// What enters tile j of a sequence (of nt; row `tile` of the workspace) is put
// together from the pairs of the tiles and groups before it by NT threads to
// a channel: two halves of its own group's tiles (parts 0, 1) and the groups
// before (part 2), all waited for at once.  dir = 1: tiles in the
// order of the tokens; -1: against it, j counted from the sequence's end.
// The first tile publishes a state, with the value that enters the sequence
// worked in, and so does the first group.
constexpr int NT = 3;
// part 0 or 1; start: the value that enters the sequence
__device__ __forceinline__ void enter_own(const LinrecLaunch& p, int64_t tile, int j, int dir, int64_t c, int part,
                                          float start, float* A, float* H) {
    const int in = j % GROUP, s0 = part * (GROUP / 2), n = min(in - s0, GROUP / 2);
    int polls = POLLS;
    *A = 1.f;
    *H = 0.f;
    compose(p.pairs + (tile + (int64_t)dir * (s0 - in)) * p.D, (int64_t)dir * p.D, n, c, A, H, &polls, p.words + 1);
    if (part == 0 && j == 0) *H = start;
    if (part == 0 && j < GROUP) *A = 0.f;          // a state, whatever the A of the pairs after the first
    if (polls <= 0) atomicExch(p.words + 1, 1);
}
// Part 2: the state that leaves the group before (0: there is none).  Every eighth
// group from the last one back is looked at, without a wait; from the latest one in
// which every channel of the wave has a state (or the first) on, the groups are waited for and
// applied.  Up to 16 groups two batches of loads read them all, and the look would be a third.
__device__ __forceinline__ float enter_groups(const LinrecLaunch& p, int64_t tile, int j, int dir, int64_t c) {
    // a group's row is a sixteenth of its last tile's, which no other group's is
    const int64_t first = (tile + (int64_t)dir * (GROUP - 1 - j)) / GROUP, step = (int64_t)dir * p.D;
    const uint64_t* row = p.groups + first * p.D;
    const int ng = j / GROUP;
    int s = 0;
    for (int last = ng - 1; s == 0 && last >= 16; last -= BATCH * BATCH) {
        unsigned v[BATCH];
#pragma unroll
        for (int k = 0; k < BATCH; ++k) v[k] = (unsigned)peek(row + max(last - k * BATCH, 0) * step, (unsigned)c * 8);
#pragma unroll
        for (int k = BATCH - 1; k >= 0; --k)
            if (__ballot(v[k] != STATE) == 0) s = max(last - k * BATCH, 0);
    }
    int polls = POLLS;
    float A = 1.f, H = 0.f;
    compose(row + s * step, step, ng - s, c, &A, &H, &polls, p.words + 1);
    if (polls <= 0) atomicExch(p.words + 1, 1);
    return H;
}
// the tile's own pair; and once the parts of its group are there, the group's
__device__ __forceinline__ void publish_tile(const LinrecLaunch& p, int64_t tile, int j, int nt, int64_t c, float A,
                                             float H, float start) {
    if (j + 1 >= nt) return;
    if (j == 0) publish_state(p.pairs + tile * p.D + c, A * start + H);
    else publish(p.pairs + tile * p.D + c, A, H);
}
// (only of a group that has tiles behind it: closes_group)
__device__ __forceinline__ bool closes_group(int j, int nt) { return j % GROUP == GROUP - 1 && j + 1 < nt; }
// LEFT: once the state that enters the group is there too, the state that leaves it, by the
// operations that a tile which reads the pair applies to that state.
template <bool LEFT, int CB>
__device__ __forceinline__ void publish_group(const LinrecLaunch& p, int64_t tile, int j, int64_t c, float A, float H,
                                              const float (*s_pA)[CB], const float (*s_pH)[CB], int k) {
    uint64_t* to = p.groups + (tile / GROUP) * p.D + c;
    const float gA = s_pA[0][k] * s_pA[1][k] * A;
    const float gH = __builtin_fmaf(A, __builtin_fmaf(s_pA[1][k], s_pH[0][k], s_pH[1][k]), H);
    if (LEFT) publish_state(to, __builtin_fmaf(gA, s_pH[2][k], gH));
    else if (j < GROUP) publish_state(to, gH);
    else publish(to, gA, gH);
}
template <int CB> __device__ __forceinline__ float entering(const float (*s_pA)[CB], const float (*s_pH)[CB], int k) {
    const float v = s_pA[0][k] * s_pH[2][k] + s_pH[0][k];
    return s_pA[1][k] * v + s_pH[1][k];
}

// Every pair that some tile reads is marked absent, the ticket and the words
// are cleared; and sequences without a token hand their state through
// (forward: ht = h0, backward: dh0 = dht), by the workgroups past the tiles'.
__global__ __launch_bounds__(256) void linrec_clear_kernel(LinrecLaunch p, const float* from, float* to) {
    const unsigned nb = (unsigned)((p.D + 511) / 512), i = blockIdx.x / nb;
    const int64_t c0 = (int64_t)(blockIdx.x - i * nb) * 512 + threadIdx.x;
    if (blockIdx.x == 0 && threadIdx.x == 0 && p.pairs) {
        if (!p.map.table) p.words[0] = 0;
        if (!p.keep_status) p.words[1] = 0;
        p.words[TICKET] = 0;
    }
    const int64_t tiles = p.pairs ? p.map.max_tiles : 0;
    if (i >= tiles) {
        const int64_t n = i - tiles;
        if ((p.map.seqs ? p.map.seqs[n].y : p.map.T) > 0) return;
        for (int64_t c = c0; c < min(c0 + 512, p.D); c += 256) to[n * p.D + c] = from ? from[n * p.D + c] : 0.f;
        return;
    }
    const Tile t = tile_of(p.map, i);
    if (t.n <= 0 || t.nt <= 1) return;
    for (int64_t c = c0; c < min(c0 + 512, p.D); c += 256) {
        p.pairs[i * p.D + c] = ABSENT;
        if (t.nt > GROUP) p.groups[(i / GROUP) * p.D + c] = ABSENT;
    }
}

// Tile and channel block of this workgroup (of nb blocks): by ticket where tiles
// wait for each other.  With sequences that run without hand-offs most rows of
// the table may be unused: then the chip's fill of workgroups takes tickets
// until the rows in use are done (a workgroup to each row: 54 us for 2559 unused
// ones).  Else the word that tells the rows in use is not waited for.
// False: none left.
constexpr int64_t FILL = 512;
enum { ALONE, TILES, QUEUE };   // HAND: without hand-offs, with, and with them row after row
template <int HAND>
__device__ __forceinline__ bool tile_by_ticket(const LinrecLaunch& p, unsigned nb, bool backward, unsigned* tile,
                                               unsigned* block, unsigned* s) {
    unsigned k = blockIdx.x, used = (unsigned)p.map.max_tiles;
    if (HAND && p.pairs) {                 // else every sequence is one tile: no words
        if (HAND == QUEUE) used = __builtin_amdgcn_readfirstlane((unsigned)p.words[2]);
        if (threadIdx.x == 0) *s = atomicAdd(reinterpret_cast<unsigned*>(p.words) + TICKET, 1u);
        __syncthreads();
        k = __builtin_amdgcn_readfirstlane(*s);
    }
    const unsigned i = k / nb;
    *block = k - i * nb;
    *tile = HAND && backward ? used - 1 - i : i;
    return HAND != QUEUE || i < used;
}

// A wave's place in its tile.
struct Spot {
    int w, lane, first, nv;   // wave, lane; first token in the tile; its tokens (0 and less: none)
    int64_t c0, c;            // first channel of the block; of the lane (idle lanes repeat the last)
    bool in;                  // the lane has channels
};
template <int V, int S>
__device__ __forceinline__ Spot spot_of(const LinrecLaunch& p, const Tile& t, int64_t c0) {
    Spot s;
    s.w = wave_id();
    s.lane = threadIdx.x & 63;
    s.first = s.w * S;
    s.nv = min(S, t.n - s.first);
    s.c0 = c0;
    s.in = c0 + s.lane * V < p.D;
    s.c = min(c0 + s.lane * V, p.D - V);
    return s;
}
// A tile that is not FULL is worked on four tokens at a time: those past its end
// repeat its last row and count as a = 1, u = 0, groups that are wholly past it are left
// out (a condition to every token would leave nothing to overlap).
constexpr int QUAD = 4;
// row of the wave's token i
template <bool FULL, typename T>
__device__ __forceinline__ const T* row_at(const T* tile, int64_t stride, const Spot& s, const Tile& t, int i) {
    return in_scalar(tile + (int64_t)(FULL ? s.first + i : min(s.first + i, t.n - 1)) * stride);
}

// HAND: tiles of a sequence hand their pairs on; without it every sequence is one tile.
template <bool FULL, int HAND, typename X, typename G, bool ACT, bool NORM, int V, int S, int NW>
__device__ __forceinline__ void fwd_tile(const LinrecLaunch& p, const Tile& t, int64_t tile, int64_t c0,
                                         float (*s_A)[64 * V], float (*s_H)[64 * V], float (*s_pA)[64 * V],
                                         float (*s_pH)[64 * V]) {
    constexpr int CB = 64 * V;
    const Spot s = spot_of<V, S>(p, t, c0);
    const X* x = static_cast<const X*>(p.x) + t.row0 * p.xs;
    const G* g = static_cast<const G*>(p.g) + t.row0 * p.gs;
    const unsigned ox = (unsigned)s.c * sizeof(X), og = (unsigned)s.c * sizeof(G);
    Raw<X, V> rx[S];
    Raw<G, V> rg[S];
#pragma unroll
    for (int q = 0; q < S; q += QUAD) {
        if (!FULL && q >= s.nv) continue;     // the same for the whole wave, here and below
#pragma unroll
        for (int i = q; i < q + QUAD; ++i) {
            rg[i].load(row_at<FULL>(g, p.gs, s, t, i), og);
            rx[i].load(row_at<FULL>(x, p.xs, s, t, i), ox);
        }
    }
    float rate2[V], bias[V], A[V], H[V], a[S][V], u[S][V];
#pragma unroll
    for (int e = 0; e < V; ++e) {
        rate2[e] = ACT ? -LOG2E * expf(p.act.A_log[s.c + e]) : 0.f;
        bias[e] = ACT ? p.act.dt_bias[s.c + e] : 0.f;
        A[e] = 1.f;
        H[e] = 0.f;
    }
#pragma unroll
    for (int q = 0; q < S; q += QUAD) {
        if (!FULL && q >= s.nv) continue;
#pragma unroll
        for (int i = q; i < q + QUAD; ++i)
#pragma unroll
            for (int e = 0; e < V; ++e) {
                const Gate w = gate_of<ACT, NORM, false>(rg[i].get(e), rate2[e], bias[e]);
                a[i][e] = FULL || i < s.nv ? w.a : 1.f;
                u[i][e] = FULL || i < s.nv ? w.m * rx[i].get(e) : 0.f;
                H[e] = a[i][e] * H[e] + u[i][e];
                A[e] *= a[i][e];
            }
    }
#pragma unroll
    for (int e = 0; e < V; ++e) {
        s_A[s.w][s.lane * V + e] = A[e];
        s_H[s.w][s.lane * V + e] = H[e];
    }
    float h[V];
    if constexpr (!HAND) {   // read by every wave before one of them may write ht, which may be h0
#pragma unroll
        for (int e = 0; e < V; ++e) h[e] = p.h0 ? p.h0[t.seq * p.D + s.c + e] : 0.f;
    }
    __syncthreads();
    const int tid = threadIdx.x;
    if constexpr (HAND) {
        const int part = s.w * 64 / CB, k = tid - part * CB;      // the same part for the whole wave
        const bool own = part == 0 && c0 + k < p.D;
        float tA = 1.f, tH = 0.f;
        const bool live = part < NT && c0 + k < p.D, closes = closes_group(t.j, t.nt);
        if (own) {
#pragma unroll 4
            for (int i = 0; i < NW; ++i) {
                tH = s_A[i][k] * tH + s_H[i][k];
                tA *= s_A[i][k];
            }
        }
        if (live && part < 2) {
            const float start = t.j == 0 && part == 0 && p.h0 ? p.h0[t.seq * p.D + c0 + k] : 0.f;
            if (part == 0) publish_tile(p, tile, t.j, t.nt, c0 + k, tA, tH, start);
            enter_own(p, tile, t.j, 1, c0 + k, part, start, &s_pA[part][k], &s_pH[part][k]);
        }
        if (closes) {        // before waiting for other groups, or the groups would wait in a row
            __syncthreads();
            if (own) publish_group<false, CB>(p, tile, t.j, c0 + k, tA, tH, s_pA, s_pH, k);
        }
        if (live && part == 2) s_pH[2][k] = enter_groups(p, tile, t.j, 1, c0 + k);
        __syncthreads();
        if (own) {
            if (closes && t.j >= GROUP) publish_group<true, CB>(p, tile, t.j, c0 + k, tA, tH, s_pA, s_pH, k);
            const float in = entering<CB>(s_pA, s_pH, k);
            if (p.states) p.states[tile * p.D + c0 + k] = in;
            if (p.ht && t.j + 1 == t.nt) p.ht[t.seq * p.D + c0 + k] = tA * in + tH;
        }
        if (!p.y) return;
#pragma unroll
        for (int e = 0; e < V; ++e) h[e] = entering<CB>(s_pA, s_pH, s.lane * V + e);
    }
#pragma unroll
    for (int e = 0; e < V; ++e)
        for (int i = 0; i < s.w; ++i) h[e] = s_A[i][s.lane * V + e] * h[e] + s_H[i][s.lane * V + e];
    if (!s.in) return;
    X* y = static_cast<X*>(p.y) + (t.row0 + s.first) * p.ys;
#pragma unroll
    for (int i = 0; i < S; ++i) {
        if (!FULL && i >= s.nv) continue;
#pragma unroll
        for (int e = 0; e < V; ++e) h[e] = a[i][e] * h[e] + u[i][e];
        if (p.y) Raw<X, V>::store(in_scalar(y + i * p.ys), ox, h);
    }
    // the wave of the sequence's last token
    if (!HAND && p.ht && s.nv > 0 && s.first + s.nv == t.n) {
#pragma unroll
        for (int e = 0; e < V; ++e) p.ht[t.seq * p.D + s.c + e] = h[e];
    }
}

template <int HAND, typename X, typename G, bool ACT, bool NORM, int V, int S, int NW>
__global__ __launch_bounds__(64 * NW, 4) void linrec_fwd_kernel(LinrecLaunch p) {
    constexpr int CB = 64 * V;
    static_assert(!HAND || NT * CB <= 64 * NW, "NT threads to a channel of the block");
    __shared__ float s_A[NW][CB], s_H[NW][CB], s_pA[HAND ? 2 : 1][CB], s_pH[HAND ? NT : 1][CB];
    __shared__ unsigned s_ticket;
    unsigned tile, block;
    while (tile_by_ticket<HAND>(p, (unsigned)((p.D + CB - 1) / CB), false, &tile, &block, &s_ticket)) {
        const int64_t c0 = (int64_t)block * CB;
        const Tile t = tile_of(p.map, tile);
        if (HAND != QUEUE && t.n <= 0) return;
        if (t.n == S * NW) fwd_tile<true, HAND, X, G, ACT, NORM, V, S, NW>(p, t, tile, c0, s_A, s_H, s_pA, s_pH);
        else if (HAND != QUEUE || t.n > 0)
            fwd_tile<false, HAND, X, G, ACT, NORM, V, S, NW>(p, t, tile, c0, s_A, s_H, s_pA, s_pH);
        if (HAND != QUEUE) return;
        __syncthreads();                       // the waves are done with the tile's LDS
    }
}

// The same tiles taken from the last token: e = a (dy + e') is what a token
// hands to the one before it, again a composition of affine maps, with the
// same A.  The states before each token come from the state entering the
// tile, kept by the forward.  16 waves of 8 tokens: a, m, x, dy and the states
// of 16 values a thread are what 128 registers hold.  2 x 8192 tokens of 2048
// channels, bf16, raw gates, normalised: 116 us against 66 us of bytes and 73
// us of ALU slots; one workgroup fills a CU (159 KB of LDS, 16 waves of 128 registers), so
// the loads and the hand-off of a tile are not hidden by another.
template <bool FULL, int HAND, typename X, typename G, bool ACT, bool NORM, int V, int S, int NW>
__device__ __forceinline__ void bwd_tile(const LinrecLaunch& p, const Tile& t, int64_t tile, int64_t c0,
                                         float (*s_A)[64 * V], float (*s_H)[64 * V], float (*s_E)[64 * V],
                                         float (*s_pA)[64 * V], float (*s_pE)[64 * V], float* s_in,
                                         f32x2v (*s_gate)[64 * NW]) {
    constexpr int CB = 64 * V;
    const Spot s = spot_of<V, S>(p, t, c0);
    const int tid = threadIdx.x;
    const X* x = static_cast<const X*>(p.x) + t.row0 * p.xs;
    const G* g = static_cast<const G*>(p.g) + t.row0 * p.gs;
    const X* dy = static_cast<const X*>(p.dy) + t.row0 * p.ys;
    const unsigned ox = (unsigned)s.c * sizeof(X), og = (unsigned)s.c * sizeof(G);
    Raw<X, V> rx[S], rd[S];
    float a[S][V], m[S][V];
    float rate2[V], bias[V], A[V], H[V], E[V];
    {
        Raw<G, V> rg[S];
#pragma unroll
        for (int q = 0; q < S; q += QUAD) {
            if (!FULL && q >= s.nv) continue;
#pragma unroll
            for (int i = q; i < q + QUAD; ++i) {
                rg[i].load(row_at<FULL>(g, p.gs, s, t, i), og);
                rx[i].load(row_at<FULL>(x, p.xs, s, t, i), ox);
                rd[i].load(row_at<FULL>(dy, p.ys, s, t, i), ox);
            }
        }
#pragma unroll
        for (int e = 0; e < V; ++e) {
            rate2[e] = ACT ? -LOG2E * expf(p.act.A_log[s.c + e]) : 0.f;
            bias[e] = ACT ? p.act.dt_bias[s.c + e] : 0.f;
            A[e] = 1.f;
            H[e] = 0.f;
            E[e] = 0.f;
        }
#pragma unroll
        for (int q = 0; q < S; q += QUAD) {
            if (!FULL && q >= s.nv) continue;
#pragma unroll
            for (int i = q; i < q + QUAD; ++i) {
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    const Gate w = gate_of<ACT, NORM, true>(rg[i].get(e), rate2[e], bias[e]);
                    a[i][e] = FULL || i < s.nv ? w.a : 1.f;
                    m[i][e] = w.m;
                    if (ACT) s_gate[i * V + e][tid] = f32x2v{w.l2, w.sg};
                    H[e] = a[i][e] * H[e] + (FULL || i < s.nv ? w.m * rx[i].get(e) : 0.f);
                    A[e] *= a[i][e];
                }
                // a token at a time where registers, not overlap, are short
                if (HAND) __builtin_amdgcn_sched_barrier(0);
            }
        }
    }
#pragma unroll
    for (int i = S - 1; i >= 0; --i) {
        if (!FULL && i >= s.nv) continue;
#pragma unroll
        for (int e = 0; e < V; ++e) E[e] = a[i][e] * (rd[i].get(e) + E[e]);
    }
#pragma unroll
    for (int e = 0; e < V; ++e) {
        s_A[s.w][s.lane * V + e] = A[e];
        s_H[s.w][s.lane * V + e] = H[e];
        s_E[s.w][s.lane * V + e] = E[e];
    }
    __syncthreads();
    float h[V], d[V], sA[V], sb[V], before[S][V];
    if constexpr (HAND) {
        const int part = s.w * 64 / CB, k = tid - part * CB;      // the same part for the whole wave
        const bool own = part == 0 && c0 + k < p.D;
        const int back = t.nt - 1 - t.j;                           // the tile counted from the sequence's end
        float tA = 1.f, tE = 0.f;
        const bool live = part < NT && c0 + k < p.D, closes = closes_group(back, t.nt);
        if (own) {
#pragma unroll 2
            for (int i = NW - 1; i >= 0; --i) {
                tE = s_A[i][k] * tE + s_E[i][k];
                tA *= s_A[i][k];
            }
            s_in[k] = p.states[tile * p.D + c0 + k];
        }
        if (live && part < 2) {
            const float start = back == 0 && part == 0 && p.dht ? p.dht[t.seq * p.D + c0 + k] : 0.f;
            if (part == 0) publish_tile(p, tile, back, t.nt, c0 + k, tA, tE, start);
            enter_own(p, tile, back, -1, c0 + k, part, start, &s_pA[part][k], &s_pE[part][k]);
        }
        if (closes) {        // before waiting for other groups, or the groups would wait in a row
            __syncthreads();
            if (own) publish_group<false, CB>(p, tile, back, c0 + k, tA, tE, s_pA, s_pE, k);
        }
        if (live && part == 2) s_pE[2][k] = enter_groups(p, tile, back, -1, c0 + k);
        __syncthreads();
        if (own) {
            if (closes && back >= GROUP) publish_group<true, CB>(p, tile, back, c0 + k, tA, tE, s_pA, s_pE, k);
            if (p.dh0 && t.j == 0) p.dh0[t.seq * p.D + c0 + k] = tA * entering<CB>(s_pA, s_pE, k) + tE;
        }
#pragma unroll
        for (int e = 0; e < V; ++e) {
            h[e] = s_in[s.lane * V + e];
            d[e] = entering<CB>(s_pA, s_pE, s.lane * V + e);
        }
    } else {
#pragma unroll
        for (int e = 0; e < V; ++e) {
            h[e] = p.h0 ? p.h0[t.seq * p.D + s.c + e] : 0.f;
            d[e] = p.dht ? p.dht[t.seq * p.D + s.c + e] : 0.f;
        }
    }
#pragma unroll
    for (int e = 0; e < V; ++e) {
        for (int i = 0; i < s.w; ++i) h[e] = s_A[i][s.lane * V + e] * h[e] + s_H[i][s.lane * V + e];
        for (int i = NW - 1; i > s.w; --i) d[e] = s_A[i][s.lane * V + e] * d[e] + s_E[i][s.lane * V + e];
        sA[e] = 0.f;
        sb[e] = 0.f;
    }
#pragma unroll
    for (int i = 0; i < S; ++i) {
        if (!FULL && i >= s.nv) continue;
#pragma unroll
        for (int e = 0; e < V; ++e) {
            before[i][e] = h[e];
            h[e] = a[i][e] * h[e] + m[i][e] * rx[i].get(e);
        }
    }
    X* dx = static_cast<X*>(p.dx) + (t.row0 + s.first) * p.D;
    G* dg = static_cast<G*>(p.dg) + (t.row0 + s.first) * p.D;
#pragma unroll
    for (int i = S - 1; i >= 0; --i) {
        if (!FULL && i >= s.nv) continue;
        float vx[V], vg[V];
#pragma unroll
        for (int e = 0; e < V; ++e) {
            const float dh = rd[i].get(e) + d[e];
            d[e] = a[i][e] * dh;
            float dla = d[e] * before[i][e];
            if (NORM)
                dla -= m[i][e] > 0.f ? d[e] * rx[i].get(e) * (a[i][e] * __builtin_amdgcn_rcpf(m[i][e])) : 0.f;
            vx[e] = m[i][e] * dh;
            vg[e] = dla;
            if (ACT) {
                const f32x2v q = s_gate[i * V + e][tid];
                vg[e] = dla * (LN2 * rate2[e]) * q.y;
                sA[e] += dla * q.x;
                sb[e] += vg[e];
            }
        }
        if (s.in) {
            Raw<X, V>::store(in_scalar(dx + i * p.D), ox, vx);
            Raw<G, V>::store(in_scalar(dg + i * p.D), og, vg);
        }
        __builtin_amdgcn_sched_barrier(0);
    }
    if (!HAND && p.dh0 && s.w == 0 && s.in) {
#pragma unroll
        for (int e = 0; e < V; ++e) p.dh0[t.seq * p.D + s.c + e] = d[e];
    }
    if (!ACT) return;
    __syncthreads();                                          // the waves have read the pairs
#pragma unroll
    for (int e = 0; e < V; ++e) {
        s_A[s.w][s.lane * V + e] = sA[e];
        s_H[s.w][s.lane * V + e] = sb[e];
    }
    __syncthreads();
    for (int k = tid; k < CB && c0 + k < p.D; k += 64 * NW) {
        float tA = 0.f, tb = 0.f;
#pragma unroll
        for (int i = 0; i < NW; ++i) {
            tA += s_A[i][k];
            tb += s_H[i][k];
        }
        p.part[2 * tile * p.D + c0 + k] = LN2 * tA;
        p.part[(2 * tile + 1) * p.D + c0 + k] = tb;
    }
}

template <int HAND, typename X, typename G, bool ACT, bool NORM, int V, int S, int NW>
__global__ __launch_bounds__(64 * NW) void linrec_bwd_kernel(LinrecLaunch p) {
    constexpr int CB = 64 * V;
    static_assert(!HAND || NT * CB <= 64 * NW, "NT threads to a channel of the block");
    __shared__ float s_A[NW][CB], s_H[NW][CB], s_E[NW][CB];
    __shared__ float s_pA[HAND ? 2 : 1][CB], s_pE[HAND ? NT : 1][CB], s_in[CB];
    // log2 a and sigmoid of every token, each thread's own: they are wanted again only at
    // the end, and next to a, m, x and dy there are no registers for them
    __shared__ f32x2v s_gate[ACT ? S * V : 1][64 * NW];
    __shared__ unsigned s_ticket;
    unsigned tile, block;
    while (tile_by_ticket<HAND>(p, (unsigned)((p.D + CB - 1) / CB), true, &tile, &block, &s_ticket)) {
        const int64_t c0 = (int64_t)block * CB;
        const Tile t = tile_of(p.map, tile);
        if (t.n <= 0) {
            if (ACT)
                for (int k = threadIdx.x; k < CB && c0 + k < p.D; k += 64 * NW) {
                    p.part[(int64_t)(2 * tile) * p.D + c0 + k] = 0.f;
                    p.part[(int64_t)(2 * tile + 1) * p.D + c0 + k] = 0.f;
                }
            if (HAND != QUEUE) return;
        } else if (t.n == S * NW) {
            bwd_tile<true, HAND, X, G, ACT, NORM, V, S, NW>(p, t, tile, c0, s_A, s_H, s_E, s_pA, s_pE, s_in, s_gate);
        } else {
            bwd_tile<false, HAND, X, G, ACT, NORM, V, S, NW>(p, t, tile, c0, s_A, s_H, s_E, s_pA, s_pE, s_in, s_gate);
        }
        if (HAND != QUEUE) return;
        __syncthreads();                       // the waves are done with the tile's LDS
    }
}

// One token: y and the state, in place.  32 x 2048 takes 3 us, the time of a launch.
template <typename X, typename G, bool ACT, bool NORM, int V>
__global__ __launch_bounds__(64) void linrec_step_kernel(LinrecLaunch p) {
    const int64_t nb = (p.D + 64 * V - 1) / (64 * V), n = blockIdx.x / nb;
    const int64_t c = ((blockIdx.x - n * nb) * 64 + threadIdx.x) * V;
    if (c >= p.D) return;
    Raw<X, V> x;
    Raw<G, V> g;
    Raw<float, V> h;
    const unsigned ox = (unsigned)c * sizeof(X);
    x.load(static_cast<const X*>(p.x) + n * p.xs, ox);
    g.load(static_cast<const G*>(p.g) + n * p.gs, (unsigned)c * sizeof(G));
    h.load(p.ht + n * p.D, (unsigned)c * 4);
    float o[V];
#pragma unroll
    for (int e = 0; e < V; ++e) {
        const float rate2 = ACT ? -LOG2E * expf(p.act.A_log[c + e]) : 0.f, bias = ACT ? p.act.dt_bias[c + e] : 0.f;
        const Gate q = gate_of<ACT, NORM, false>(g.get(e), rate2, bias);
        o[e] = q.a * h.get(e) + q.m * x.get(e);
    }
    Raw<float, V>::store(p.ht + n * p.D, (unsigned)c * 4, o);
    Raw<X, V>::store(static_cast<X*>(p.y) + n * p.ys, ox, o);
}

// ---- launches
enum { FWD, FWDQ, FWD16, FWD64, BWD, BWDQ, BWD16, BWD64, STEP };
template <int HAND, typename X, typename G, bool ACT, bool NORM, int V, int S, int NW>
static void fwd(const LinrecLaunch& p, int64_t blocks) {
    hipLaunchKernelGGL((linrec_fwd_kernel<HAND, X, G, ACT, NORM, V, S, NW>), dim3((unsigned)blocks), dim3(64 * NW), 0,
                       p.stream, p);
}
template <int HAND, typename X, typename G, bool ACT, bool NORM, int V, int S, int NW>
static void bwd(const LinrecLaunch& p, int64_t blocks) {
    hipLaunchKernelGGL((linrec_bwd_kernel<HAND, X, G, ACT, NORM, V, S, NW>), dim3((unsigned)blocks), dim3(64 * NW), 0,
                       p.stream, p);
}
template <int WHICH, typename X, typename G, bool ACT, bool NORM, int V>
static hipError_t go2(const LinrecLaunch& p) {
    const int64_t nb = (p.D + 64 * V - 1) / (64 * V), tiles = nb * (p.map.shorts ? p.map.N : p.map.max_tiles);
    if constexpr (WHICH == FWD) fwd<TILES, X, G, ACT, NORM, V, 16, 8>(p, tiles);
    else if constexpr (WHICH == FWDQ) fwd<QUEUE, X, G, ACT, NORM, V, 16, 8>(p, std::min(tiles, FILL));
    else if constexpr (WHICH == FWD16) fwd<ALONE, X, G, ACT, NORM, V, 16, 1>(p, tiles);
    else if constexpr (WHICH == FWD64) fwd<ALONE, X, G, ACT, NORM, V, 16, 4>(p, tiles);
    else if constexpr (WHICH == BWD) bwd<TILES, X, G, ACT, NORM, V, 8, 16>(p, tiles);
    else if constexpr (WHICH == BWDQ) bwd<QUEUE, X, G, ACT, NORM, V, 8, 16>(p, std::min(tiles, FILL));
    else if constexpr (WHICH == BWD16) bwd<ALONE, X, G, ACT, NORM, V, 8, 2>(p, tiles);
    else if constexpr (WHICH == BWD64) bwd<ALONE, X, G, ACT, NORM, V, 8, 8>(p, tiles);
    else
        hipLaunchKernelGGL((linrec_step_kernel<X, G, ACT, NORM, V>), dim3((unsigned)(nb * p.map.N)), dim3(64), 0,
                           p.stream, p);
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

// in front of the tiles' kernel; from, to: the state that sequences without a token hand through
static hipError_t clear(const LinrecLaunch& p, const float* from, float* to) {
    const bool empties = to && (p.map.seqs || p.map.T == 0);
    const int64_t rows = (p.pairs ? p.map.max_tiles : 0) + (empties ? p.map.N : 0);
    if (rows == 0) return hipSuccess;
    hipLaunchKernelGGL(linrec_clear_kernel, dim3((unsigned)((p.D + 511) / 512 * rows)), dim3(256), 0, p.stream, p, from,
                       to);
    return hipGetLastError();
}

// the packed sequences of up to p.shorts tokens
static LinrecLaunch short_ones(const LinrecLaunch& p) {
    LinrecLaunch q = p;
    q.map.shorts = p.shorts;
    q.states = nullptr;
    return q;
}
static hipError_t fwd_few(const LinrecLaunch& p, int few) { return few == 16 ? go<FWD16>(p) : go<FWD64>(p); }
static hipError_t bwd_few(const LinrecLaunch& p, int few) { return few == 16 ? go<BWD16>(p) : go<BWD64>(p); }

hipError_t launch_linrec_fwd(const LinrecLaunch& p) {
    hipError_t e = clear(p, p.h0, p.ht);
    if (e != hipSuccess || p.map.T == 0) return e;
    if (p.small) return fwd_few(p, p.small);
    if (p.shorts && (p.y || p.ht) && (e = fwd_few(short_ones(p), p.shorts)) != hipSuccess) return e;
    return p.shorts ? go<FWDQ>(p) : go<FWD>(p);
}

hipError_t launch_linrec_bwd(const LinrecLaunch& p) {
    hipError_t e;
    if (p.own_states && !p.small && p.map.T > 0) {   // the states entering the tiles were not kept
        LinrecLaunch f = p;
        f.y = nullptr;
        f.ht = nullptr;
        if ((e = launch_linrec_fwd(f)) != hipSuccess) return e;
    }
    LinrecLaunch c = p;
    c.keep_status = p.own_states && !p.small;        // of the states' waits
    if (p.shorts) c.part += 2 * p.map.N * p.D;
    if ((e = clear(c, p.dht, p.dh0)) != hipSuccess) return e;
    if (p.map.T > 0) {
        if (p.small) e = bwd_few(p, p.small);
        else if (p.shorts && (e = bwd_few(short_ones(p), p.shorts)) != hipSuccess) return e;
        else e = p.shorts ? go<BWDQ>(c) : go<BWD>(c);
        if (e != hipSuccess) return e;
    }
    if (!(p.act.flags & ACT_GATE)) return hipSuccess;
    const int64_t rows = p.map.T > 0 ? p.map.max_tiles + (p.shorts ? p.map.N : 0) : 0;
    return launch_row_sum(RowSumLaunch{p.part, rows, p.D, 1, 2, p.dA_log, p.ddt_bias, p.sums, p.stream, 1,
                                       p.shorts ? p.words + 2 : nullptr, p.map.max_tiles});
}

hipError_t launch_linrec_step(const LinrecLaunch& p) { return go<STEP>(p); }

}  // namespace gdn
