// Linear attention with a decay for each head, in chunks of 64 tokens.
//
// Forward, per state head, with G_i = g_first + ... + g_i inside a chunk and
// S the state entering it:
//   o_i = scale (e^{G_i} q_i S + sum_{j<=i} e^{G_i-G_j} (q_i k_j) v_j)
//   S'  = e^{G_last} S + sum_j e^{G_last-G_j} k_j v_j^T
// Its gradients are the same walk over other operands: with E the gradient of
// the state behind a chunk,
//   dq_i = scale (e^{G_i} do_i S^T + sum_{j<=i} e^{G_i-G_j} (do_i v_j) k_j)
//   dk_j = e^{G_last-G_j} v_j E^T + scale sum_{i>=j} e^{G_i-G_j} (v_j do_i) q_i
//   dv_j = e^{G_last-G_j} k_j E + scale sum_{i>=j} e^{G_i-G_j} (k_j q_i) do_i
//   E'   = e^{G_last} E + scale sum_i e^{G_i} q_i do_i^T
// so one kernel does all of them: out = a S + (a b^T) c, S += b c^T, with
// (a, b, c) = (q, k, v), (do, v, k), (v, do, q) and (k, q, do), the last two
// from the last chunk to the first.  dg_t sums every pair i >= t > j, the
// states before and the gradients behind; per chunk
//   dg_t = e^{G_last} <S, E> + sum_{i>=t} (qs_i + R_i - C_i) + sum_{j<t} ks_j,
// qs_i = q_i times the state's part of dq_i, ks_i = k_i times that of dk_i,
// R and C the row and column sums of the pairs (q_i k_j)(do_i v_j) e^{G_i-G_j},
// j < i: sums of terms that a gate has decayed, so strong decays keep their digits.
// In the chunks before a segment's last one E itself is decayed, and
//   dg_t = <S', E> + sum_{i>=t} (qs_i + R_i - C_i - ks_i)
// carries the sum on, <S', E> being dg of the next chunk's first token.  (In the last one
// ks of the last token, k (dht v), has met no gate and would have to cancel.)
//
// A workgroup of four waves walks the chunks of one segment of one head.  Each
// wave owns a quarter of the columns of c and S; S stays in MFMA accumulators,
// whose layout is that of an operand over its own rows, so S never passes
// through LDS.  The pairs' products of the chunk are made once, a tile row to a
// wave, and handed round in LDS.  Long sequences are cut into segments: a first
// walk makes each segment's own state, launch_decay_join chains them (of few
// segments the walk itself), and the segments then run side by side.
//
// What bounds it: two workgroups fill a compute unit's registers and LDS, two
// waves to a SIMD, which take turns at the matrix unit, the vector ALU and LDS
// (of 64 tokens of a head the output walk has 150 matrix and 600 vector
// instructions a wave).  16 heads of 128 x 128 in bf16, 16384 tokens, medians of a
// trace: segments' states 38 us (134 MB read, 3.5 TB/s), output 71 us (268 MB,
// 3.8 TB/s; with the chaining of the states of eight segments), the three gradient walks
// together 257 us, the matrix unit busy for a quarter of it, the vector ALU and LDS for
// about two fifths each.  Eight waves of 16 columns each: 76 us for the output instead of 68, each
// then reads all of a and b for half as many products.
//
// Roundings: products are of the inputs' type, sums in 32 bits.  With bf16 the
// pairs' weights and the state are rounded to bf16 where they are multiplied
// into an output of that type.  Each is a rounding of factors of many terms, the two
// together as much as the output's own: o's error is 0.0023 of its norm, where its
// rounding alone makes 0.0017 (4 x 4096 tokens of 16 heads of 128); a second part would
// double the state's and the pairs' products.  Where
// a 32-bit result depends on them (the state itself, dg) the factor is split into
// three bf16 parts, 24 bits, and multiplied part by part.
#pragma once

#include "gdn_mixer.hpp"
#include "gdn_mma8.hpp"

namespace gdn {

// A chunk's rows on their way from memory to LDS: PER 16-byte units to each of NT threads.
// Past the chunk's n rows the last one is read again (the gates give those rows no
// weight).  Addresses are the rows' base in scalar registers and a 32-bit offset:
// token strides are below 2^24 elements.
template <typename T, int D, int NT> struct Ahead {
    typedef Rows<T, D> R;
    static constexpr int STEP = NT / R::UR, PER = 64 / STEP;     // rows between a thread's units
    u32x4 u[PER];
    __device__ __forceinline__ void load(const T* base, unsigned ts, int n, int tid) {
        unsigned at = tid;
        asm volatile("" : "+v"(at));   // (offsets made here are not kept over the loop)
        const unsigned tb = ts * sizeof(T), row = at / R::UR * tb, unit = at % R::UR * 16, last = (n - 1) * tb;
        const T* p = in_scalar(base);
#pragma unroll
        for (int i = 0; i < PER; ++i) u[i] = peek_row<u32x4>(p, min(row + STEP * i * tb, last) + unit);
    }
    __device__ __forceinline__ void put(const R& r, int tid) const {
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int q = tid + NT * i;
            *reinterpret_cast<u32x4*>(r.p + R::at(q / R::UR, q % R::UR * R::U)) = u[i];
        }
    }
};

// Gates of a chunk in log2, as a multiple of 1/16 and a rest of up to 1/32.  Running
// sums of the multiples are exact; those of the rests, below 2, are off by a few 2^-24
// (the sum of the gates themselves would lose the small ones behind a large one).  A gate below -150 (2^-150 is 0 in 32 bits)
// counts as -8192, whose power and every sum with it is 0: nothing passes it.
struct GateParts {
    float hi, lo;
};
__device__ __forceinline__ GateParts gate_parts(float g) {
    const float x = g * LOG2E;
    if (x < -150.f) return {-8192.f, 0.f};
    if (x > 8192.f) return {8192.f, 0.f};
    const float h = rintf(x * 16.f) * 0.0625f;
    return {h, fmaf(g, LOG2E, -h)};   // NaN stays one
}

// Inclusive prefix sum over the wave's 64 lanes, by DPP row shifts and broadcasts.
template <int CTRL, int MASK> __device__ __forceinline__ float dpp_from(float v) {
    return v + __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), CTRL, MASK, 0xf, false));
}
__device__ __forceinline__ float scan64(float x) {
    x = dpp_from<0x111, 0xf>(x);   // row_shr:1, 2, 4, 8
    x = dpp_from<0x112, 0xf>(x);
    x = dpp_from<0x114, 0xf>(x);
    x = dpp_from<0x118, 0xf>(x);
    x = dpp_from<0x142, 0xa>(x);   // row_bcast:15 into rows 1 and 3
    x = dpp_from<0x143, 0xc>(x);   // row_bcast:31 into rows 2 and 3
    return x;
}
__device__ __forceinline__ float lane_of(float x, int lane) {
    return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(x), lane));
}
// Sum of the lanes behind each lane: of its row of 16 by DPP row shifts, then the rows behind.
__device__ __forceinline__ float behind64(float x, int lane) {
    x = dpp_from<0x101, 0xf>(x);   // row_shl:1, 2, 4, 8
    x = dpp_from<0x102, 0xf>(x);
    x = dpp_from<0x104, 0xf>(x);
    x = dpp_from<0x108, 0xf>(x);
    const float t1 = lane_of(x, 16), t2 = lane_of(x, 32), t3 = lane_of(x, 48);
    x += lane < 16 ? t1 + (t2 + t3) : lane < 32 ? t2 + t3 : lane < 48 ? t3 : 0.f;
    const float y = __shfl_down(x, 1, 64);
    return lane < 63 ? y : 0.f;
}

// What the waves need of a chunk's gates: sums up to each token (reversed walks:
// from behind it), the factors of the state in and out, and of the whole chunk.
// Rows past the chunk's n tokens get sums that give every pair with them the weight
// 0, and factors of 0.
struct alignas(16) ChunkGates {
    float hi[64], lo[64], in[64], out[64];
    float dec;
};
// Token of the chunk whose gate a lane brings: reversed walks sum from the end, so that a gate that is
// not finite stays out of the sums behind it.
template <bool REV> __device__ __forceinline__ int gate_token(int lane) { return REV ? 63 - lane : lane; }
template <bool REV>
__device__ __forceinline__ void make_gates(ChunkGates& s, float g, int n, float in_scale, float up_scale, int lane) {
    const GateParts p = gate_parts(gate_token<REV>(lane) < n ? g : 0.f);
    float hi = scan64(p.hi), lo = scan64(p.lo);
    const float th = lane_of(hi, 63), tl = lane_of(lo, 63);
    int at = lane;
    if (REV) {     // a lane has the sum from its token on, which is the one behind the token before it
        at = lane < 63 ? 62 - lane : 63;
        if (lane == 63) hi = lo = 0.f;
    }
    const bool on = at < n;
    s.hi[at] = on ? hi : REV ? 8192.f * 64 : -8192.f * 64;
    s.lo[at] = lo;
    s.in[at] = on ? in_scale * exp2_hw(hi + lo) : 0.f;
    s.out[at] = on ? up_scale * exp2_hw((th - hi) + (tl - lo)) : 0.f;
    if (lane == 0) s.dec = exp2_hw(th + tl);
}

// DA: elements of a and b, DC: of c.  TR: the state in memory is S^T ([K][V] with DA = V).
// DOT: 1: the state's part of the output times x, for dg; 2: the pairs' sums as well.
template <typename T, int DA, int DC, bool REV, bool TR, int DOT, bool LOCAL>
struct DecayBody {
    typedef Eight<T> E8;
    typedef typename E8::frag frag;
    static constexpr int CT = DC / 64;        // tiles of 16 columns of a wave
    static constexpr int W = 4;               // waves
    static constexpr int KT = DA / 16;        // row tiles of S
    static constexpr int PW = 64 + 16 / sizeof(T);   // pitch of the pairs' rows

    // the gaps of the rows hold the sums for dg: a's and b's those of the waves' columns, c's
    // the pairs' column sums, x's their row sums
    struct Shared {
        T a[LOCAL ? 16 : 64 * Rows<T, DA>::PITCH], b[64 * Rows<T, DA>::PITCH], c[64 * Rows<T, DC>::PITCH];
        T x[DOT ? 64 * Rows<T, DC>::PITCH : 16];
        T pairs[LOCAL ? 16 : 64 * PW];
        ChunkGates gates[2];
        float ends[8];
    };

    // offset of S tile (kt, ct)'s element e in the state's memory; the two tiles of a wave interleave
    // by four columns, so that a lane's outputs are eight in a row
    __device__ __forceinline__ static int state_at(int w, int lane, int kt, int ct, int e) {
        const int g = lane >> 4, r = lane & 15, k = 16 * kt + 4 * g + e;
        const int c = CT == 2 ? 32 * w + 8 * (r >> 2) + 4 * ct + (r & 3) : 16 * w + r;
        return TR ? c * DA + k : k * DC + c;
    }

    // The forward's states between segments lie in the accumulators' order, 16 bytes of a lane
    // next to the next lane's (own_order of DecayJoin).
    static constexpr bool OWN = !TR && !REV;
    __device__ __forceinline__ static int own_at(int w, int lane, int kt, int ct) {
        return ((kt * CT + ct) * 4 + w) * 256 + lane * 4;
    }

    // the wave's share of dec <S, E>, E in memory (nullptr: zeros)
    __device__ __forceinline__ static void end_dot(const f32x4 (&S)[KT][CT], const float* e0, float dec, int w, int lane,
                                                   Shared& s) {
        float d = 0.f;
        if (e0) {
            asm volatile("" : "+v"(lane));   // (the addresses are made here)
#pragma unroll
            for (int kt = 0; kt < KT; ++kt)
#pragma unroll
                for (int ct = 0; ct < CT; ++ct) {
                    const f32x4 v = *reinterpret_cast<const f32x4*>(e0 + state_at(w, lane, kt, ct, 0));
#pragma unroll
                    for (int e = 0; e < 4; ++e) d += v[e] * S[kt][ct][e];
                }
        }
        d = wave_sum(d);
        if (lane == 0) s.ends[w] = dec * d;
    }

    // block: the workgroup's number among those of this walk
    __device__ static void run(const DecayWalk& p, unsigned block, Shared& s) {
        const int tid = threadIdx.x, lane = tid & 63, w = wave_id(), g16 = lane >> 4, r16 = lane & 15;
        // workgroups go to the eight XCDs in turn: the heads that share q and k are put on one, next
        // to each other, and read them through one L2
        const unsigned xcd = block & 7, slot = block >> 3, m = p.share, Hq = (unsigned)p.H / m;
        const unsigned unit = slot / m * 8 + xcd;
        const int64_t blk = unit / Hq, h = (unit - blk * Hq) * m + slot % m;
        if (blk >= p.tiles + (LOCAL ? 0 : p.singles)) return;   // (the grid is a multiple of 8 heads)
        const bool single = blk >= p.tiles;
        Tile t;
        if (single && p.map.seqs) {
            const int4 q = p.map.seqs[blk - p.tiles];
            t.row0 = __builtin_amdgcn_readfirstlane(q.x);
            t.len = __builtin_amdgcn_readfirstlane(q.y);
            if (t.len > p.map.tile) return;      // it has segments
            t.n = t.len;
            t.seq = (int)(blk - p.tiles);
            t.j = 0;
            t.nt = 1;
        } else if (single) {
            t = Tile{(blk - p.tiles) * p.map.T, (int)p.map.T, (int)(blk - p.tiles), 0, 1, (int)p.map.T};
        } else {
            t = tile_of(p.map, blk);
            if (t.n == 0) return;
            if (LOCAL && t.j == (REV ? 0 : t.nt - 1)) return;   // nothing follows it
        }
        const int nch = (t.n + 63) >> 6;
        const int64_t KV = (int64_t)DA * DC;

        const T* pa = LOCAL ? nullptr : static_cast<const T*>(p.a.p) + t.row0 * p.a.ts + (h / p.a.div) * p.a.hs;
        const T* pb = static_cast<const T*>(p.b.p) + t.row0 * p.b.ts + (h / p.b.div) * p.b.hs;
        const T* pc = static_cast<const T*>(p.c.p) + t.row0 * p.c.ts + (h / p.c.div) * p.c.hs;
        const T* px = DOT ? static_cast<const T*>(p.x.p) + t.row0 * p.x.ts + (h / p.x.div) * p.x.hs : nullptr;
        const float* pg = p.g + t.row0 * p.gs + h;

        const Rows<T, DA> ra{s.a}, rb{s.b};
        const Rows<T, DC> rc{s.c}, rx{s.x};
        Ahead<T, DA, 64 * W> na, nb;
        Ahead<T, DC, 64 * W> nc, nx;
        const auto first_of = [&](int j) { return 64 * (REV ? nch - 1 - j : j); };   // j-th chunk walked
        const auto fetch = [&](int j) {
            const int64_t t0 = first_of(j);
            const int n = min(64, t.n - (int)t0);
            if (!LOCAL) na.load(pa + t0 * p.a.ts, (unsigned)p.a.ts, n, tid);
            nb.load(pb + t0 * p.b.ts, (unsigned)p.b.ts, n, tid);
            nc.load(pc + t0 * p.c.ts, (unsigned)p.c.ts, n, tid);
            if (DOT) nx.load(px + t0 * p.x.ts, (unsigned)p.x.ts, n, tid);
        };
        const auto gate_of = [&](int j) {
            const int at = min(first_of(j) + gate_token<REV>(lane), t.n - 1);
            return pg[at * p.gs];
        };

        constexpr int GW = REV ? 1 : 2;   // a wave with one block of pairs makes the gates
        float gfirst = 0.f, gnext = 0.f;
        if (nch > 0) {
            fetch(0);
            if (w == GW) {
                gfirst = gate_of(0);
                if (nch > 1) gnext = gate_of(1);
            }
        }
        f32x4 S[KT][CT];
        const bool chained = OWN && !LOCAL && !single && t.nt <= p.chain;
        const float* sin = LOCAL ? nullptr
                           : single || chained ? (p.seq_state ? p.seq_state + (t.seq * p.H + h) * KV : nullptr)
                                    : p.tile_state + (blk * p.H + h) * KV;
        if (!sin) {
#pragma unroll
            for (int kt = 0; kt < KT; ++kt)
#pragma unroll
                for (int ct = 0; ct < CT; ++ct) S[kt][ct] = zero4();
        } else if (OWN && !single && !chained) {
#pragma unroll
            for (int kt = 0; kt < KT; ++kt)
#pragma unroll
                for (int ct = 0; ct < CT; ++ct)
                    S[kt][ct] = *reinterpret_cast<const f32x4*>(sin + own_at(w, lane, kt, ct));
        } else {
#pragma unroll
            for (int kt = 0; kt < KT; ++kt)
#pragma unroll
                for (int ct = 0; ct < CT; ++ct) {
                    if constexpr (TR) {
                        S[kt][ct] = *reinterpret_cast<const f32x4*>(sin + state_at(w, lane, kt, ct, 0));
                    } else {
#pragma unroll
                        for (int e = 0; e < 4; ++e) S[kt][ct][e] = sin[state_at(w, lane, kt, ct, e)];
                    }
                }
        }
        if (chained) {       // as launch_decay_join would
            const int64_t step = p.H * KV;
            const float *own = p.tile_state + ((blk - t.j) * p.H + h) * KV, *d = p.dec + (blk - t.j) * p.H + h;
            for (int j = 0; j < t.j; ++j, own += step, d += p.H) {
                const float dj = *d;
#pragma unroll
                for (int kt = 0; kt < KT; ++kt)
#pragma unroll
                    for (int ct = 0; ct < CT; ++ct) {
                        const f32x4 x = *reinterpret_cast<const f32x4*>(own + own_at(w, lane, kt, ct));
#pragma unroll
                        for (int e = 0; e < 4; ++e) S[kt][ct][e] = fmaf(dj, S[kt][ct][e], x[e]);
                    }
            }
        }
        float total = 1.f;   // LOCAL: decay of the segment
        // DOT 2: the gradient behind the segment
        const float* e0 = DOT != 2 ? nullptr
                          : single ? (p.seq_end ? p.seq_end + (t.seq * p.H + h) * KV : nullptr)
                                   : p.tile_end + (blk * p.H + h) * KV;

        if (nch > 0 && w == GW)
            make_gates<REV>(s.gates[0], gfirst, t.n - first_of(0), p.in_scale, p.up_scale, lane);
        for (int j = 0; j < nch; ++j) {
            if (!LOCAL) na.put(ra, tid);
            nb.put(rb, tid);
            nc.put(rc, tid);
            if (DOT) nx.put(rx, tid);
            lds_barrier();
            const ChunkGates& gt = s.gates[j & 1];
            if (w == GW && j + 1 < nch) {
                make_gates<REV>(s.gates[(j + 1) & 1], gnext, t.n - first_of(j + 1), p.in_scale, p.up_scale, lane);
                if (j + 2 < nch) gnext = gate_of(j + 2);
            }

            if constexpr (DOT == 2) {   // what reaches the gradient behind the last chunk from before it
                if (j + 1 == nch) end_dot(S, e0, gt.dec, w, lane, s);
            }

            // What the others wait for at the next barrier goes before the other workgroup's products
            // (4 x 4096 tokens of 16 heads: output 68 -> 65 us, dq 114 -> 105, dk 102 -> 91).
            __builtin_amdgcn_s_setprio(1);
            // ---- pairs: blocks of 16 rows and 32 columns of a b^T, transposed in the accumulators
            // (rows b's tokens), as the products read them.  Of the six that reach the diagonal or
            // lie before it each wave has one of its own rows, and two waves another one.
            int rr = r16, gg = g16;
            asm volatile("" : "+v"(rr), "+v"(gg));   // (addresses made from these are not kept over the loop)
            if constexpr (!LOCAL) {
                const auto block = [&](int it, int js) {
                    const int i = 16 * it + rr;
                    f32x4 P[2] = {zero4(), zero4()};
#pragma unroll
                    for (int q = 0; q < DA / 32; ++q) {
                        const frag af = ra.row8(i, 32 * q + 8 * gg);
#pragma unroll
                        for (int u = 0; u < 2; ++u)
                            P[u] = E8::mma(rb.row8(32 * js + 16 * u + rr, 32 * q + 8 * gg), af, P[u]);
                    }
                    const float hi = gt.hi[i], lo = gt.lo[i];
#pragma unroll
                    for (int u = 0; u < 2; ++u) {
                        const int j0 = 32 * js + 16 * u + 4 * gg;
                        const f32x4 jh = *reinterpret_cast<const f32x4*>(&gt.hi[j0]);
                        const f32x4 jl = *reinterpret_cast<const f32x4*>(&gt.lo[j0]);
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const float y = P[u][e] * (p.pair_scale * exp2_hw((hi - jh[e]) + (lo - jl[e])));
                            P[u][e] = (REV ? j0 + e >= i : j0 + e <= i) ? y : 0.f;
                        }
                        store4(s.pairs + i * PW + 32 * js + 8 * gg + 4 * u, P[u]);
                    }
                    if constexpr (DOT == 2) {
                        f32x4 M[2] = {zero4(), zero4()};
#pragma unroll
                        for (int q = 0; q < DC / 32; ++q) {
                            const frag xf = rx.row8(i, 32 * q + 8 * gg);
#pragma unroll
                            for (int u = 0; u < 2; ++u)
                                M[u] = E8::mma(rc.row8(32 * js + 16 * u + rr, 32 * q + 8 * gg), xf, M[u]);
                        }
                        float rsum = 0.f;
#pragma unroll
                        for (int u = 0; u < 2; ++u) {
                            const int j0 = 32 * js + 16 * u + 4 * gg;
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                M[u][e] = j0 + e < i ? M[u][e] * P[u][e] : 0.f;
                                rsum += M[u][e];
                            }
                            const f32x4 cs = row_sum16(M[u]);
                            if (rr == 15) {
#pragma unroll
                                for (int e = 0; e < 4; ++e) rc.gap(j0 + e)[it] = cs[e];
                            }
                        }
                        rsum = sum_groups(rsum);
                        if (gg == 0) rx.gap(i)[js] = rsum;
                    }
                };
                block(w, REV ? 1 : 0);
                if (REV ? w >= 2 : w < 2) block(3 - w, REV ? 0 : 1);
                if constexpr (DOT == 2) {
                    if (w < 2 && gg < 2) rc.gap(32 + 16 * gg + rr)[w] = 0.f;   // no pairs there
                    if (w < 2 && gg == 0) rx.gap(16 * w + rr)[1] = 0.f;
                }
            }

            __builtin_amdgcn_sched_barrier(0);   // phases kept apart: fewer registers at once
            // ---- the state's part: O^T = S^T a^T, rows the wave's columns, columns the tokens
            f32x4 O[4][CT];
            if constexpr (!LOCAL) {
                constexpr int NP = DOT ? E8::PARTS : 1;
#pragma unroll
                for (int it = 0; it < 4; ++it)
#pragma unroll
                    for (int ct = 0; ct < CT; ++ct) O[it][ct] = zero4();
#pragma unroll
                for (int q = 0; q < DA / 32; ++q) {
                    frag sf[CT][NP];
#pragma unroll
                    for (int ct = 0; ct < CT; ++ct) {
                        float f[8];
#pragma unroll
                        for (int e = 0; e < 8; ++e) f[e] = S[2 * q + (e >> 2)][ct][e & 3];
                        E8::template split<NP>(f, sf[ct]);
                    }
#pragma unroll
                    for (int it = 0; it < 4; ++it) {
                        const frag b = ra.row44(16 * it + r16, 32 * q + 4 * g16);
#pragma unroll
                        for (int n = 0; n < NP; ++n)
#pragma unroll
                            for (int ct = 0; ct < CT; ++ct) O[it][ct] = E8::mma(sf[ct][n], b, O[it][ct]);
                    }
                }
#pragma unroll
                for (int it = 0; it < 4; ++it) {
                    const int i = 16 * it + rr;
                    const float f = gt.in[i];
                    float d = 0.f;
#pragma unroll
                    for (int ct = 0; ct < CT; ++ct) {
#pragma unroll
                        for (int e = 0; e < 4; ++e) O[it][ct][e] *= f;
                        if constexpr (DOT != 0) {
                            const f32x4 xv = rx.row4(i, 16 * CT * w + 4 * CT * gg + 4 * ct);
#pragma unroll
                            for (int e = 0; e < 4; ++e) d += O[it][ct][e] * xv[e];
                        }
                    }
                    if constexpr (DOT != 0) {
                        d = sum_groups(d);
                        if (gg == 0) ra.gap(i)[w] = d;
                    }
                }
            }

            __builtin_amdgcn_sched_barrier(0);
            __builtin_amdgcn_s_setprio(0);
            // the next chunk's rows: not earlier, for their registers
            if (j + 1 < nch) fetch(j + 1);
            // ---- the state: S <- dec S + b^T (out c)
            frag cf[2][CT];
#pragma unroll
            for (int js = 0; js < 2; ++js)
#pragma unroll
                for (int ct = 0; ct < CT; ++ct)
                    cf[js][ct] = rc.template col8<CT == 2>(32 * js, 16 * CT * w + 4 * ct, lane);
            const float dec = gt.dec;
            if (LOCAL) total *= dec;
#pragma unroll
            for (int kt = 0; kt < KT; ++kt)
#pragma unroll
                for (int ct = 0; ct < CT; ++ct)
#pragma unroll
                    for (int e = 0; e < 4; ++e) S[kt][ct][e] *= dec;
#pragma unroll
            for (int js = 0; js < 2; ++js) {
                frag cp[CT][E8::PARTS];
                const f32x4 wl = *reinterpret_cast<const f32x4*>(&gt.out[32 * js + 4 * g16]);
                const f32x4 wh = *reinterpret_cast<const f32x4*>(&gt.out[32 * js + 16 + 4 * g16]);
#pragma unroll
                for (int ct = 0; ct < CT; ++ct) {
                    float f[8];
                    E8::unpack(cf[js][ct], f);
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        f[e] *= wl[e];
                        f[4 + e] *= wh[e];
                    }
                    E8::template split<E8::PARTS>(f, cp[ct]);
                }
#pragma unroll
                for (int kt = 0; kt < KT; kt += 2) {
                    frag b[2];
#pragma unroll
                    for (int u = 0; u < 2; ++u) b[u] = rb.template col8<false>(32 * js, 16 * (kt + u), lane);
#pragma unroll
                    for (int n = 0; n < E8::PARTS; ++n)      // (sums that do not wait for each other)
#pragma unroll
                        for (int u = 0; u < 2; ++u)
#pragma unroll
                            for (int ct = 0; ct < CT; ++ct) S[kt + u][ct] = E8::mma(b[u], cp[ct][n], S[kt + u][ct]);
                }
            }

            if constexpr (!LOCAL) {
                // A value of c that is not finite has made its column of S so.  It may not reach, as 0
                // times itself, the outputs that do not see it: such a chunk goes token by token.
                bool odd = false;
#pragma unroll
                for (int ct = 0; ct < CT; ++ct) odd |= !(__builtin_fabsf(S[0][ct][0]) < INFINITY);
                lds_barrier();   // the pairs of all tile rows are there
                if (__builtin_expect(__any(odd), 0)) {
#pragma unroll
                    for (int it = 0; it < 4; ++it) {
                        const int i = 16 * it + rr;
#pragma unroll 1
                        for (int m = REV ? i : 0; m <= (REV ? min(63, t.n - first_of(j) - 1) : i); ++m) {
                            const int at = (m & 32) + 8 * (m >> 2 & 3) + 4 * (m >> 4 & 1) + (m & 3);   // as put
                            const float y = Elem<T>::load(s.pairs + i * PW + at);
#pragma unroll
                            for (int ct = 0; ct < CT; ++ct) {
                                const f32x4 v = rc.row4(m, 16 * CT * w + 4 * CT * gg + 4 * ct);
#pragma unroll
                                for (int e = 0; e < 4; ++e) O[it][ct][e] = fmaf(y, v[e], O[it][ct][e]);
                            }
                        }
                    }
                } else {
#pragma unroll
                for (int it = 0; it < 4; ++it)
#pragma unroll
                    for (int js = 0; js < 2; ++js) {
                        if (REV ? 2 * js + 1 < it : 2 * js > it) continue;
                        frag b;
                        const T* q = s.pairs + (16 * it + r16) * PW + 32 * js + 8 * g16;
                        if constexpr (sizeof(T) == 2) {
                            b = *reinterpret_cast<const frag*>(q);
                        } else {
                            b = __builtin_shufflevector(reinterpret_cast<const f32x4*>(q)[0],
                                                        reinterpret_cast<const f32x4*>(q)[1], 0, 1, 2, 3, 4, 5, 6, 7);
                        }
#pragma unroll
                        for (int ct = 0; ct < CT; ++ct) O[it][ct] = E8::mma(cf[js][ct], b, O[it][ct]);
                    }
                }
                const int64_t t0 = first_of(j);
                const int n = min(64, t.n - (int)t0);
                const int64_t first = ((t.row0 + t0) * p.H + h) * DC;
                unsigned at = (unsigned)r16 * (unsigned)(p.H * DC) + 16 * CT * w + 4 * CT * g16;
                asm volatile("" : "+v"(at));   // (a 64-bit form of it would be kept over the loop)
#pragma unroll
                for (int it = 0; it < 4; ++it) {
                    if (r16 >= n - 16 * it) continue;
                    const int64_t row = first + 16 * it * p.H * DC;
                    if (sizeof(T) == 4 || p.out32) {
                        float* q = in_scalar((p.out32 ? p.out32 : static_cast<float*>(p.out)) + row);
#pragma unroll
                        for (int ct = 0; ct < CT; ++ct) poke_row(q, (at + 4 * ct) * 4, O[it][ct]);
                    } else {
                        unsigned x[2 * CT];
#pragma unroll
                        for (int ct = 0; ct < CT; ++ct) {
                            x[2 * ct] = pack_bf16x2(O[it][ct][0], O[it][ct][1]);
                            x[2 * ct + 1] = pack_bf16x2(O[it][ct][2], O[it][ct][3]);
                        }
                        T* q = in_scalar(static_cast<T*>(p.out) + row);
                        if constexpr (CT == 2) poke_row(q, at * 2, u32x4{x[0], x[1], x[2], x[3]});
                        else poke_row(q, at * 2, u32x2{x[0], x[1]});
                    }
                }
                if constexpr (DOT != 0) {
                    if (tid < n) {
                        const auto four = [](const float* q) {
                            const f32x4 v = *reinterpret_cast<const f32x4*>(q);
                            return (v[0] + v[1]) + (v[2] + v[3]);
                        };
                        float d = four(ra.gap(tid));
                        if constexpr (DOT == 2) d += (rx.gap(tid)[0] + rx.gap(tid)[1]) - four(rc.gap(tid));
                        p.dots[h * p.tokens + t.row0 + t0 + tid] = d;
                    }
                }
            }
            lds_barrier();   // everything of this chunk has been read
        }

        // the state's addresses made anew: kept over the loop they would take a third of the registers
        int lane2 = lane;
        asm volatile("" : "+v"(lane2));
        float* sout = LOCAL ? p.local + (blk * p.H + h) * KV
                      : (p.seq_out && t.j == (REV ? 0 : t.nt - 1)) ? p.seq_out + (t.seq * p.H + h) * KV : nullptr;
        if (sout) {
#pragma unroll
            for (int kt = 0; kt < KT; ++kt)
#pragma unroll
                for (int ct = 0; ct < CT; ++ct) {
                    if constexpr (OWN && LOCAL) {
                        *reinterpret_cast<f32x4*>(sout + own_at(w, lane2, kt, ct)) = S[kt][ct];
                    } else if constexpr (TR) {
                        *reinterpret_cast<f32x4*>(sout + state_at(w, lane2, kt, ct, 0)) = S[kt][ct];
                    } else {
#pragma unroll
                        for (int e = 0; e < 4; ++e) sout[state_at(w, lane2, kt, ct, e)] = S[kt][ct][e];
                    }
                }
        }
        if (LOCAL && tid == 0) p.dec[blk * p.H + h] = total;
        if constexpr (DOT == 2) {
            __syncthreads();
            if (tid == 0 && nch > 0) {
                float all = 0.f;
                for (int i = 0; i < W; ++i) all += s.ends[i];
                p.ends[blk * p.H + h] = all;
            }
        }
    }
};

// workgroups of a walk, a multiple of 8 heads' (see run)
inline unsigned walk_blocks(const DecayWalk& p, bool local) {
    const int64_t units = (p.tiles + (local ? 0 : p.singles)) * (p.H / p.share);
    return (unsigned)((units + 7) / 8 * 8 * p.share);
}

}  // namespace gdn
