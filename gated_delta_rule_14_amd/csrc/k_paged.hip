// A paged cache of keys and values: the append with the norm and the rotation
// on the way, and the attention of one new token over it.
//
// The cache is a pool of pages of `page` tokens; row n of the table lists the
// pages of sequence n.  A token whose page is not there (past the table, or an
// entry outside the pool) is not written and not attended to, so no table or
// length can lead out of the pool.
#include <algorithm>

#include "gdn_mixer.hpp"
#include "gdn_mma8.hpp"
#include "gdn_rope.hpp"

namespace gdn {

// offset of token `pos` of sequence n in pages counted in tokens: (page, slot); page < 0: not there
template <typename A>
__device__ __forceinline__ int2 slot_of(const A& a, int64_t n, int64_t pos) {
    if (pos < 0 || pos >= a.M * a.page) return make_int2(-1, 0);
    const unsigned pg = (unsigned)pos / (unsigned)a.page;    // M * page is below 2^30
    const int id = a.table[n * a.M + pg];
    return make_int2((unsigned)id < (unsigned)a.pages ? id : -1, (int)((unsigned)pos - pg * (unsigned)a.page));
}

// ---------------------------------------------------------------- append
// As in qk_norm_rope a wave takes a token: its angles once, then its rows; q's
// go out, k's to their page, and v's are copied to theirs.  Few tokens share
// their rows out over several waves.
template <typename T, int LPR, bool INTER>
__global__ __launch_bounds__(256) void append_kernel(PagedAppend a) {
    __shared__ float2 s_cs[4][128];
    constexpr int RPW = 64 / LPR;
    const QkLaunch& p = a.qk;
    const int lane = threadIdx.x & 63, w = wave_id();
    const int64_t task = (int64_t)blockIdx.x * 4 + w, all = p.tokens * p.split;
    if (task >= all) return;
    const int64_t token = task / p.split, part = task - token * p.split;
    int64_t n, t;
    bool live = true;
    if (a.cu) {
        // the last sequence that starts at or before the token: 64 probes at a time
        int64_t lo = 0, hi = a.N;
        while (hi - lo > 1) {
            const int64_t step = (hi - lo + 63) / 64, at = lo + (lane + 1) * step;
            lo += step * __popcll(__ballot(at < hi && a.cu[at] <= token));
            lo = min(lo, hi - 1);
            hi = min(lo + step, hi);
        }
        n = lo;
        t = token - a.cu[n];
        live = t >= 0 && token < a.cu[n + 1];
    } else {
        n = token / p.T;
        t = token - n * p.T;
    }
    const int64_t len = a.lens[n], pos = len + t;
    int2 at = slot_of(a, n, live && len >= 0 && len <= a.M * a.page ? pos : -1);
    const int page = __builtin_amdgcn_readfirstlane(at.x), slot = __builtin_amdgcn_readfirstlane(at.y);
    Spin<INTER> spin;
    spin_at<INTER>(p, p.R > 0 && p.positions ? p.positions[token] : pos, s_cs[w], lane, lane % LPR, &spin);
    // this wave's share of the token's row groups: q's, k's, then v's by 512 elements
    const int64_t gq = (p.Hq + RPW - 1) / RPW, gk = (p.Hk + RPW - 1) / RPW, gv = (p.Hk * p.D + 511) / 512;
    const int64_t per = (gq + gk + gv + p.split - 1) / p.split, b = part * per, e = min(b + per, gq + gk + gv);
    if (b < gq)
        heads_fwd<T, LPR, INTER>(p, spin, static_cast<const T*>(p.q) + token * p.qs,
                                 static_cast<T*>(p.qo) + token * p.Hq * p.D, p.qw, p.qhs, p.D, b * RPW,
                                 min(e * RPW, p.Hq), lane, true);
    if (page < 0) return;
    if (e > gq && b < gq + gk)
        heads_fwd<T, LPR, INTER>(p, spin, static_cast<const T*>(p.k) + token * p.ks,
                                 static_cast<T*>(a.kc.p) + page * a.kc.ps + slot * a.kc.ts, p.kw, p.khs, a.kc.hs,
                                 (max(b, gq) - gq) * RPW, min((e - gq) * RPW, p.Hk), lane, true);
    if (e > gq + gk) {
        const T* v = static_cast<const T*>(a.v) + token * a.vs;
        T* out = static_cast<T*>(a.vc.p) + page * a.vc.ps + slot * a.vc.ts;
        const int64_t end = min((e - gq - gk) * 512, p.Hk * p.D);
        for (int64_t i = (max(b, gq + gk) - gq - gk) * 512 + lane * 8; i < end; i += 512) {
            const int64_t h = i / p.D, d = i - h * p.D;
            Oct<T> r;
            r.load(v + h * a.vhs + d);
            T* o = out + h * a.vc.hs + d;
            if constexpr (sizeof(T) == 2) {
                *reinterpret_cast<uint4*>(o) = r.r;
            } else {
                reinterpret_cast<float4*>(o)[0] = r.a;
                reinterpret_cast<float4*>(o)[1] = r.b;
            }
        }
    }
}

template <typename T, int LPR, bool INTER>
static hipError_t append2(const PagedAppend& in) {
    PagedAppend a = in;
    const int64_t rpw = 64 / LPR;
    const int64_t groups = (a.qk.Hq + rpw - 1) / rpw + (a.qk.Hk + rpw - 1) / rpw + (a.qk.Hk * a.qk.D + 511) / 512;
    // waves for at least half of the chip's slots, as in qk_norm_rope
    a.qk.split = std::min(groups, std::max((int64_t)1, 4096 / a.qk.tokens));
    hipLaunchKernelGGL((append_kernel<T, LPR, INTER>), dim3((unsigned)((a.qk.tokens * a.qk.split + 3) / 4)), dim3(256), 0,
                       a.qk.stream, a);
    return hipGetLastError();
}
template <typename T, bool INTER>
static hipError_t append1(const PagedAppend& a) {
    if (a.qk.D <= 32) return append2<T, 4, INTER>(a);
    if (a.qk.D <= 64) return append2<T, 8, INTER>(a);
    if (a.qk.D <= 128) return append2<T, 16, INTER>(a);
    return append2<T, 32, INTER>(a);
}
hipError_t launch_paged_append(const PagedAppend& a) {
    if (a.qk.tokens == 0) return hipSuccess;
    if (a.qk.bf16) return a.qk.interleaved ? append1<bf16, true>(a) : append1<bf16, false>(a);
    return a.qk.interleaved ? append1<float, true>(a) : append1<float, false>(a);
}

// ------------------------------------------------- attention of one token
// o = sum_t p_t v_t / sum_t p_t, p_t = exp(scale q k_t - m), with the running
// maximum m and sum of a softmax taken in one pass over the keys and values.
//
// The sequences' tokens are cut into pieces of one size, chosen so that all
// sequences together make about `share` pieces whatever their lengths; a
// workgroup takes a piece for one key head and up to 16 of the query heads that
// share it, and a second launch joins the pieces of the sequences that have
// several.  Its four waves take 32 tokens in turn (16 of heads wider than 128, so that
// keys and values on their way and the output fit the registers of two workgroups to a
// compute unit), each with a maximum, sum and output of its own, and meet at the end.
//
// Scores are K Q^T, tokens in the accumulator's rows, so they are at once the
// operand of the output's product V^T P^T, whose V^T comes out of LDS by
// transposing reads.  With bf16 the weights go into that product in two parts,
// 16 bits, whose error of 2^-16 is lost in the output's rounding of 2^-8 (in one part it
// would be as large); the sum that divides them keeps 32.
//
// Bound by HBM: 16 requests of 20000 to 65536 tokens (3.0 GB of keys and values,
// 8 heads of 128) 545 us, 5.5 TB/s; 64 of 1 to 8192 (2 heads of 256) 146 us,
// 4.4 TB/s.  One request of 1000 tokens: 8 us, the look-ups of length and page, three
// turns of loads and the meeting of the waves, and 4 us for the join.
constexpr int UNIT = 128;       // tokens that a piece is a multiple of
constexpr int MOST = 1 << 23;   // units of a sequence at most (a table's row is below 2^30 tokens)

// Units of a piece where all sequences together have `all`.  No piece needs more than a sequence has; the
// quotient alone passes 31 bits with 2048 key heads (one piece) and 256 rows of 2^30 tokens that share pages.
constexpr int piece_units(int64_t all, int64_t share) {
    const int64_t per = (all + share - 1) / share;
    return per < 1 ? 1 : per > MOST ? MOST : (int)per;
}
static_assert(piece_units(0, 7) == 1 && piece_units(8, 7) == 2 && piece_units(14, 7) == 2, "rounded up");
static_assert(piece_units((int64_t)512 << 23, 1) == MOST && piece_units((int64_t)1 << 54, 1) == MOST, "in 31 bits");

struct Piece {
    int64_t n;                  // sequence; < 0: none
    int first, last;            // tokens [first, last) as multiples of 32 from below, last cut at the length
    int lo;                     // first token attended to
    int count, index;           // pieces of the sequence, and which one this is
    int64_t base;               // number of its first piece
};

// the sequence's tokens: [lo, len)
__device__ __forceinline__ void range_of(const PagedAttn& a, int64_t n, int* lo, int* len) {
    const int64_t x = min(max(a.lens[n], (int64_t)0), a.M * a.page);
    *len = (int)x;
    *lo = a.window > 0 && a.window < x ? (int)(x - a.window) : 0;
}
__device__ __forceinline__ int units_of(int lo, int len) { return (len - (lo & ~31) + UNIT - 1) / UNIT; }

// Piece number `at` (of sequence `seq` if that is not negative: its first one); the whole
// wave calls it.  A piece has as many units as the sum over the sequences asks for.
__device__ __forceinline__ Piece find_piece(const PagedAttn& a, int64_t at, int64_t seq, int lane) {
    int lo0 = 0, len0 = 0;                        // the first 64 sequences' stay in registers
    if (lane < a.N) range_of(a, lane, &lo0, &len0);
    int64_t all = units_of(lo0, len0);
    for (int64_t b = 64; b < a.N; b += 64) {
        int lo = 0, len = 0;
        if (b + lane < a.N) range_of(a, b + lane, &lo, &len);
        all += units_of(lo, len);
    }
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) all += __shfl_xor(all, off, 64);
    const int per = piece_units(all, a.share);
    Piece p;
    p.n = -1;
    int64_t before = 0;
    for (int64_t b = 0; b < a.N; b += 64) {
        int lo = lo0, len = len0, cnt = 0;
        if (b + lane < a.N) {
            if (b > 0) range_of(a, b + lane, &lo, &len);
            cnt = max(1, (units_of(lo, len) + per - 1) / per);
        }
        int inc = cnt;
#pragma unroll
        for (int off = 1; off < 64; off <<= 1) {
            const int y = __shfl_up(inc, off, 64);
            if (lane >= off) inc += y;
        }
        const uint64_t hit = __ballot(seq >= 0 ? b + lane == seq : before + inc > at);
        if (hit) {
            const int i = __ffsll((unsigned long long)hit) - 1;
            const int c = __shfl(cnt, i, 64), l0 = __shfl(lo, i, 64), ln = __shfl(len, i, 64);
            p.n = b + i;
            p.base = before + __shfl(inc, i, 64) - c;
            p.count = c;
            p.index = (int)(at - p.base);
            p.lo = l0;
            const int64_t f = (l0 & ~31) + (int64_t)p.index * per * UNIT;
            p.first = (int)f;
            p.last = (int)min((int64_t)ln, f + (int64_t)per * UNIT);
            return p;
        }
        before += __shfl(inc, 63, 64);
    }
    return p;
}

template <typename T, int D>
__global__ __launch_bounds__(256, sizeof(T) == 2 ? 2 : 1) void attn_kernel(PagedAttn a) {
    typedef Eight<T> E8;
    typedef typename E8::frag frag;
    typedef Rows<T, D> R;
    constexpr int TT = D <= 128 ? 32 : 16, TH = TT / 16, TURN = 4 * TT;   // tokens of a wave and of the four in a turn
    constexpr int UR = R::UR, NV = TT * UR / 64;     // 16-byte units of a row; units of a tile of V to a lane
    constexpr int DT = D / 16, KS = D / 32, NP = sizeof(T) == 2 ? 2 : 1;
    __shared__ __attribute__((aligned(16))) union {
        T v[4][TT * Rows<T, D>::PITCH];
        float o[4][16 * D];
    } s;
    __shared__ float s_m[4][16], s_l[4][16];

    const int tid = threadIdx.x, lane = tid & 63, w = wave_id(), g = lane >> 4, r = lane & 15;
    const int m = a.Hq / a.Hk;
    const int kv = blockIdx.y, h0 = kv * m + 16 * blockIdx.z, nh = min(16, m - 16 * (int)blockIdx.z);
    const Piece pc = find_piece(a, blockIdx.x, -1, lane);
    if (pc.n < 0) return;
    const int64_t n = pc.n;

    const T* kc = static_cast<const T*>(a.kc.p) + kv * a.kc.hs;
    const T* vc = static_cast<const T*>(a.vc.p) + kv * a.vc.hs;
    frag qf[KS];
#pragma unroll
    for (int s_ = 0; s_ < KS; ++s_) {
        float f[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
        const int d = 32 * s_ + 8 * g;
        if (r < nh && d < a.D) {
            Oct<T> x;
            x.load(static_cast<const T*>(a.q) + n * a.qs + (h0 + r) * a.qhs + d);
#pragma unroll
            for (int e = 0; e < 8; ++e) f[e] = x.get(e);
        }
        qf[s_] = E8::pack(f);
    }

    const R vt{s.v[w]};
    frag kf[TH][KS];
    u32x4 vf[NV];
    unsigned seen = 0;
    // the page and slot of token t0 + lane % TT, if it is seen
    const auto look = [&](int t0) {
        const int t = t0 + (lane & (TT - 1));
        return slot_of(a, n, t >= pc.lo && t < pc.last ? t : -1);
    };
    // keys and values of TT tokens that are seen; zeros for the others
    const auto fetch = [&](int2 at) {
        seen = (unsigned)__ballot(at.x >= 0);
        const int64_t ko = at.x * a.kc.ps + at.y * a.kc.ts, vo = at.x * a.vc.ps + at.y * a.vc.ts;
#pragma unroll
        for (int h = 0; h < TH; ++h) {
            const T* p = kc + __shfl(ko, 16 * h + r, 64) + 8 * g;
#pragma unroll
            for (int q = 0; q < KS; ++q) {
                const bool on = (seen >> (16 * h + r) & 1) && 32 * q + 8 * g < a.D;
                if constexpr (sizeof(T) == 2) {
                    u32x4 x = {0, 0, 0, 0};
                    if (on) x = *reinterpret_cast<const u32x4*>(p + 32 * q);
                    kf[h][q] = __builtin_bit_cast(frag, x);
                } else {
                    frag x = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
                    if (on) {
                        const f32x4* y = reinterpret_cast<const f32x4*>(p + 32 * q);
                        x = __builtin_shufflevector(y[0], y[1], 0, 1, 2, 3, 4, 5, 6, 7);
                    }
                    kf[h][q] = x;
                }
            }
        }
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int q = lane + 64 * i, row = q / UR, d = q % UR * R::U;
            const int64_t off = __shfl(vo, row, 64);
            vf[i] = u32x4{0, 0, 0, 0};
            if ((seen >> row & 1) && d < a.D) vf[i] = *reinterpret_cast<const u32x4*>(vc + off + d);
        }
    };

    f32x4 O[DT];
#pragma unroll
    for (int i = 0; i < DT; ++i) O[i] = zero4();
    float mx = -INFINITY, sum = 0.f;
    int t0 = pc.first + TT * w;
    int2 next = make_int2(-1, 0);
    if (t0 < pc.last) {
        fetch(look(t0));
        next = look(t0 + TURN);        // (a turn ahead: the table's latency is not waited for)
    }
    for (; t0 < pc.last; t0 += TURN) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int q = lane + 64 * i;
            *reinterpret_cast<u32x4*>(vt.p + R::at(q / UR, q % UR * R::U)) = vf[i];
        }
        __builtin_amdgcn_wave_barrier();   // (the wave's own rows: its LDS accesses stay in order)
        f32x4 S[TH];
#pragma unroll
        for (int h = 0; h < TH; ++h) {
            S[h] = zero4();
#pragma unroll
            for (int q = 0; q < KS; ++q) S[h] = E8::mma(kf[h][q], qf[q], S[h]);
        }
        const unsigned in = seen;
        if (t0 + TURN < pc.last) {
            fetch(next);
            next = look(t0 + 2 * TURN);
        }
        float x[8], top = -INFINITY;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            x[e] = -INFINITY;
            if (e < 4 * TH) {
                const int t = 16 * (e >> 2) + 4 * g + (e & 3);
                if (in >> t & 1) x[e] = S[(e >> 2) % TH][e & 3] * a.scale;
                top = fmaxf(top, x[e]);
            }
        }
        top = fmaxf(top, __shfl_xor(top, 16, 64));
        top = fmaxf(top, __shfl_xor(top, 32, 64));
        const float m1 = fmaxf(mx, top), ref = m1 == -INFINITY ? 0.f : m1;
        const float keep = exp2_hw(mx - ref);
        mx = m1;
        float l = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            x[e] = exp2_hw(x[e] - ref);
            l += x[e];
        }
        sum = sum * keep + l;
        frag pf[NP];
        E8::template split<NP>(x, pf);
#pragma unroll
        for (int i = 0; i < DT; ++i) {
#pragma unroll
            for (int e = 0; e < 4; ++e) O[i][e] *= keep;
            const frag v = TT == 32 ? vt.template col8<false>(0, 16 * i, lane) : vt.col4(16 * i, lane);
#pragma unroll
            for (int k = 0; k < NP; ++k) O[i] = E8::mma(v, pf[k], O[i]);
        }
    }
    sum = sum_groups(sum);
    if (g == 0) {
        s_m[w][r] = mx;
        s_l[w][r] = sum;
    }
    __syncthreads();
    const float M = fmaxf(fmaxf(s_m[0][r], s_m[1][r]), fmaxf(s_m[2][r], s_m[3][r]));
    const float ref = M == -INFINITY ? 0.f : M, f = exp2_hw(mx - ref);
#pragma unroll
    for (int i = 0; i < DT; ++i) {
        f32x4 v = O[i];
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] *= f;
        *reinterpret_cast<f32x4*>(&s.o[w][r * D + 16 * i + 4 * g]) = v;
    }
    __syncthreads();
    const bool whole = pc.count == 1;
    const int64_t at = blockIdx.x;
    for (int i = tid; i < 16 * D / 4; i += 256) {
        const int h = i / (D / 4), d = i % (D / 4) * 4;
        if (h >= nh || d >= a.D) continue;
        f32x4 v = zero4();
#pragma unroll
        for (int k = 0; k < 4; ++k) v += *reinterpret_cast<const f32x4*>(&s.o[k][h * D + d]);
        float mh = fmaxf(fmaxf(s_m[0][h], s_m[1][h]), fmaxf(s_m[2][h], s_m[3][h]));
        const float rh = mh == -INFINITY ? 0.f : mh;
        float lh = 0.f;
#pragma unroll
        for (int k = 0; k < 4; ++k) lh += s_l[k][h] * exp2_hw(s_m[k][h] - rh);
        if (whole) {
            const float inv = lh > 0.f || lh != lh ? 1.f / lh : 0.f;
#pragma unroll
            for (int e = 0; e < 4; ++e) v[e] *= inv;
            store4(static_cast<T*>(a.o) + (n * a.Hq + h0 + h) * a.D + d, v);
        } else {
            *reinterpret_cast<f32x4*>(a.part + (at * a.Hq + h0 + h) * a.D + d) = v;
            if (d == 0) {
                a.ml[(at * a.Hq + h0 + h) * 2] = mh;
                a.ml[(at * a.Hq + h0 + h) * 2 + 1] = lh;
            }
        }
    }
}

// The pieces of a sequence that has several: o = sum of theirs, each times
// exp(m_piece - m), over the sum of l alike.  A workgroup takes a head.
template <typename T>
__global__ __launch_bounds__(256) void join_kernel(PagedAttn a) {
    __shared__ f32x4 s_o[256];
    __shared__ float s_l[256];
    const int tid = threadIdx.x, lane = tid & 63;
    const int64_t n = blockIdx.x / a.Hq, h = blockIdx.x - n * a.Hq;
    const Piece p = find_piece(a, 0, n, lane);
    if (p.count <= 1) return;
    const int C = a.D / 4, G = 256 / C, grp = tid / C, c = tid % C;   // D is a multiple of 8 up to 256
    float M = -INFINITY;
    for (int i = lane; i < p.count; i += 64) M = fmaxf(M, a.ml[((p.base + i) * a.Hq + h) * 2]);
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) M = fmaxf(M, __shfl_xor(M, off, 64));
    const float ref = M == -INFINITY ? 0.f : M;
    f32x4 o = zero4();
    float l = 0.f;
    if (grp < G)
        for (int i = grp; i < p.count; i += G) {
            const int64_t row = (p.base + i) * a.Hq + h;
            const float f = exp2_hw(a.ml[row * 2] - ref);
            const f32x4 x = *reinterpret_cast<const f32x4*>(a.part + row * a.D + 4 * c);
#pragma unroll
            for (int e = 0; e < 4; ++e) o[e] = fmaf(f, x[e], o[e]);
            l = fmaf(f, a.ml[row * 2 + 1], l);
        }
    s_o[tid] = o;
    s_l[tid] = l;
    __syncthreads();
    if (grp != 0) return;
    for (int i = 1; i < G; ++i) {
        o += s_o[i * C + c];
        l += s_l[i * C + c];
    }
    const float inv = l > 0.f || l != l ? 1.f / l : 0.f;
#pragma unroll
    for (int e = 0; e < 4; ++e) o[e] *= inv;
    store4(static_cast<T*>(a.o) + (n * a.Hq + h) * a.D + 4 * c, o);
}

// Pieces that all sequences together are cut into: eight workgroups to a compute unit,
// so that they end together without too many starts (16 requests of 20000 to 65536
// tokens: 541 us, with half as many 589, with twice as many 532; 64 of 1 to 8192, wide
// heads: 147, 151 and 157 us).
int64_t paged_attn_share(int64_t Hq, int64_t Hk) {
    const int64_t per = Hk * ((Hq / Hk + 15) / 16);
    return std::max((int64_t)1, 2048 / per);
}

template <typename T>
static hipError_t attn_of(const PagedAttn& in) {
    PagedAttn a = in;
    // no more pieces than the table's rows have units: each workgroup without one still
    // costs its start (2000 of them 3 us)
    const int64_t most = a.window > 0 ? std::min(a.M * a.page, a.window) : a.M * a.page;
    a.share = std::min(a.share, a.N * ((most + UNIT - 1) / UNIT + 1));
    const dim3 grid((unsigned)(a.share + a.N), (unsigned)a.Hk, (unsigned)((a.Hq / a.Hk + 15) / 16));
    if (a.D <= 64)
        hipLaunchKernelGGL((attn_kernel<T, 64>), grid, dim3(256), 0, a.stream, a);
    else if (a.D <= 128)
        hipLaunchKernelGGL((attn_kernel<T, 128>), grid, dim3(256), 0, a.stream, a);
    else
        hipLaunchKernelGGL((attn_kernel<T, 256>), grid, dim3(256), 0, a.stream, a);
    hipError_t e = hipGetLastError();
    // a table of one unit cannot be cut
    if (e != hipSuccess || a.M * a.page <= UNIT) return e;
    hipLaunchKernelGGL((join_kernel<T>), dim3((unsigned)(a.N * a.Hq)), dim3(256), 0, a.stream, a);
    return hipGetLastError();
}
hipError_t launch_paged_attn(const PagedAttn& a) {
    if (a.N == 0) return hipSuccess;
    return a.bf16 ? attn_of<bf16>(a) : attn_of<float>(a);
}

}  // namespace gdn
