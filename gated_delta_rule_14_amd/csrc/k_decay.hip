// Linear attention with a decay for each head: the gradients' walks of segments
// alone, the chaining of the segments' states, the gates' gradient and the
// single-token step.  The chunk walk itself, its mathematics and its figures are in
// k_decay.hpp.
#include "k_decay.hpp"

namespace gdn {

// The segments' own states, forward (b, c) = (k, v) for the output; for the gradients
// those of S^T, (v, k), and of E^T, (do, q) from the end, in one launch: each alone
// leaves a fifth of the chip idle at its end.
template <typename T, int DA, int DC>
__global__ __launch_bounds__(256, sizeof(T) == 2 ? 3 : 1) void decay_local2_kernel(DecayWalk f, DecayWalk r, unsigned half) {
    typedef DecayBody<T, DA, DC, false, true, 0, true> F;
    typedef DecayBody<T, DA, DC, true, true, 0, true> R;
    __shared__ typename F::Shared s;
    static_assert(sizeof(typename F::Shared) == sizeof(typename R::Shared), "one layout");
    if (blockIdx.x < half) F::run(f, blockIdx.x, s);
    else R::run(r, blockIdx.x - half, reinterpret_cast<typename R::Shared&>(s));
}
template <typename T, int K, int V>
static hipError_t local2(const DecayWalk& f, const DecayWalk& r) {
    const unsigned half = walk_blocks(f, true);
    if (half == 0) return hipSuccess;
    hipLaunchKernelGGL((decay_local2_kernel<T, V, K>), dim3(2 * half), dim3(256), 0, f.stream, f, r, half);
    return hipGetLastError();
}
hipError_t launch_decay_local2(const DecayWalk& f, const DecayWalk& r, int K, int V, bool bf) {
    if (K == 64 && V == 64) return bf ? local2<bf16, 64, 64>(f, r) : local2<float, 64, 64>(f, r);
    if (K == 64 && V == 128) return bf ? local2<bf16, 64, 128>(f, r) : local2<float, 64, 128>(f, r);
    if (K == 128 && V == 64) return bf ? local2<bf16, 128, 64>(f, r) : local2<float, 128, 64>(f, r);
    if (K == 128 && V == 128) return bf ? local2<bf16, 128, 128>(f, r) : local2<float, 128, 128>(f, r);
    return hipErrorInvalidValue;
}

// S_0 = first, S_{j+1} = dec_j S_j + local_j over a sequence's segments; S_j takes
// the place of local_j.  A workgroup takes 1024 elements of a sequence's state.  Bound by
// HBM, each state in and out: 2 x 8192 tokens of 16 heads of 128, 512 segments, 14 us.
__device__ __forceinline__ void join(const DecayJoin& a, unsigned block) {
    const int64_t per = (a.KV + 1023) / 1024, hb = a.H * per;
    const int64_t i = block / hb, c = a.map.table ? i : i * a.map.nt, rest = block - i * hb, h = rest / per;
    const int64_t e = (rest - h * per) * 1024 + threadIdx.x * 4;
    const Tile t = tile_of(a.map, c);
    if (t.n == 0 || t.j != 0 || t.nt <= a.chain || e >= a.KV) return;
    f32x4 s = zero4();
    if (a.first) {
        const float* first = a.first + (t.seq * a.H + h) * a.KV;
        if (a.own_order) {                 // element e in the walk's order (DecayBody::own_at, state_at)
            const int ct2 = a.V == 128, i = (int)e >> 2, lane = i & 63, w = i >> 6 & 3, tile = i >> 8;
            const int kt = tile >> ct2, ct = tile & ct2, r = lane & 15;
            const int k = 16 * kt + 4 * (lane >> 4), c = ct2 ? 32 * w + 8 * (r >> 2) + 4 * ct + (r & 3) : 16 * w + r;
#pragma unroll
            for (int x = 0; x < 4; ++x) s[x] = first[(k + x) * a.V + c];
        } else {
            s = *reinterpret_cast<const f32x4*>(first + e);
        }
    }
    // eight segments' states on their way at a time: one after the other they would each
    // be waited for
    constexpr int U = 8;
    const int64_t step = a.rev ? -1 : 1, at = c + (a.rev ? t.nt - 1 : 0);
    for (int j0 = 0; j0 < t.nt; j0 += U) {
        f32x4 own[U];
        float d[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t row = (at + (j0 + u) * step) * a.H + h;
            if (j0 + u + 1 < t.nt) {       // (the last one walked has no local state)
                own[u] = *reinterpret_cast<const f32x4*>(a.state + row * a.KV + e);
                d[u] = a.dec[row];
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (j0 + u >= t.nt) break;
            *reinterpret_cast<f32x4*>(a.state + ((at + (j0 + u) * step) * a.H + h) * a.KV + e) = s;
            if (j0 + u + 1 < t.nt) {
#pragma unroll
                for (int i = 0; i < 4; ++i) s[i] = fmaf(d[u], s[i], own[u][i]);
            }
        }
    }
}
__global__ __launch_bounds__(256) void decay_join_kernel(DecayJoin a, DecayJoin b, unsigned half) {
    if (blockIdx.x < half) join(a, blockIdx.x);
    else join(b, blockIdx.x - half);
}

hipError_t launch_decay_join(const DecayJoin& a, const DecayJoin* b) {
    if (a.tiles == 0) return hipSuccess;
    // a sequence's first segment: every table row might be one
    const int64_t half = (a.map.table ? a.tiles : a.map.N) * a.H * ((a.KV + 1023) / 1024);
    hipLaunchKernelGGL(decay_join_kernel, dim3((unsigned)(b ? 2 * half : half)), dim3(256), 0, a.stream, a, b ? *b : a,
                       (unsigned)half);
    return hipGetLastError();
}

// dg_t = the product of the state before the segment's last chunk and the gradient behind
// it, plus the dots of dq and dk that the walks left (k_decay.hpp): from t on those of dq,
// less those of dk, of the last chunk those of dk before t instead.  Carried in 64 bits from 256
// tokens to the next; 0 where the gate lets nothing through.  A workgroup
// takes a segment of a head from its end.  With one gate for each head only the
// segment's sum goes out (3 x 1001 tokens of 6 heads, with the sum over the segments:
// 16 -> 9 us).
__global__ __launch_bounds__(256) void decay_gate_kernel(DecayGate a) {
    __shared__ float s_sum[2][4];
    __shared__ double s_all[4];
    const int tid = threadIdx.x, lane = tid & 63, w = wave_id();
    const int64_t blk = blockIdx.x / a.H, h = blockIdx.x - blk * a.H;
    int64_t row0;
    int n;
    if (blk < a.tiles) {
        const Tile t = tile_of(a.map, blk);
        row0 = t.row0;
        n = t.n;
    } else if (a.map.seqs) {
        const int4 q = a.map.seqs[blk - a.tiles];
        row0 = q.x;
        n = q.y > a.map.tile ? 0 : q.y;
    } else {
        row0 = (blk - a.tiles) * a.map.T;
        n = (int)a.map.T;
    }
    double carry = n > 0 ? (double)a.ends[blk * a.H + h] : 0.0;
    const float *dq = a.dq + h * a.tokens + row0, *dk = a.dk + h * a.tokens + row0;
    const float* g = a.g + row0 * a.gs + h;
    int first = (n + 255) / 256 * 256 - 256, turn = 0;     // thread 0 takes the last token
    int t = first + 255 - tid;
    float x = 0.f, gt = 0.f, before_t = 0.f;
    double all = 0.0;
    const bool end = t >> 6 == (n - 1) >> 6;               // (a wave's 64 tokens are a chunk)
    if (n > 0 && t < n) {
        x = end ? dq[t] : dq[t] - dk[t];
        gt = g[t * a.gs];
    }
    if (n > 0 && end) before_t = behind64(t < n ? dk[t] : 0.f, lane);   // lanes behind: tokens before
    for (; first >= 0; first -= 256, t -= 256, turn ^= 1, before_t = 0.f) {
        const float now = scan64(x), gn = gt;
        if (first > 0) {                                   // the next ones are on their way
            x = dq[t - 256] - dk[t - 256];
            gt = g[(t - 256) * a.gs];
        }
        if (lane == 63) s_sum[turn][w] = now;
        __syncthreads();
        const float s0 = s_sum[turn][0], s1 = s_sum[turn][1], s2 = s_sum[turn][2], s3 = s_sum[turn][3];
        const double before = carry + (w > 0 ? (double)s0 : 0.0) + (w > 1 ? (double)s1 : 0.0) + (w > 2 ? (double)s2 : 0.0);
        const double y = gate_parts(gn).hi == -8192.f ? 0.0 : before + now + before_t;
        if (t < n) {
            if (a.part) all += y;
            else a.dg[(row0 + t) * a.H + h] = (float)y;
        }
        carry += ((double)s0 + s1) + ((double)s2 + s3);
    }
    if (!a.part) return;
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) all += __shfl_xor(all, off, 64);
    if (lane == 0) s_all[w] = all;
    __syncthreads();
    if (tid == 0) a.part[blk * a.H + h] = (float)((s_all[0] + s_all[1]) + (s_all[2] + s_all[3]));
}

hipError_t launch_decay_gate(const DecayGate& a) {
    const int64_t blocks = (a.tiles + a.singles) * a.H;
    if (blocks == 0) return hipSuccess;
    hipLaunchKernelGGL(decay_gate_kernel, dim3((unsigned)blocks), dim3(256), 0, a.stream, a);
    return hipGetLastError();
}

// One token: S <- e^g S + k v^T, o = scale q S, the state read and written once.
// A workgroup takes VS columns of a state; thread t the four columns t % (VS / 4)
// of its rows, all on their way before the token's own values are needed.  Bound by
// HBM: 256 requests of 32 heads of 128 x 128, 1.08 GB in and out, 161 us in a trace
// and 212 back to back (5.1 TB/s; a copy reaches 4.9); 8 requests of 16 heads 5 us.
template <typename T, int K, int V, int VS>
__global__ __launch_bounds__(256) void decay_step_kernel(DecayStep a) {
    constexpr int CG = VS / 4, RG = 256 / CG, ROWS = K / RG, NS = V / VS;
    static_assert(CG * RG == 256 && ROWS * RG == K, "shape");
    __shared__ float s_q[K], s_k[K];
    __shared__ f32x4 s_o[RG][CG];
    const int64_t pair = blockIdx.x / NS;
    const int slice = (int)(blockIdx.x - pair * NS), tid = threadIdx.x, cg = tid % CG, rg = tid / CG;
    const int64_t n = pair / a.H, h = pair - n * a.H;
    const int col = slice * VS + 4 * cg;
    float* st = a.state + pair * (K * V) + (int64_t)rg * ROWS * V + col;
    f32x4 s[ROWS];
#pragma unroll
    for (int i = 0; i < ROWS; ++i) s[i] = *reinterpret_cast<const f32x4*>(st + i * V);
    const T* q = static_cast<const T*>(a.q.p) + n * a.q.ts + (h / a.q.div) * a.q.hs;
    const T* k = static_cast<const T*>(a.k.p) + n * a.k.ts + (h / a.k.div) * a.k.hs;
    const T* v = static_cast<const T*>(a.v.p) + n * a.v.ts + h * a.v.hs + col;
    const f32x4 vv = Quad<T>::get(Quad<T>::load(v));
    const float d = expf(a.g[n * a.gs + h]);
    if (tid < K) {
        s_q[tid] = Elem<T>::load(q + tid);
        s_k[tid] = Elem<T>::load(k + tid);
    }
    __syncthreads();
    f32x4 o = zero4();
#pragma unroll
    for (int i = 0; i < ROWS; ++i) {
        const float kr = s_k[rg * ROWS + i], qr = s_q[rg * ROWS + i];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            s[i][e] = fmaf(d, s[i][e], kr * vv[e]);
            o[e] = fmaf(qr, s[i][e], o[e]);
        }
        __builtin_nontemporal_store(s[i], reinterpret_cast<f32x4*>(st + i * V));
    }
    s_o[rg][cg] = o;
    __syncthreads();
    if (rg != 0) return;
    for (int i = 1; i < RG; ++i) {
        const f32x4 x = s_o[i][cg];
#pragma unroll
        for (int e = 0; e < 4; ++e) o[e] += x[e];
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) o[e] *= a.scale;
    store4(static_cast<T*>(a.o) + pair * V + col, o);
}

template <typename T, int K, int V>
static hipError_t step_of(const DecayStep& a) {
    // a state is cut into slices of 32 columns where whole states would not fill the chip twice
    const int64_t pairs = a.N * a.H;
    if (pairs < 512)
        hipLaunchKernelGGL((decay_step_kernel<T, K, V, 32>), dim3((unsigned)(pairs * (V / 32))), dim3(256), 0, a.stream, a);
    else
        hipLaunchKernelGGL((decay_step_kernel<T, K, V, V>), dim3((unsigned)pairs), dim3(256), 0, a.stream, a);
    return hipGetLastError();
}
template <typename T>
static hipError_t step_dt(const DecayStep& a) {
    if (a.K == 64) return a.V == 64 ? step_of<T, 64, 64>(a) : step_of<T, 64, 128>(a);
    return a.V == 64 ? step_of<T, 128, 64>(a) : step_of<T, 128, 128>(a);
}
hipError_t launch_decay_step(const DecayStep& a) {
    if (a.N * a.H == 0) return hipSuccess;
    return a.bf16 ? step_dt<bf16>(a) : step_dt<float>(a);
}

}  // namespace gdn
