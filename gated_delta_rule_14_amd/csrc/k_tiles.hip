// The tile table of packed input for the layer operators: tiles of `tile`
// tokens that restart at every sequence start, made on the device from the
// caller's cu_seqlens.  Offsets are clamped into [0, T] (end >= start), so
// invalid ones give wrong results but never an access out of bounds.
//
// One workgroup: a prefix sum over the sequences' tile counts, 1024 at a
// time, then each wave writes the rows of whole sequences, 64 at a time.
#include "gdn_layer.hpp"

namespace gdn {

__global__ __launch_bounds__(1024) void tile_table_kernel(TileTableLaunch a) {
    __shared__ int64_t s_sum[16];
    __shared__ int4 s_seq[1024];
    __shared__ int s_bad;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    int64_t carry = 0;
    if (tid == 0) s_bad = 0;
    for (int64_t base = 0; base < a.N; base += 1024) {
        __syncthreads();
        const int64_t n = base + tid;
        int64_t s = 0, len = 0, nc = 0;
        if (n < a.N) {
            const int64_t rs = a.cu_seqlens[n], re = a.cu_seqlens[n + 1];
            if (re < rs || (n == 0 && rs != 0) || (n == a.N - 1 && re != a.T)) atomicOr(&s_bad, 1);
            s = min(max(rs, (int64_t)0), a.T);
            len = min(max(re, s), a.T) - s;
            nc = (len + a.tile - 1) / a.tile;
        }
        int64_t inc = nc;                               // inclusive scan over the wave
        for (int off = 1; off < 64; off <<= 1) {
            const int64_t y = __shfl_up(inc, off, 64);
            if (lane >= off) inc += y;
        }
        if (lane == 63) s_sum[wave] = inc;
        __syncthreads();
        int64_t before = carry, total = 0;
        for (int w = 0; w < 16; ++w) {
            if (w < wave) before += s_sum[w];
            total += s_sum[w];
        }
        const int64_t first = min(before + inc - nc, a.max_tiles);
        s_seq[tid] = make_int4((int)s, (int)len, (int)first, (int)nc);
        if (n < a.N) a.seqs[n] = make_int4((int)s, (int)len, (int)first, 0);
        __syncthreads();
        for (int i = wave; i < 1024 && base + i < a.N; i += 16) {
            const int4 q = s_seq[i];
            for (int64_t j = lane; j < q.w && q.z + j < a.max_tiles; j += 64)
                a.table[q.z + j] = TileRow{(int)(q.x + j * a.tile), (int)min((int64_t)a.tile, q.y - j * a.tile),
                                           (int)(base + i), (int)j, q.w, q.y, {0, 0}};
        }
        carry += total;
    }
    for (int64_t c = carry + tid; c < a.max_tiles; c += 1024) a.table[c] = TileRow{};
    __syncthreads();   // every thread's check of the offsets is in s_bad
    if (tid == 0) {
        a.words[0] = s_bad;
        a.words[1] = 0;
    }
}

hipError_t launch_tile_table(const TileTableLaunch& a) {
    hipLaunchKernelGGL(tile_table_kernel, dim3(1), dim3(1024), 0, a.stream, a);
    return hipGetLastError();
}

}  // namespace gdn
