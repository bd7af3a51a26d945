// What the layer operators share: the tile table of packed input, and the sums
// of partial rows that make the gradients of parameters.
//
// The tile table: tiles of `tile`
// tokens that restart at every sequence start, made on the device from the
// caller's cu_seqlens.  Offsets are clamped into [0, T] (end >= start), and a
// sequence whose tiles do not all fit the table (which takes offsets that
// decrease) is taken as empty, so invalid ones give wrong results but never an
// access out of bounds or a wait for a tile that is not there.
//
// One workgroup: a prefix sum over the sequences' tile counts, 1024 at a time;
// each thread writes its sequence's first row, then each wave the other rows
// of whole sequences, 64 at a time.  5 us for a few sequences.
#include "gdn_layer.hpp"

namespace gdn {

// row j of sequence n: q = (first token, length, first row, rows)
__device__ __forceinline__ void put(const TileTableLaunch& a, const int4& q, int64_t n, int64_t j) {
    a.table[q.z + j] = q.y == 0 ? TileRow{}
                                : TileRow{(int)(q.x + j * a.tile), (int)min((int64_t)a.tile, q.y - j * a.tile), (int)n,
                                          (int)j, q.w, q.y, {0, 0}};
}

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
            nc = len <= a.shorts ? 0 : (len + a.tile - 1) / a.tile;
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
        if (nc > 0 && before + inc > a.max_tiles) len = 0;
        s_seq[tid] = make_int4((int)s, (int)len, (int)first, (int)min(nc, a.max_tiles - first));
        if (n < a.N) a.seqs[n] = make_int4((int)s, (int)len, (int)first, 0);
        __syncthreads();
        if (n < a.N && s_seq[tid].w > 0) put(a, s_seq[tid], n, 0);
        const int mine = wave + 16 * lane;             // the wave's sequences are every 16th
        for (uint64_t m = __ballot(base + mine < a.N && s_seq[mine].w > 1); m; m &= m - 1) {
            const int i = wave + 16 * (__ffsll((unsigned long long)m) - 1);
            const int4 q = s_seq[i];
            for (int64_t j = 1 + lane; j < q.w; j += 64) put(a, q, base + i, j);
        }
        carry += total;
    }
    for (int64_t c = carry + tid; c < a.max_tiles; c += 1024) a.table[c] = TileRow{};
    __syncthreads();   // every thread's check of the offsets is in s_bad
    if (tid == 0) {
        a.words[0] = s_bad;
        a.words[1] = 0;
        a.words[2] = (int)min(carry, a.max_tiles);
    }
}

// A workgroup takes 64 columns and a share of the rows: 16 strands of rows to a
// column, 8 loads of a strand in flight, met in LDS.  With many rows and few
// columns the rows are shared out over a.shares workgroups and their sums
// added by a second launch: one workgroup per 64 columns would leave most of
// the chip idle (4103 rows of 256 columns: 28 us by 16 workgroups; of a backward
// with 2559 rows of 8192 columns it saves 25 us of 314).  Where the columns
// are many, the second launch costs more than it saves (627 rows of 20480 columns:
// 130 -> 162 us).
template <bool LAST>
__global__ __launch_bounds__(1024) void row_sum_kernel(RowSumLaunch a) {
    __shared__ double s[16][64];
    const int64_t cols = a.count * a.D;
    const unsigned nb = (unsigned)((cols + 63) / 64), share = blockIdx.x / nb;
    const int64_t col = (int64_t)(blockIdx.x - share * nb) * 64 + (threadIdx.x & 63);
    const int strand = threadIdx.x >> 6;
    double v = 0;
    if (col < cols) {
        if (LAST && a.shares > 1) {
            for (int64_t i = strand; i < a.shares; i += 16) v += a.sums[i * cols + col];
        } else {
            const int64_t rows = a.used ? a.rows - a.most + *a.used : a.rows;
            const int64_t per = (rows + a.shares - 1) / a.shares, end = min(rows, (share + 1) * per);
            const float* p = a.part + col;
            for (int64_t i = share * per + strand; i < end; i += 8 * 16) {
                float x[8];
#pragma unroll
                for (int k = 0; k < 8; ++k) x[k] = i + k * 16 < end ? p[(i + k * 16) * cols] : 0.f;
#pragma unroll
                for (int k = 0; k < 8; ++k) v += x[k];
            }
        }
    }
    s[strand][threadIdx.x & 63] = v;
    __syncthreads();
    if (strand != 0 || col >= cols) return;
    for (int i = 1; i < 16; ++i) v += s[i][threadIdx.x];
    if (!LAST) {
        a.sums[share * cols + col] = v;
        return;
    }
    const int64_t j = col / a.D, c = col - j * a.D;
    if (j < a.W) {
        if (a.out0) a.out0[c * a.W + j] = (float)v;
    } else if (a.out1) {
        a.out1[c] = (float)v;
    }
}

int64_t row_sum_shares(int64_t rows, int64_t cols) { return rows > 512 && rows > cols / 8 ? 32 : 1; }

hipError_t launch_row_sum(const RowSumLaunch& in) {
    RowSumLaunch a = in;
    const int64_t cols = a.count * a.D, nb = (cols + 63) / 64;
    a.shares = row_sum_shares(a.rows, cols);
    if (a.shares > 1) {
        hipLaunchKernelGGL((row_sum_kernel<false>), dim3((unsigned)(nb * a.shares)), dim3(1024), 0, a.stream, a);
        hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    hipLaunchKernelGGL((row_sum_kernel<true>), dim3((unsigned)nb), dim3(1024), 0, a.stream, a);
    return hipGetLastError();
}

hipError_t launch_tile_table(const TileTableLaunch& a) {
    hipLaunchKernelGGL(tile_table_kernel, dim3(1), dim3(1024), 0, a.stream, a);
    return hipGetLastError();
}

}  // namespace gdn
