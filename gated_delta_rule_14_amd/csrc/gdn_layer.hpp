// Internal launcher interface of the layer operators (gated linear
// recurrence, q/k norm with rotation, short convolution) between
// gdn_layer_api.hip and their kernel translation units, and the device
// helpers these share.  Not part of the public ABI.
#pragma once

#include "../../include/gdn.h"
#include "gdn_device.hpp"
#include "gdn_launch.hpp"

namespace gdn {

// error reporting of the C ABI (gdn_api.hip): the status, with its detail
// left for gdn_last_error()
gdn_status api_fail(gdn_status s, const char* fmt, ...) __attribute__((format(printf, 2, 3)));
gdn_status api_ok();

// A row's address, held in scalar registers (the row is the same for the whole
// wave, the channel a 32-bit byte offset of it): left to itself the compiler
// adds the channel to the tensor's base first, and every row then costs a
// 64-bit vector addition and two vector registers while its load is in flight.
#define GDN_GLOBAL __attribute__((address_space(1)))
template <typename T> __device__ __forceinline__ T* in_scalar(T* row) {
    asm("" : "+s"(row));
    return row;
}
template <typename U> __device__ __forceinline__ U peek_row(const void* row, unsigned off) {
    return *(const GDN_GLOBAL U*)((const GDN_GLOBAL char*)row + off);
}
template <typename U> __device__ __forceinline__ void poke_row(void* row, unsigned off, U v) {
    *(GDN_GLOBAL U*)((GDN_GLOBAL char*)row + off) = v;
}

// Tiles of `tile` tokens that never cross a sequence.  Without packed offsets
// tile c is tokens (c % nt) * tile .. of sequence c / nt; with them a table
// built on the device has a row for each, all that a workgroup needs in one load.
struct TileRow {
    int row0, n, seq, j;   // first token, tokens (0: unused row), sequence, tile of its sequence
    int nt, len, pad[2];   // tiles and tokens of the sequence
};
struct SeqMap {
    const TileRow* table = nullptr;   // [max_tiles] or nullptr
    const int4* seqs = nullptr;    // [N] (first token, length, first tile, 0) or nullptr
    int64_t T = 0;                 // tokens per sequence when table == nullptr
    int64_t nt = 0;                // tiles per sequence when table == nullptr
    int64_t N = 0;
    int64_t max_tiles = 0;
    int tile = 0;
    int shorts = 0;                // > 0: tile c is sequence c where it has at most this many
                                   // tokens, and unused where it has more (seqs != nullptr)
};

struct Tile {
    int64_t row0;   // first token (row of the activations)
    int n;          // tokens; 0: unused
    int seq;
    int j, nt;      // tile j of the nt of its sequence
    int len;        // tokens of the sequence
};

// c is the same for the whole wave, and so is what comes back: in scalar
// registers, for the row addresses
__device__ __forceinline__ Tile tile_of(const SeqMap& m, int64_t c) {
    Tile t;
    if (m.shorts) {
        const int4 s = m.seqs[c];
        t.row0 = __builtin_amdgcn_readfirstlane(s.x);
        t.len = __builtin_amdgcn_readfirstlane(s.y);
        t.n = t.len <= m.shorts ? t.len : 0;
        t.seq = (int)c;
        t.j = 0;
        t.nt = 1;
    } else if (m.table) {
        const TileRow r = m.table[c];
        t.row0 = __builtin_amdgcn_readfirstlane(r.row0);
        t.n = __builtin_amdgcn_readfirstlane(r.n);
        t.seq = __builtin_amdgcn_readfirstlane(r.seq);
        t.j = __builtin_amdgcn_readfirstlane(r.j);
        t.nt = __builtin_amdgcn_readfirstlane(r.nt);
        t.len = __builtin_amdgcn_readfirstlane(r.len);
    } else {
        const unsigned nt = (unsigned)m.nt, b = (unsigned)c / nt;   // both below 2^31
        t.j = (int)((unsigned)c - b * nt);
        t.seq = (int)b;
        const int64_t at = (int64_t)t.j * m.tile;
        t.row0 = b * m.T + at;
        t.n = (int)min((int64_t)m.tile, m.T - at);
        t.nt = (int)nt;
        t.len = (int)m.T;
    }
    return t;
}

// Packed offsets to the table of SeqMap; words[0] = the check of the offsets,
// words[2] = the rows in use (the others are at the end).
// Sequences of up to `shorts` tokens get no tile (they run by SeqMap::shorts).
struct TileTableLaunch {
    const int64_t* cu_seqlens;
    int64_t N, T, max_tiles;
    int tile, shorts;
    TileRow* table;
    int4* seqs;
    int* words;
    hipStream_t stream;
};
hipError_t launch_tile_table(const TileTableLaunch& a);

// Gradients of parameters: the sums of `rows` partial rows [count][D], in a
// fixed order and 64 bits.  Parts 0 .. W-1 of a row go to out0 [D][W] (W >= 1),
// part W to out1 [D]; either may be nullptr.
struct RowSumLaunch {
    const float* part;
    int64_t rows, D;
    int W, count;
    float *out0, *out1;
    double* sums;                 // [shares][count][D], used where shares > 1
    hipStream_t stream;
    int64_t shares = 1;           // set by the launch
    const int* used = nullptr;    // or the last `most` rows are only so many (a device word)
    int64_t most = 0;
};
int64_t row_sum_shares(int64_t rows, int64_t cols);
hipError_t launch_row_sum(const RowSumLaunch& a);

constexpr int TICKET = 32;        // word of the ticket counter, a cache line away from the others
struct LinrecLaunch {
    SeqMap map;
    Act act;                      // ACT_GATE: A_log, dt_bias [D]
    bool normalize = false;
    const void *x = nullptr, *g = nullptr, *dy = nullptr;
    const float *h0 = nullptr, *dht = nullptr;
    void *y = nullptr, *dx = nullptr, *dg = nullptr;
    float *ht = nullptr, *dh0 = nullptr, *dA_log = nullptr, *ddt_bias = nullptr;
    // Sequences of up to 16 or 64 tokens run without hand-offs: all of an unpacked call's
    // (small: which of the two, 0: tiles of map.tile), or the packed ones among others (shorts)
    int small = 0, shorts = 0;
    float* states = nullptr;      // [max_tiles][D] the states entering the tiles
    bool own_states = false;      // backward: states is workspace, to be filled first
    float* part = nullptr;        // [N with shorts, then max_tiles][2][D] sums of dA_log and ddt_bias (backward)
    double* sums = nullptr;       // shares of the sums of part
    // hand-offs between the tiles of a sequence; nullptr where every sequence is one tile
    uint64_t *pairs = nullptr, *groups = nullptr;   // [max_tiles][D], [max_tiles / 16 + 1][D]
    bool keep_status = false;     // clear: words[1] is already this call's
    int* words = nullptr;         // check of the offsets, failed waits, table rows in use; [TICKET]
    int64_t D = 0, xs = 0, gs = 0, ys = 0;   // channels; token strides of x, g, y / dy
    bool x_bf16 = false, g_bf16 = false;
    hipStream_t stream = nullptr;
};
hipError_t launch_linrec_fwd(const LinrecLaunch& a);
hipError_t launch_linrec_bwd(const LinrecLaunch& a);
hipError_t launch_linrec_step(const LinrecLaunch& a);

struct QkLaunch {
    const void *q, *k;
    const float *qw, *kw;
    const double* inv_freq;
    const int64_t* positions;
    void *qo, *ko;                // forward: outputs; backward: dq, dk
    const void *dqo = nullptr, *dko = nullptr;
    float *dqw = nullptr, *dkw = nullptr, *part = nullptr;
    double* sums = nullptr;       // shares of the sums of part
    int64_t tokens, T, Hq, Hk, qs, ks, qhs, khs;
    int64_t split = 1;            // waves to a token (forward)
    int D, R, norm;
    bool interleaved, bf16;
    float eps, offset;
    hipStream_t stream;
};
int64_t qk_bwd_blocks(int64_t tokens);   // rows of part [blocks][2][D]
hipError_t launch_qk(const QkLaunch& a);
hipError_t launch_qk_bwd(const QkLaunch& a);

struct ConvLaunch {
    SeqMap map;
    const void *x = nullptr, *s0 = nullptr, *dy = nullptr, *dst = nullptr;
    const float *w = nullptr, *b = nullptr;
    void *y = nullptr, *st = nullptr, *dx = nullptr, *ds0 = nullptr;
    float *dw = nullptr, *db = nullptr;
    float* part = nullptr;         // [tiles / 4, rounded up][W + 1][D] sums of dweight and dbias
    double* sums = nullptr;        // shares of the sums of part
    int64_t D = 0, xs = 0, ys = 0;
    int W = 0;
    bool silu = false, bf16 = false;
    hipStream_t stream = nullptr;
};
hipError_t launch_conv_fwd(const ConvLaunch& a);
hipError_t launch_conv_bwd(const ConvLaunch& a);
hipError_t launch_conv_step(const ConvLaunch& a);

}  // namespace gdn
