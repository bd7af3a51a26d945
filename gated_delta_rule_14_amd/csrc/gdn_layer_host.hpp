// Host helpers that the C ABI files of the layer operators and of the token mixers
// share: checks of sizes and workspaces, the tile table of packed input, and the
// arguments of the q/k norm with rotation.
#pragma once

#include <algorithm>

#include "gdn_layer.hpp"

namespace {

using gdn::api_fail;
using gdn::api_ok;

size_t align256(size_t x) { return (x + 255) & ~(size_t)255; }
bool aligned(const void* p, size_t n) { return ((uintptr_t)p & (n - 1)) == 0; }
// shares of the sums over `rows` partial rows of `cols`
size_t sums_bytes(int64_t rows, int64_t cols) {
    const int64_t n = gdn::row_sum_shares(rows, cols);
    return n > 1 ? align256((size_t)(n * cols) * 8) : 0;
}
bool dtype_ok(int32_t t) { return t == GDN_DTYPE_F32 || t == GDN_DTYPE_BF16; }
size_t size_of(int32_t t) { return t == GDN_DTYPE_BF16 ? 2 : 4; }
gdn_status hip_fail(hipError_t e, const char* what) {
    return api_fail(GDN_ERR_HIP, "%s: %s", what, hipGetErrorString(e));
}

// sizes of a call over tokens and channels
gdn_status check_rows(int64_t B, int64_t T, int64_t D, int64_t N, bool packed) {
    if (B <= 0 || T < 0 || D <= 0 || N < 0)
        return api_fail(GDN_ERR_BAD_SHAPE, "batch, channels > 0 and seq_len, num_seqs >= 0 (B=%lld T=%lld D=%lld N=%lld)",
                        (long long)B, (long long)T, (long long)D, (long long)N);
    if (packed && (B != 1 || N <= 0))
        return api_fail(GDN_ERR_BAD_SHAPE, "packed sequences need batch == 1 and num_seqs > 0");
    if (!packed && N != 0) return api_fail(GDN_ERR_BAD_SHAPE, "num_seqs must be 0 without cu_seqlens");
    const int64_t lim = (int64_t)1 << 31;   // channels: byte offsets in a row are 32-bit
    if (B >= lim || T >= lim || D >= (lim >> 3) || N >= lim || B * T >= lim)
        return api_fail(GDN_ERR_BAD_SHAPE, "B*T and num_seqs must be below 2^31, channels below 2^28");
    return GDN_OK;
}

gdn_status check_strides(const int64_t* s, int n, int64_t D) {
    for (int i = 0; i < n; ++i)
        if (s[i] != 0 && s[i] < D)
            return api_fail(GDN_ERR_BAD_SHAPE, "token stride %lld below %lld channels", (long long)s[i], (long long)D);
    return GDN_OK;
}

// a launch of `blocks` workgroups of `threads`: the grid's 32-bit limits
gdn_status check_grid(double blocks, double threads) {
    if (blocks >= 2147483648.0 || blocks * threads >= 4294967296.0)
        return api_fail(GDN_ERR_BAD_SHAPE, "tokens x channels too large for one launch");
    return GDN_OK;
}

// ---- tiles: the words, the records of packed input and the tile table
struct TileLayout {
    size_t seqs, table, end;
    int64_t tiles, nt;
};
// (sequences of up to `shorts` tokens have no tiles)
TileLayout tile_layout(int64_t B, int64_t T, int64_t N, int tile, int shorts = 0) {
    TileLayout L;
    L.nt = (T + tile - 1) / tile;
    L.tiles = N > 0 ? L.nt + std::min(N, T / (shorts + 1)) : B * L.nt;
    L.seqs = 256;
    L.table = L.seqs + align256(N > 0 ? (size_t)N * 16 : 0);
    L.end = L.table + align256(N > 0 ? (size_t)L.tiles * sizeof(gdn::TileRow) : 0);
    return L;
}

gdn::SeqMap seq_map(const TileLayout& L, int64_t B, int64_t T, int64_t N, int tile, void* ws) {
    gdn::SeqMap m;
    char* p = static_cast<char*>(ws);
    m.T = T;
    m.nt = L.nt;
    m.N = N > 0 ? N : B;
    m.max_tiles = L.tiles;
    m.tile = tile;
    if (N > 0) {
        m.seqs = reinterpret_cast<const int4*>(p + L.seqs);
        m.table = reinterpret_cast<const gdn::TileRow*>(p + L.table);
    }
    return m;
}

gdn_status make_table(const gdn::SeqMap& m, const int64_t* cu, void* ws, hipStream_t st, int shorts = 0) {
    gdn::TileTableLaunch t;
    t.cu_seqlens = cu;
    t.N = m.N;
    t.T = m.T;
    t.max_tiles = m.max_tiles;
    t.tile = m.tile;
    t.shorts = shorts;
    t.table = const_cast<gdn::TileRow*>(m.table);
    t.seqs = const_cast<int4*>(m.seqs);
    t.words = static_cast<int*>(ws);
    t.stream = st;
    hipError_t e = gdn::launch_tile_table(t);
    return e == hipSuccess ? GDN_OK : hip_fail(e, "tile table launch");
}

gdn_status check_workspace(const void* ws, size_t have, size_t need) {
    if (need == 0) return GDN_OK;
    if (!ws) return api_fail(GDN_ERR_NULL_ARG, "workspace is required (%zu bytes)", need);
    if (!aligned(ws, 256)) return api_fail(GDN_ERR_MISALIGNED, "workspace must be 256-byte aligned");
    if (have < need)
        return api_fail(GDN_ERR_WORKSPACE_TOO_SMALL, "workspace %zu bytes, need %zu", have, need);
    return GDN_OK;
}

// ---- q/k norm and rotation
gdn_status check_qk(const gdn_qk_desc* d) {
    if (!d) return api_fail(GDN_ERR_NULL_ARG, "desc is NULL");
    if (!dtype_ok(d->dtype)) return api_fail(GDN_ERR_BAD_DTYPE, "dtype %d", d->dtype);
    if (d->norm < GDN_NORM_NONE || d->norm > GDN_NORM_RMS || (d->flags & ~GDN_QK_INTERLEAVED))
        return api_fail(GDN_ERR_UNSUPPORTED, "norm %d flags 0x%x", d->norm, d->flags);
    if (d->batch < 0 || d->seq_len < 0 || d->q_heads <= 0 || d->k_heads <= 0)
        return api_fail(GDN_ERR_BAD_SHAPE, "B=%lld T=%lld Hq=%lld Hk=%lld", (long long)d->batch,
                        (long long)d->seq_len, (long long)d->q_heads, (long long)d->k_heads);
    const int64_t lim = (int64_t)1 << 31;
    if (d->batch >= lim || d->seq_len >= lim || d->batch * d->seq_len >= lim || d->q_heads > 65535 ||
        d->k_heads > 65535)
        return api_fail(GDN_ERR_BAD_SHAPE, "B*T must be below 2^31, heads at most 65535");
    if (d->head_dim <= 0 || d->head_dim > 256 || d->head_dim % 8)
        return api_fail(GDN_ERR_UNSUPPORTED, "head_dim %lld (a multiple of 8 up to 256)", (long long)d->head_dim);
    if (d->rot_dim < 0 || d->rot_dim > d->head_dim || d->rot_dim % 16)
        return api_fail(GDN_ERR_UNSUPPORTED, "rot_dim %lld (a multiple of 16 up to head_dim)", (long long)d->rot_dim);
    const int64_t hs[2] = {d->q_head_stride, d->k_head_stride}, ts[2] = {d->q_stride, d->k_stride};
    const int64_t H[2] = {d->q_heads, d->k_heads};
    for (int i = 0; i < 2; ++i) {
        const int64_t h = hs[i] ? hs[i] : d->head_dim;
        if (h < d->head_dim || (ts[i] && ts[i] < (H[i] - 1) * h + d->head_dim))
            return api_fail(GDN_ERR_BAD_SHAPE, "head stride %lld, token stride %lld: rows overlap",
                            (long long)hs[i], (long long)ts[i]);
        if (h % 8 || ts[i] % 8)
            return api_fail(GDN_ERR_MISALIGNED, "strides must be multiples of 8 elements");
    }
    return check_grid(((double)(d->batch * d->seq_len) + 4096) / 4, 256);
}

gdn::QkLaunch qk_launch(const gdn_qk_desc* d, const void* q, const void* k, const float* qw, const float* kw,
                        const double* inv_freq, const int64_t* positions, void* qo, void* ko, void* stream) {
    gdn::QkLaunch a;
    a.q = q;
    a.k = k;
    a.qw = qw;
    a.kw = kw;
    a.inv_freq = inv_freq;
    a.positions = positions;
    a.qo = qo;
    a.ko = ko;
    a.tokens = d->batch * d->seq_len;
    a.T = d->seq_len;
    a.Hq = d->q_heads;
    a.Hk = d->k_heads;
    a.D = (int)d->head_dim;
    a.R = (int)d->rot_dim;
    a.qhs = d->q_head_stride ? d->q_head_stride : a.D;
    a.khs = d->k_head_stride ? d->k_head_stride : a.D;
    a.qs = d->q_stride ? d->q_stride : a.Hq * a.qhs;
    a.ks = d->k_stride ? d->k_stride : a.Hk * a.khs;
    a.norm = d->norm;
    a.interleaved = d->flags & GDN_QK_INTERLEAVED;
    a.bf16 = d->dtype == GDN_DTYPE_BF16;
    a.eps = d->eps;
    a.offset = d->weight_offset;
    a.stream = static_cast<hipStream_t>(stream);
    return a;
}

gdn_status check_qk_args(const gdn_qk_desc* d, const void* const* p16, int n, const float* qw, const float* kw,
                         const double* inv_freq, const int64_t* positions) {
    for (int i = 0; i < n; ++i) {
        if (!p16[i]) return api_fail(GDN_ERR_NULL_ARG, "q, k and their outputs (and gradients) are required");
        if (!aligned(p16[i], 16)) return api_fail(GDN_ERR_MISALIGNED, "q, k and their outputs need 16-byte alignment");
    }
    if (d->rot_dim > 0 && !inv_freq) return api_fail(GDN_ERR_NULL_ARG, "inv_freq is required with rot_dim > 0");
    if (!aligned(qw, 4) || !aligned(kw, 4) || !aligned(inv_freq, 8) || !aligned(positions, 8))
        return api_fail(GDN_ERR_MISALIGNED, "weights need 4-byte, inv_freq and positions 8-byte alignment");
    return GDN_OK;
}

}  // namespace
