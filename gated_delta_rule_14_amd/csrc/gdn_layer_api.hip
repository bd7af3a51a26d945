// Host side of the layer operators' C ABI (gdn_linrec_*, gdn_qk_norm_rope*,
// gdn_short_conv_*): argument checks, workspace layouts and launches.  As in
// gdn_api.hip nothing here allocates or synchronises, and a call that returns
// an error has launched nothing.
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

// ---- gated linear recurrence
constexpr int LINREC_TILE = 128;

gdn_status check_linrec(const gdn_linrec_desc* d, const gdn_activation* act, gdn::Act* out, bool packed) {
    if (!d) return api_fail(GDN_ERR_NULL_ARG, "desc is NULL");
    if (!dtype_ok(d->x_dtype) || !dtype_ok(d->g_dtype))
        return api_fail(GDN_ERR_BAD_DTYPE, "x_dtype %d g_dtype %d", d->x_dtype, d->g_dtype);
    if (d->flags & ~GDN_LINREC_NORMALIZE)
        return api_fail(GDN_ERR_UNSUPPORTED, "flags 0x%x", d->flags);
    gdn_status s = check_rows(d->batch, d->seq_len, d->channels, d->num_seqs, packed);
    if (s != GDN_OK) return s;
    const int64_t st[3] = {d->x_stride, d->g_stride, d->y_stride};
    if ((s = check_strides(st, 3, d->channels)) != GDN_OK) return s;
    *out = gdn::Act{};
    if (act && act->flags) {
        if (act->flags != GDN_ACT_GATE)
            return api_fail(GDN_ERR_UNSUPPORTED, "activation flags 0x%x: only GDN_ACT_GATE applies", act->flags);
        if (!act->A_log || !act->dt_bias)
            return api_fail(GDN_ERR_NULL_ARG, "GDN_ACT_GATE needs A_log and dt_bias");
        if (!aligned(act->A_log, 4) || !aligned(act->dt_bias, 4))
            return api_fail(GDN_ERR_MISALIGNED, "A_log and dt_bias need 4-byte alignment");
        out->flags = act->flags;
        out->A_log = act->A_log;
        out->dt_bias = act->dt_bias;
    }
    return GDN_OK;
}

// Workspace: the words and the tile table, the hand-offs between tiles (where
// some sequence may have two), and for the backward the states entering the
// tiles (where the caller kept none) and the tiles' parameter sums.
struct LinrecLayout {
    TileLayout t;
    int small, shorts;         // as in LinrecLaunch
    bool hand_offs;
    size_t pairs, groups, states, part, sums, total;
};
LinrecLayout linrec_layout(const gdn_linrec_desc* d, bool backward) {
    LinrecLayout L;
    const int64_t D = d->channels;
    // Sequences of up to 16 tokens run by a wave or two instead of a tile's workgroup of 8 or
    // 16, of up to 64 by half of it (256 sequences of 4 tokens, 4096 channels: forward 124 ->
    // 10 us, backward 339 -> 29). Of packed input only the mean length is known here: short
    // ones are looked for where it is below half a tile (2500 sequences of 3 tokens: 1267 ->
    // 88 and 3507 -> 222 us; lengths that differ much are not measured).
    const bool packed = d->num_seqs > 0;
    const int64_t T = d->seq_len, mean = packed ? T / d->num_seqs : T;
    const int few = mean > 64 - packed ? 0 : mean > 16 - packed ? 64 : 16;
    L.small = packed ? 0 : few;
    L.shorts = packed ? few : 0;
    L.t = tile_layout(d->batch, T, d->num_seqs, LINREC_TILE, L.shorts);
    L.hand_offs = packed || L.t.nt > 1;
    const int64_t rows = L.t.tiles + (L.shorts ? d->num_seqs : 0);
    size_t off = L.hand_offs || backward ? L.t.end : 0;
    L.pairs = off;
    if (L.hand_offs) off += align256((size_t)L.t.tiles * D * 8);
    L.groups = off;
    if (L.hand_offs) off += align256((size_t)(L.t.tiles / 16 + 1) * D * 8);
    L.states = off;
    if (backward) off += align256((size_t)L.t.tiles * D * 4);
    L.part = off;
    if (backward) off += align256((size_t)rows * 2 * D * 4);
    L.sums = off;
    if (backward) off += sums_bytes(rows, 2 * D);
    L.total = off;
    return L;
}

// the grids of the tiles, the hand-offs' clearing, the empty sequences and the parameter sums
gdn_status check_linrec_grid(const gdn_linrec_desc* d, const LinrecLayout& L) {
    const double D = (double)d->channels, N = (double)(d->num_seqs > 0 ? d->num_seqs : d->batch);
    const double threads = L.small == 16 ? 128 : L.small == 64 ? 512 : 1024;
    gdn_status s = check_grid((double)L.t.tiles * ((D + 63) / 64), threads);
    if (s == GDN_OK && L.shorts) s = check_grid(N * ((D + 63) / 64), 512);
    if (s == GDN_OK) s = check_grid((N + (double)L.t.tiles) * ((D + 511) / 512), 256);
    return s != GDN_OK ? s : check_grid(2 * ((D + 15) / 16), 1024);
}

void linrec_place(gdn::LinrecLaunch* a, const gdn_linrec_desc* d, const LinrecLayout& L, void* workspace) {
    char* ws = static_cast<char*>(workspace);
    a->map = seq_map(L.t, d->batch, d->seq_len, d->num_seqs, LINREC_TILE, workspace);
    a->words = reinterpret_cast<int*>(ws);
    a->small = L.small;
    a->shorts = L.shorts;
    if (L.hand_offs) {
        a->pairs = reinterpret_cast<uint64_t*>(ws + L.pairs);
        a->groups = reinterpret_cast<uint64_t*>(ws + L.groups);
    }
}

gdn::LinrecLaunch linrec_launch(const gdn_linrec_desc* d, const gdn::Act& act, const void* x, const void* g,
                                void* stream) {
    gdn::LinrecLaunch a;
    a.act = act;
    a.normalize = d->flags & GDN_LINREC_NORMALIZE;
    a.x = x;
    a.g = g;
    a.D = d->channels;
    a.xs = d->x_stride ? d->x_stride : a.D;
    a.gs = d->g_stride ? d->g_stride : a.D;
    a.ys = d->y_stride ? d->y_stride : a.D;
    a.x_bf16 = d->x_dtype == GDN_DTYPE_BF16;
    a.g_bf16 = d->g_dtype == GDN_DTYPE_BF16;
    a.stream = static_cast<hipStream_t>(stream);
    return a;
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

// ---- short convolution
constexpr int CONV_TILE = 64;

gdn_status check_conv(const gdn_conv_desc* d, bool packed) {
    if (!d) return api_fail(GDN_ERR_NULL_ARG, "desc is NULL");
    if (!dtype_ok(d->dtype)) return api_fail(GDN_ERR_BAD_DTYPE, "dtype %d", d->dtype);
    if (d->width < 2 || d->width > 4 || (d->flags & ~GDN_CONV_SILU))
        return api_fail(GDN_ERR_UNSUPPORTED, "width %d (2..4), flags 0x%x", d->width, d->flags);
    gdn_status s = check_rows(d->batch, d->seq_len, d->channels, d->num_seqs, packed);
    if (s != GDN_OK) return s;
    const int64_t st[2] = {d->x_stride, d->y_stride};
    return check_strides(st, 2, d->channels);
}

struct ConvLayout {
    TileLayout t;
    size_t part, sums, total;
};
ConvLayout conv_layout(const gdn_conv_desc* d, bool backward) {
    ConvLayout L;
    L.t = tile_layout(d->batch, d->seq_len, d->num_seqs, CONV_TILE);
    // without packed offsets the forward needs no workspace
    size_t off = d->num_seqs > 0 || backward ? L.t.end : 0;
    L.part = off;
    if (backward) off += align256((size_t)((L.t.tiles + 3) / 4) * (d->width + 1) * d->channels * 4);
    L.sums = off;
    if (backward) off += sums_bytes((L.t.tiles + 3) / 4, (d->width + 1) * d->channels);
    L.total = off;
    return L;
}

gdn::ConvLaunch conv_launch(const gdn_conv_desc* d, const void* x, const float* w, const float* b, const void* s0,
                            void* stream) {
    gdn::ConvLaunch a;
    a.x = x;
    a.w = w;
    a.b = b;
    a.s0 = s0;
    a.D = d->channels;
    a.xs = d->x_stride ? d->x_stride : a.D;
    a.ys = d->y_stride ? d->y_stride : a.D;
    a.W = d->width;
    a.silu = d->flags & GDN_CONV_SILU;
    a.bf16 = d->dtype == GDN_DTYPE_BF16;
    a.stream = static_cast<hipStream_t>(stream);
    return a;
}

// the grids of the tiles with the empty sequences, and of the parameter sums
gdn_status check_conv_grid(const gdn::ConvLaunch& a) {
    const double nb = (double)((a.D + 63) / 64);
    const gdn_status s = check_grid(((double)a.map.max_tiles + (double)a.map.N + 8) * nb, 64);
    return s != GDN_OK ? s : check_grid((a.W + 1) * nb, 1024);
}

}  // namespace

extern "C" {

gdn_status gdn_linrec_workspace(const gdn_linrec_desc* d, int32_t backward, size_t* bytes, int64_t* state_rows) {
    gdn::Act act;
    gdn_status s = check_linrec(d, nullptr, &act, d && d->num_seqs > 0);
    if (s != GDN_OK) return s;
    const LinrecLayout L = linrec_layout(d, backward != 0);
    if (bytes) *bytes = L.total;
    if (state_rows) *state_rows = L.t.tiles;
    return api_ok();
}

gdn_status gdn_linrec_fwd(const gdn_linrec_desc* d, const gdn_activation* act_in, const void* x, const void* g,
                          const float* h0, const int64_t* cu_seqlens, void* y, float* ht, float* states,
                          void* workspace, size_t workspace_bytes, void* stream) {
    gdn::Act act;
    gdn_status s = check_linrec(d, act_in, &act, cu_seqlens != nullptr);
    if (s != GDN_OK) return s;
    const bool any = d->batch * d->seq_len > 0;   // without tokens there is nothing to point to
    if (any && (!x || !g)) return api_fail(GDN_ERR_NULL_ARG, "x and g are required");
    const size_t ex = size_of(d->x_dtype), eg = size_of(d->g_dtype);
    if (!aligned(x, ex) || !aligned(y, ex) || !aligned(g, eg) || !aligned(h0, 4) || !aligned(ht, 4) ||
        !aligned(states, 4) || !aligned(cu_seqlens, 8))
        return api_fail(GDN_ERR_MISALIGNED, "tensors need their element size, cu_seqlens 8 bytes");
    const LinrecLayout L = linrec_layout(d, false);
    if ((s = check_workspace(workspace, workspace_bytes, L.total)) != GDN_OK) return s;
    if ((s = check_linrec_grid(d, L)) != GDN_OK) return s;
    gdn::LinrecLaunch a = linrec_launch(d, act, x, g, stream);
    linrec_place(&a, d, L, workspace);
    a.h0 = h0;
    a.y = y;
    a.ht = ht;
    a.states = states;
    if (cu_seqlens && (s = make_table(a.map, cu_seqlens, workspace, a.stream, L.shorts)) != GDN_OK) return s;
    hipError_t e = gdn::launch_linrec_fwd(a);
    return e == hipSuccess ? api_ok() : hip_fail(e, "linear recurrence launch");
}

gdn_status gdn_linrec_bwd(const gdn_linrec_desc* d, const gdn_activation* act_in, const void* x, const void* g,
                          const float* h0, const int64_t* cu_seqlens, const void* dy, const float* dht,
                          const float* states, void* dx, void* dg, float* dh0, float* dA_log, float* ddt_bias,
                          void* workspace, size_t workspace_bytes, void* stream) {
    gdn::Act act;
    gdn_status s = check_linrec(d, act_in, &act, cu_seqlens != nullptr);
    if (s != GDN_OK) return s;
    const bool any = d->batch * d->seq_len > 0;   // without tokens there is nothing to point to
    if (any && (!x || !g || !dy || !dx || !dg)) return api_fail(GDN_ERR_NULL_ARG, "x, g, dy, dx and dg are required");
    if ((act.flags & GDN_ACT_GATE) && (!dA_log || !ddt_bias))
        return api_fail(GDN_ERR_NULL_ARG, "GDN_ACT_GATE needs the dA_log and ddt_bias outputs");
    const size_t ex = size_of(d->x_dtype), eg = size_of(d->g_dtype);
    if (!aligned(x, ex) || !aligned(dy, ex) || !aligned(dx, ex) || !aligned(g, eg) || !aligned(dg, eg) ||
        !aligned(h0, 4) || !aligned(dht, 4) || !aligned(dh0, 4) || !aligned(states, 4) || !aligned(dA_log, 4) ||
        !aligned(ddt_bias, 4) || !aligned(cu_seqlens, 8))
        return api_fail(GDN_ERR_MISALIGNED, "tensors need their element size, cu_seqlens 8 bytes");
    const LinrecLayout L = linrec_layout(d, true);
    if ((s = check_workspace(workspace, workspace_bytes, L.total)) != GDN_OK) return s;
    if ((s = check_linrec_grid(d, L)) != GDN_OK) return s;
    gdn::LinrecLaunch a = linrec_launch(d, act, x, g, stream);
    char* ws = static_cast<char*>(workspace);
    linrec_place(&a, d, L, workspace);
    a.h0 = h0;
    a.dy = dy;
    a.dht = dht;
    a.dx = dx;
    a.dg = dg;
    a.dh0 = dh0;
    a.dA_log = dA_log;
    a.ddt_bias = ddt_bias;
    a.own_states = !states;
    a.states = states ? const_cast<float*>(states) : reinterpret_cast<float*>(ws + L.states);
    a.part = reinterpret_cast<float*>(ws + L.part);
    a.sums = reinterpret_cast<double*>(ws + L.sums);
    if (cu_seqlens && (s = make_table(a.map, cu_seqlens, workspace, a.stream, L.shorts)) != GDN_OK) return s;
    hipError_t e = gdn::launch_linrec_bwd(a);
    return e == hipSuccess ? api_ok() : hip_fail(e, "linear recurrence backward launch");
}

gdn_status gdn_linrec_step(const gdn_linrec_desc* d, const gdn_activation* act_in, const void* x, const void* g,
                           float* state, void* y, void* stream) {
    gdn::Act act;
    gdn_linrec_desc one;
    const bool none = d && d->batch == 0;   // no sequences: the sizes are still checked
    if (none) {
        one = *d;
        one.batch = 1;
        d = &one;
    }
    gdn_status s = check_linrec(d, act_in, &act, false);
    if (s != GDN_OK) return s;
    if (d->seq_len != 1) return api_fail(GDN_ERR_BAD_SHAPE, "a step takes seq_len 1");
    if (none) return api_ok();
    if (!x || !g || !state || !y) return api_fail(GDN_ERR_NULL_ARG, "x, g, state and y are required");
    const size_t ex = size_of(d->x_dtype), eg = size_of(d->g_dtype);
    if (!aligned(x, ex) || !aligned(y, ex) || !aligned(g, eg) || !aligned(state, 4))
        return api_fail(GDN_ERR_MISALIGNED, "tensors need their element size");
    if ((s = check_grid((double)d->batch * (double)((d->channels + 63) / 64), 64)) != GDN_OK) return s;
    gdn::LinrecLaunch a = linrec_launch(d, act, x, g, stream);
    a.map.N = d->batch;
    a.map.T = 1;
    a.h0 = state;
    a.ht = state;
    a.y = y;
    hipError_t e = gdn::launch_linrec_step(a);
    return e == hipSuccess ? api_ok() : hip_fail(e, "linear recurrence step launch");
}

gdn_status gdn_qk_norm_rope(const gdn_qk_desc* d, const void* q, const void* k, const float* q_weight,
                            const float* k_weight, const double* inv_freq, const int64_t* positions, void* q_out,
                            void* k_out, void* stream) {
    gdn_status s = check_qk(d);
    if (s != GDN_OK) return s;
    if (d->batch * d->seq_len == 0) return api_ok();
    const void* p[4] = {q, k, q_out, k_out};
    if ((s = check_qk_args(d, p, 4, q_weight, k_weight, inv_freq, positions)) != GDN_OK) return s;
    hipError_t e = gdn::launch_qk(qk_launch(d, q, k, q_weight, k_weight, inv_freq, positions, q_out, k_out, stream));
    return e == hipSuccess ? api_ok() : hip_fail(e, "q/k norm launch");
}

gdn_status gdn_qk_norm_rope_bwd_workspace(const gdn_qk_desc* d, size_t* bytes) {
    if (!bytes) return api_fail(GDN_ERR_NULL_ARG, "bytes is NULL");
    gdn_status s = check_qk(d);
    if (s != GDN_OK) return s;
    const int64_t blocks = gdn::qk_bwd_blocks(d->batch * d->seq_len);
    *bytes = align256((size_t)blocks * 2 * d->head_dim * 4) + sums_bytes(blocks, 2 * d->head_dim);
    return api_ok();
}

gdn_status gdn_qk_norm_rope_bwd(const gdn_qk_desc* d, const void* q, const void* k, const float* q_weight,
                                const float* k_weight, const double* inv_freq, const int64_t* positions,
                                const void* dq_out, const void* dk_out, void* dq, void* dk, float* dq_weight,
                                float* dk_weight, void* workspace, size_t workspace_bytes, void* stream) {
    size_t need = 0;
    gdn_status s = gdn_qk_norm_rope_bwd_workspace(d, &need);
    if (s != GDN_OK) return s;
    if ((dq_weight && !q_weight) || (dk_weight && !k_weight))
        return api_fail(GDN_ERR_NULL_ARG, "the gradient of a weight needs the weight");
    if (!aligned(dq_weight, 4) || !aligned(dk_weight, 4))
        return api_fail(GDN_ERR_MISALIGNED, "weight gradients need 4-byte alignment");
    const bool none = d->batch * d->seq_len == 0;
    const void* p[6] = {q, k, dq_out, dk_out, dq, dk};
    if (!none && (s = check_qk_args(d, p, 6, q_weight, k_weight, inv_freq, positions)) != GDN_OK) return s;
    if ((dq_weight || dk_weight) && (s = check_workspace(workspace, workspace_bytes, need)) != GDN_OK) return s;
    gdn::QkLaunch a = qk_launch(d, q, k, q_weight, k_weight, inv_freq, positions, dq, dk, stream);
    a.dqo = dq_out;
    a.dko = dk_out;
    a.dqw = dq_weight;
    a.dkw = dk_weight;
    a.part = static_cast<float*>(workspace);
    a.sums = reinterpret_cast<double*>(static_cast<char*>(workspace) +
                                       align256((size_t)gdn::qk_bwd_blocks(a.tokens) * 2 * a.D * 4));
    hipError_t e = gdn::launch_qk_bwd(a);
    return e == hipSuccess ? api_ok() : hip_fail(e, "q/k norm backward launch");
}

gdn_status gdn_short_conv_workspace(const gdn_conv_desc* d, int32_t backward, size_t* bytes) {
    if (!bytes) return api_fail(GDN_ERR_NULL_ARG, "bytes is NULL");
    gdn_status s = check_conv(d, d && d->num_seqs > 0);
    if (s != GDN_OK) return s;
    *bytes = conv_layout(d, backward != 0).total;
    return api_ok();
}

gdn_status gdn_short_conv_fwd(const gdn_conv_desc* d, const void* x, const float* weight, const float* bias,
                              const void* s0, const int64_t* cu_seqlens, void* y, void* st, void* workspace,
                              size_t workspace_bytes, void* stream) {
    gdn_status s = check_conv(d, cu_seqlens != nullptr);
    if (s != GDN_OK) return s;
    const bool any = d->batch * d->seq_len > 0;   // without tokens there is nothing to point to
    if (!weight || (any && (!x || !y))) return api_fail(GDN_ERR_NULL_ARG, "x, weight and y are required");
    if (st && s0 && st == s0) return api_fail(GDN_ERR_UNSUPPORTED, "st must not overlap s0");
    const size_t e = size_of(d->dtype);
    if (!aligned(x, e) || !aligned(y, e) || !aligned(s0, e) || !aligned(st, e) || !aligned(weight, 4) ||
        !aligned(bias, 4) || !aligned(cu_seqlens, 8))
        return api_fail(GDN_ERR_MISALIGNED, "tensors need their element size, cu_seqlens 8 bytes");
    const ConvLayout L = conv_layout(d, false);
    if ((s = check_workspace(workspace, workspace_bytes, L.total)) != GDN_OK) return s;
    gdn::ConvLaunch a = conv_launch(d, x, weight, bias, s0, stream);
    a.map = seq_map(L.t, d->batch, d->seq_len, d->num_seqs, CONV_TILE, workspace);
    if ((s = check_conv_grid(a)) != GDN_OK) return s;
    a.y = y;
    a.st = st;
    if (cu_seqlens && (s = make_table(a.map, cu_seqlens, workspace, a.stream)) != GDN_OK) return s;
    hipError_t err = gdn::launch_conv_fwd(a);
    return err == hipSuccess ? api_ok() : hip_fail(err, "short convolution launch");
}

gdn_status gdn_short_conv_bwd(const gdn_conv_desc* d, const void* x, const float* weight, const float* bias,
                              const void* s0, const int64_t* cu_seqlens, const void* dy, const void* dst, void* dx,
                              float* dweight, float* dbias, void* ds0, void* workspace, size_t workspace_bytes,
                              void* stream) {
    gdn_status s = check_conv(d, cu_seqlens != nullptr);
    if (s != GDN_OK) return s;
    const bool any = d->batch * d->seq_len > 0;   // without tokens there is nothing to point to
    if (!weight || !dweight || (any && (!x || !dy || !dx)))
        return api_fail(GDN_ERR_NULL_ARG, "x, weight, dy, dx and dweight are required");
    if ((bias != nullptr) != (dbias != nullptr))
        return api_fail(GDN_ERR_NULL_ARG, "dbias is required with bias and must be NULL without");
    const size_t e = size_of(d->dtype);
    if (!aligned(x, e) || !aligned(dy, e) || !aligned(dx, e) || !aligned(s0, e) || !aligned(dst, e) ||
        !aligned(ds0, e) || !aligned(weight, 4) || !aligned(bias, 4) || !aligned(dweight, 4) || !aligned(dbias, 4) ||
        !aligned(cu_seqlens, 8))
        return api_fail(GDN_ERR_MISALIGNED, "tensors need their element size, cu_seqlens 8 bytes");
    const ConvLayout L = conv_layout(d, true);
    if ((s = check_workspace(workspace, workspace_bytes, L.total)) != GDN_OK) return s;
    gdn::ConvLaunch a = conv_launch(d, x, weight, bias, s0, stream);
    a.map = seq_map(L.t, d->batch, d->seq_len, d->num_seqs, CONV_TILE, workspace);
    if ((s = check_conv_grid(a)) != GDN_OK) return s;
    a.dy = dy;
    a.dst = dst;
    a.dx = dx;
    a.dw = dweight;
    a.db = dbias;
    a.ds0 = ds0;
    a.part = reinterpret_cast<float*>(static_cast<char*>(workspace) + L.part);
    a.sums = reinterpret_cast<double*>(static_cast<char*>(workspace) + L.sums);
    if (cu_seqlens && (s = make_table(a.map, cu_seqlens, workspace, a.stream)) != GDN_OK) return s;
    hipError_t err = gdn::launch_conv_bwd(a);
    return err == hipSuccess ? api_ok() : hip_fail(err, "short convolution backward launch");
}

gdn_status gdn_short_conv_step(const gdn_conv_desc* d, const void* x, const float* weight, const float* bias,
                               void* state, void* y, void* stream) {
    gdn_conv_desc one;
    const bool none = d && d->batch == 0;   // no sequences: the sizes are still checked
    if (none) {
        one = *d;
        one.batch = 1;
        d = &one;
    }
    gdn_status s = check_conv(d, false);
    if (s != GDN_OK) return s;
    if (d->seq_len != 1) return api_fail(GDN_ERR_BAD_SHAPE, "a step takes seq_len 1");
    if (none) return api_ok();
    if (!x || !weight || !state || !y) return api_fail(GDN_ERR_NULL_ARG, "x, weight, state and y are required");
    const size_t e = size_of(d->dtype);
    if (!aligned(x, e) || !aligned(y, e) || !aligned(state, e) || !aligned(weight, 4) || !aligned(bias, 4))
        return api_fail(GDN_ERR_MISALIGNED, "tensors need their element size");
    if ((s = check_grid((double)d->batch * (double)((d->channels + 63) / 64), 64)) != GDN_OK) return s;
    gdn::ConvLaunch a = conv_launch(d, x, weight, bias, nullptr, stream);
    a.map.N = d->batch;
    a.st = state;
    a.y = y;
    hipError_t err = gdn::launch_conv_step(a);
    return err == hipSuccess ? api_ok() : hip_fail(err, "short convolution step launch");
}

}  // extern "C"
