// Host side of the layer operators' C ABI (gdn_linrec_*, gdn_qk_norm_rope*,
// gdn_short_conv_*): argument checks, workspace layouts and launches.  As in
// gdn_api.hip nothing here allocates or synchronises, and a call that returns
// an error has launched nothing.
#include "gdn_layer_host.hpp"

namespace {

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
