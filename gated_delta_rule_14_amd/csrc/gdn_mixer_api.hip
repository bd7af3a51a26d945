// Host side of the C ABI of the token mixers next to the delta rule
// (gdn_decay_attn_*, gdn_paged_*): argument checks, workspace layouts and
// launches.  As in gdn_api.hip nothing here allocates or synchronises, and a call
// that returns an error has launched nothing.
#include <utility>

#include "gdn_layer_host.hpp"
#include "gdn_mixer.hpp"

namespace {

int64_t v_heads(const gdn_decay_desc* d) { return d->num_v_heads > 0 ? d->num_v_heads : d->num_heads; }

gdn_status check_decay(const gdn_decay_desc* d, bool packed) {
    if (!d) return api_fail(GDN_ERR_NULL_ARG, "desc is NULL");
    if (!dtype_ok(d->dtype)) return api_fail(GDN_ERR_BAD_DTYPE, "dtype %d", d->dtype);
    if (d->flags & ~GDN_DECAY_PER_HEAD) return api_fail(GDN_ERR_UNSUPPORTED, "flags 0x%x", d->flags);
    if ((d->key_dim != 64 && d->key_dim != 128) || (d->value_dim != 64 && d->value_dim != 128))
        return api_fail(GDN_ERR_UNSUPPORTED, "key_dim %lld value_dim %lld (each 64 or 128)", (long long)d->key_dim,
                        (long long)d->value_dim);
    if (d->num_heads <= 0 || d->num_v_heads < 0 || v_heads(d) > 65535 || v_heads(d) % d->num_heads)
        return api_fail(GDN_ERR_BAD_SHAPE, "H=%lld H_V=%lld (a multiple of H up to 65535)", (long long)d->num_heads,
                        (long long)d->num_v_heads);
    gdn_status s = check_rows(d->batch, d->seq_len, 1, d->num_seqs, packed);
    if (s != GDN_OK) return s;
    const int64_t H[3] = {d->num_heads, d->num_heads, v_heads(d)}, W[3] = {d->key_dim, d->key_dim, d->value_dim};
    const int64_t ts[3] = {d->q_stride, d->k_stride, d->v_stride};
    const int64_t hs[3] = {d->q_head_stride, d->k_head_stride, d->v_head_stride};
    for (int i = 0; i < 3; ++i) {
        const int64_t h = hs[i] ? hs[i] : W[i];
        if (h < W[i] || ts[i] < 0 || (ts[i] && ts[i] < (H[i] - 1) * h + W[i]))
            return api_fail(GDN_ERR_BAD_SHAPE, "head stride %lld, token stride %lld: rows overlap", (long long)hs[i],
                            (long long)ts[i]);
        if (h % 8 || ts[i] % 8) return api_fail(GDN_ERR_MISALIGNED, "strides must be multiples of 8 elements");
        if (ts[i] >= 1 << 24 || H[i] * h >= 1 << 24)   // offsets inside a chunk of 64 rows are 32-bit
            return api_fail(GDN_ERR_BAD_SHAPE, "token stride %lld: below 2^24 elements", (long long)(ts[i] ? ts[i] : H[i] * h));
    }
    return GDN_OK;
}

// Segments that long sequences are cut into, each walked by a workgroup per state
// head: as long as leaves the chip two workgroups to a compute unit (4 x 4096 tokens of
// 16 heads, forward: 118 us, with half as many 120, with 768 143, with 1024 145), at
// most 4096 tokens (a longer walk would end alone; 64 sequences of 100 to 4000 tokens,
// 16 heads of 128: 642 us, with 2048 894, with 8192 637; 65536 and 6 x 10000: 851, 772,
// 852; 65536 and 15 of up to 8192, 32 heads: 1153, 1223, 1218), and at least 128 (3 x 1001
// tokens of 6 heads in fp32, training step: 126 us, with 64 or 256 144), or 64 where the
// gradients' three walks then have a compute unit for each workgroup (4 heads of 128,
// forward and backward: 300 tokens in bf16 16 and 29 us, with 128 19 and 36; in fp32 33 and
// 45, with 128 47 and 66; beyond, 2 x 2048 tokens in bf16 34 and 62, with 128 33 and 52).
int decay_tile(const gdn_decay_desc* d) {
    const double work = (double)d->batch * (double)d->seq_len * (double)v_heads(d);
    const int64_t want = (int64_t)(work / 512.0), least = 3 * work <= 256 * 64 ? 64 : 128;
    return (int)std::min((int64_t)4096, std::max(least, (want + 63) / 64 * 64));
}

struct DecayLayout {
    TileLayout t;
    int tile;
    int64_t N, tiles, singles, tokens;   // workgroups (per head) for segments and for whole sequences
    size_t table_end, state, dec, estate, edec, dq, dk, ends, dg, sums, dq32, dk32, total;
};
DecayLayout decay_layout(const gdn_decay_desc* d, bool backward) {
    DecayLayout L;
    const bool packed = d->num_seqs > 0;
    const int64_t H = v_heads(d), KV = d->key_dim * d->value_dim;
    L.tile = decay_tile(d);
    L.N = packed ? d->num_seqs : d->batch;
    L.tokens = d->batch * d->seq_len;
    // sequences of up to a segment's length are walked whole
    L.t = tile_layout(d->batch, d->seq_len, d->num_seqs, L.tile, packed ? L.tile : 0);
    const bool whole = d->seq_len <= L.tile;
    L.tiles = whole ? 0 : L.t.tiles;
    L.singles = whole || packed ? L.N : 0;
    size_t off = packed ? L.t.end : 0;
    const auto take = [&](size_t n) {
        const size_t at = off;
        off += align256(n);
        return at;
    };
    L.state = take((size_t)L.tiles * H * KV * 4);
    L.dec = take((size_t)L.tiles * H * 4);
    if (backward) {
        const bool shared = H != d->num_heads, head = d->flags & GDN_DECAY_PER_HEAD;
        L.estate = take((size_t)L.tiles * H * KV * 4);
        L.edec = take((size_t)L.tiles * H * 4);
        L.dq = take((size_t)L.tokens * H * 4);
        L.dk = take((size_t)L.tokens * H * 4);
        L.ends = take((size_t)(L.tiles + L.singles) * H * 4);
        L.dg = take(head ? (size_t)(L.tiles + L.singles) * H * 4 : 0);
        L.sums = take(head ? sums_bytes(L.tiles + L.singles, H) : 0);
        L.dq32 = take(shared ? (size_t)L.tokens * H * d->key_dim * 4 : 0);
        L.dk32 = take(shared ? (size_t)L.tokens * H * d->key_dim * 4 : 0);
    }
    L.total = off;
    return L;
}

gdn_status check_decay_grid(const gdn_decay_desc* d, const DecayLayout& L) {
    const double H = (double)v_heads(d), per = (double)(d->key_dim * d->value_dim / 1024);
    gdn_status s = check_grid(3 * ((double)L.tiles + (double)L.singles + 8) * H, 256);
    if (s == GDN_OK) s = check_grid(2 * ((double)L.tiles + 8) * H * per, 256);
    // (the sums of dq and dk over shared heads: four elements to a thread, both in one launch)
    return s != GDN_OK ? s : check_grid((double)L.tokens * (double)(d->num_heads * d->key_dim / 2) / 256, 256);
}

// rows of q, k (H heads) or v, o (H_V heads), as wide as `w`
gdn::HeadRows rows_of(const gdn_decay_desc* d, const void* p, bool value, int64_t ts, int64_t hs) {
    gdn::HeadRows r;
    const int64_t H = value ? v_heads(d) : d->num_heads, w = value ? d->value_dim : d->key_dim;
    r.p = p;
    r.hs = hs ? hs : w;
    r.ts = ts ? ts : H * r.hs;
    r.div = (int)(v_heads(d) / H);
    return r;
}

gdn::SeqMap decay_map(const gdn_decay_desc* d, const DecayLayout& L, void* ws) {
    gdn::SeqMap m = seq_map(L.t, d->batch, d->seq_len, d->num_seqs, L.tile, ws);
    m.max_tiles = d->num_seqs > 0 ? L.t.tiles : L.tiles;
    return m;
}

gdn::DecayWalk walk_of(const gdn_decay_desc* d, const DecayLayout& L, const gdn::SeqMap& m, const float* g,
                       void* stream) {
    gdn::DecayWalk w;
    w.map = m;
    w.tiles = L.tiles;
    w.singles = L.singles;
    w.g = g;
    w.H = v_heads(d);
    w.share = (int)(w.H / d->num_heads);
    w.gs = d->flags & GDN_DECAY_PER_HEAD ? 0 : w.H;
    w.tokens = L.tokens;
    w.stream = static_cast<hipStream_t>(stream);
    return w;
}

gdn_status walk(const gdn::DecayWalk& w, bool local, const gdn_decay_desc* d) {
    const hipError_t e =
        gdn::launch_decay_walk(w, local, (int)d->key_dim, (int)d->value_dim, d->dtype == GDN_DTYPE_BF16);
    return e == hipSuccess ? GDN_OK : hip_fail(e, "decay attention launch");
}

gdn::DecayWalk local_of(gdn::DecayWalk w, const gdn::HeadRows& b, const gdn::HeadRows& c, float up, float* state,
                        float* dec) {
    w.b = b;
    w.c = c;
    w.up_scale = up;
    w.local = state;
    w.dec = dec;
    return w;
}
gdn::DecayJoin join_of(const gdn_decay_desc* d, const gdn::DecayWalk& w, const float* first, bool rev,
                       bool own_order) {
    gdn::DecayJoin j;
    j.V = (int)d->value_dim;
    j.own_order = own_order;
    j.map = w.map;
    j.tiles = w.tiles;
    j.state = w.local;
    j.dec = w.dec;
    j.first = first;
    j.H = w.H;
    j.KV = d->key_dim * d->value_dim;
    j.rev = rev;
    j.chain = w.chain;
    j.stream = w.stream;
    return j;
}

gdn_status check_decay_args(const gdn_decay_desc* d, const void* const* p16, int n, const float* g, const float* h0,
                            const float* h1, const float* h2, const int64_t* cu) {
    const bool any = d->batch * d->seq_len > 0;   // without tokens there is nothing to point to
    if (any && !g) return api_fail(GDN_ERR_NULL_ARG, "g is required");
    for (int i = 0; i < n; ++i) {
        if (any && !p16[i]) return api_fail(GDN_ERR_NULL_ARG, "q, k, v, their gradients and outputs are required");
        if (!aligned(p16[i], 16)) return api_fail(GDN_ERR_MISALIGNED, "q, k, v and their like need 16-byte alignment");
    }
    if (!aligned(g, 4) || !aligned(h0, 16) || !aligned(h1, 16) || !aligned(h2, 16) || !aligned(cu, 8))
        return api_fail(GDN_ERR_MISALIGNED, "states need 16-byte, g 4-byte, cu_seqlens 8-byte alignment");
    return GDN_OK;
}

// ---- pages
gdn_status check_pages(const gdn_pages* c, int64_t heads, int64_t D, const void* kc, const void* vc, const int32_t* table,
                       const int64_t* lens) {
    if (!c) return api_fail(GDN_ERR_NULL_ARG, "pages is NULL");
    const int64_t lim = (int64_t)1 << 31;
    if (c->num_seqs < 0 || c->max_pages <= 0 || c->pages <= 0 || c->page_size <= 0 || c->num_seqs >= lim ||
        c->pages >= lim || c->max_pages >= lim || c->page_size >= lim || c->max_pages * c->page_size >= lim / 2)
        return api_fail(GDN_ERR_BAD_SHAPE, "N=%lld max_pages=%lld pages=%lld page_size=%lld (a table row below 2^30 tokens)",
                        (long long)c->num_seqs, (long long)c->max_pages, (long long)c->pages, (long long)c->page_size);
    const int64_t st[2][3] = {{c->k_page_stride, c->k_token_stride, c->k_head_stride},
                              {c->v_page_stride, c->v_token_stride, c->v_head_stride}};
    for (const auto& s : st) {
        // smallest first: each stride has to clear what lies within it
        std::pair<int64_t, int64_t> dim[3] = {{s[0], c->pages}, {s[1], c->page_size}, {s[2], heads}};
        std::sort(dim, dim + 3);
        double within = (double)D;
        for (const auto& x : dim) {
            if (x.second == 1) continue;
            if ((double)x.first < within)
                return api_fail(GDN_ERR_BAD_SHAPE, "cache strides %lld, %lld, %lld: rows overlap", (long long)s[0],
                                (long long)s[1], (long long)s[2]);
            within += (double)x.first * (double)(x.second - 1);
        }
        if (within >= 9.2e18) return api_fail(GDN_ERR_BAD_SHAPE, "cache too large");
        if (s[0] % 8 || s[1] % 8 || s[2] % 8)
            return api_fail(GDN_ERR_MISALIGNED, "cache strides must be multiples of 8 elements");
    }
    if (c->num_seqs > 0) {
        if (!kc || !vc || !table || !lens)
            return api_fail(GDN_ERR_NULL_ARG, "k_cache, v_cache, page_table and lens are required");
        if (!aligned(kc, 16) || !aligned(vc, 16) || !aligned(table, 4) || !aligned(lens, 8))
            return api_fail(GDN_ERR_MISALIGNED, "caches need 16-byte, page_table 4-byte, lens 8-byte alignment");
    }
    return GDN_OK;
}

gdn::Pages pages_of(void* p, int64_t ps, int64_t ts, int64_t hs) {
    gdn::Pages r;
    r.p = p;
    r.ps = ps;
    r.ts = ts;
    r.hs = hs;
    return r;
}

gdn_status check_attn(const gdn_paged_attn_desc* d) {
    if (!d) return api_fail(GDN_ERR_NULL_ARG, "desc is NULL");
    if (!dtype_ok(d->dtype)) return api_fail(GDN_ERR_BAD_DTYPE, "dtype %d", d->dtype);
    if (d->num_seqs < 0 || d->k_heads <= 0 || d->q_heads <= 0 || d->q_heads > 65535 || d->q_heads % d->k_heads)
        return api_fail(GDN_ERR_BAD_SHAPE, "N=%lld Hq=%lld Hk=%lld (Hq a multiple of Hk up to 65535)",
                        (long long)d->num_seqs, (long long)d->q_heads, (long long)d->k_heads);
    if (d->head_dim <= 0 || d->head_dim > 256 || d->head_dim % 8)
        return api_fail(GDN_ERR_UNSUPPORTED, "head_dim %lld (a multiple of 8 up to 256)", (long long)d->head_dim);
    if (d->window < 0) return api_fail(GDN_ERR_BAD_SHAPE, "window %lld", (long long)d->window);
    const int64_t h = d->q_head_stride ? d->q_head_stride : d->head_dim;
    if (h < d->head_dim || d->q_stride < 0 || (d->q_stride && d->q_stride < (d->q_heads - 1) * h + d->head_dim))
        return api_fail(GDN_ERR_BAD_SHAPE, "q strides %lld, %lld: rows overlap", (long long)d->q_stride,
                        (long long)d->q_head_stride);
    if (h % 8 || d->q_stride % 8) return api_fail(GDN_ERR_MISALIGNED, "strides must be multiples of 8 elements");
    const double N = (double)d->num_seqs;
    const gdn_status s = check_grid((N + 2048) * (double)d->k_heads * (double)((d->q_heads / d->k_heads + 15) / 16), 256);
    return s != GDN_OK ? s : check_grid(N * (double)d->q_heads, 256);
}
size_t attn_rows(const gdn_paged_attn_desc* d) {
    return (size_t)((gdn::paged_attn_share(d->q_heads, d->k_heads) + d->num_seqs) * d->q_heads);
}
size_t attn_bytes(const gdn_paged_attn_desc* d) {
    return d->num_seqs == 0 ? 0 : align256(attn_rows(d) * d->head_dim * 4) + align256(attn_rows(d) * 8);
}

}  // namespace

extern "C" {

gdn_status gdn_decay_attn_workspace(const gdn_decay_desc* d, int32_t backward, size_t* bytes) {
    gdn_status s = check_decay(d, d && d->num_seqs > 0);
    if (s != GDN_OK) return s;
    if (!bytes) return api_fail(GDN_ERR_NULL_ARG, "bytes is NULL");
    *bytes = decay_layout(d, backward != 0).total;
    return api_ok();
}

gdn_status gdn_decay_attn_fwd(const gdn_decay_desc* d, const void* q, const void* k, const void* v, const float* g,
                              const float* h0, const int64_t* cu_seqlens, void* o, float* ht, void* workspace,
                              size_t workspace_bytes, void* stream) {
    gdn_status s = check_decay(d, cu_seqlens != nullptr);
    if (s != GDN_OK) return s;
    const void* p16[4] = {q, k, v, o};
    if ((s = check_decay_args(d, p16, 4, g, h0, ht, nullptr, cu_seqlens)) != GDN_OK) return s;
    const DecayLayout L = decay_layout(d, false);
    if ((s = check_workspace(workspace, workspace_bytes, L.total)) != GDN_OK) return s;
    if ((s = check_decay_grid(d, L)) != GDN_OK) return s;
    const gdn::SeqMap m = decay_map(d, L, workspace);
    gdn::DecayWalk w = walk_of(d, L, m, g, stream);
    if (cu_seqlens && (s = make_table(m, cu_seqlens, workspace, w.stream, L.tile)) != GDN_OK) return s;
    char* ws = static_cast<char*>(workspace);
    const gdn::HeadRows Q = rows_of(d, q, false, d->q_stride, d->q_head_stride);
    const gdn::HeadRows K = rows_of(d, k, false, d->k_stride, d->k_head_stride);
    const gdn::HeadRows V = rows_of(d, v, true, d->v_stride, d->v_head_stride);
    float* state = reinterpret_cast<float*>(ws + L.state);
    if (L.tiles > 0) {
        // Up to eight segments chain their own states (4 x 4096 tokens, eight: 106 us, joined 114; up to
        // 16: 3 x 1001 in fp32, the walk 35 us for 27, the join 9).  Every segment then reads h0, which
        // the last one may not have replaced.
        w.chain = h0 && ht == h0 ? 0 : 8;
        w.dec = reinterpret_cast<float*>(ws + L.dec);
        const gdn::DecayWalk f = local_of(w, K, V, 1.f, state, w.dec);
        if ((s = walk(f, true, d)) != GDN_OK) return s;
        if (d->seq_len > (int64_t)w.chain * L.tile) {
            const hipError_t e = gdn::launch_decay_join(join_of(d, f, h0, false, true));
            if (e != hipSuccess) return hip_fail(e, "decay attention state launch");
        }
    }
    w.a = Q;
    w.b = K;
    w.c = V;
    w.in_scale = w.pair_scale = d->scale;
    w.tile_state = state;
    w.seq_state = h0;
    w.seq_out = ht;
    w.out = o;
    s = walk(w, false, d);
    return s == GDN_OK ? api_ok() : s;
}

gdn_status gdn_decay_attn_bwd(const gdn_decay_desc* d, const void* q, const void* k, const void* v, const float* g,
                              const float* h0, const int64_t* cu_seqlens, const void* dout, const float* dht, void* dq,
                              void* dk, void* dv, float* dg, float* dh0, void* workspace, size_t workspace_bytes,
                              void* stream) {
    gdn_status s = check_decay(d, cu_seqlens != nullptr);
    if (s != GDN_OK) return s;
    const void* p16[7] = {q, k, v, dout, dq, dk, dv};
    if ((s = check_decay_args(d, p16, 7, g, h0, dht, dh0, cu_seqlens)) != GDN_OK) return s;
    const bool head = d->flags & GDN_DECAY_PER_HEAD;
    if (!dg && (head || d->batch * d->seq_len > 0)) return api_fail(GDN_ERR_NULL_ARG, "dg is required");
    if (!aligned(dg, 4)) return api_fail(GDN_ERR_MISALIGNED, "dg needs 4-byte alignment");
    const DecayLayout L = decay_layout(d, true);
    if ((s = check_workspace(workspace, workspace_bytes, L.total)) != GDN_OK) return s;
    if ((s = check_decay_grid(d, L)) != GDN_OK) return s;
    const gdn::SeqMap m = decay_map(d, L, workspace);
    const gdn::DecayWalk w0 = walk_of(d, L, m, g, stream);
    if (cu_seqlens && (s = make_table(m, cu_seqlens, workspace, w0.stream, L.tile)) != GDN_OK) return s;
    char* ws = static_cast<char*>(workspace);
    const auto at = [&](size_t off) { return reinterpret_cast<float*>(ws + off); };
    const gdn::HeadRows Q = rows_of(d, q, false, d->q_stride, d->q_head_stride);
    const gdn::HeadRows K = rows_of(d, k, false, d->k_stride, d->k_head_stride);
    const gdn::HeadRows V = rows_of(d, v, true, d->v_stride, d->v_head_stride);
    const gdn::HeadRows O = rows_of(d, dout, true, 0, 0);
    if (L.tiles > 0) {
        const gdn::DecayWalk f = local_of(w0, V, K, 1.f, at(L.state), at(L.dec));
        const gdn::DecayWalk r = local_of(w0, O, Q, d->scale, at(L.estate), at(L.edec));
        hipError_t e = gdn::launch_decay_local2(f, r, (int)d->key_dim, (int)d->value_dim, d->dtype == GDN_DTYPE_BF16);
        const gdn::DecayJoin jr = join_of(d, r, dht, true, false);
        if (e == hipSuccess) e = gdn::launch_decay_join(join_of(d, f, h0, false, false), &jr);
        if (e != hipSuccess) return hip_fail(e, "decay attention state launch");
    }
    const bool shared = v_heads(d) != d->num_heads;

    gdn::DecayWalk wq = w0;         // dq: forward over (do, v, k)
    wq.a = O;
    wq.b = V;
    wq.c = K;
    wq.x = Q;
    wq.in_scale = wq.pair_scale = d->scale;
    wq.tile_state = at(L.state);
    wq.seq_state = h0;
    wq.tile_end = at(L.estate);
    wq.seq_end = dht;
    wq.ends = at(L.ends);
    wq.dots = at(L.dq);
    wq.out = dq;
    wq.out32 = shared ? at(L.dq32) : nullptr;
    gdn::DecayWalk wk = w0;         // dk: from the end over (v, do, q)
    wk.a = V;
    wk.b = O;
    wk.c = Q;
    wk.x = K;
    wk.pair_scale = wk.up_scale = d->scale;
    wk.tile_state = at(L.estate);
    wk.seq_state = dht;
    wk.dots = at(L.dk);
    wk.out = dk;
    wk.out32 = shared ? at(L.dk32) : nullptr;
    gdn::DecayWalk wv = w0;         // dv: from the end over (k, q, do)
    wv.a = K;
    wv.b = Q;
    wv.c = O;
    wv.pair_scale = wv.up_scale = d->scale;
    wv.tile_state = at(L.estate);
    wv.seq_state = dht;
    wv.seq_out = dh0;
    wv.out = dv;
    hipError_t e = gdn::launch_decay_grad(wq, wk, wv, (int)d->key_dim, (int)d->value_dim, d->dtype == GDN_DTYPE_BF16);
    if (e != hipSuccess) return hip_fail(e, "decay attention gradient launch");

    gdn::DecayGate a;
    a.map = m;
    a.tiles = L.tiles;
    a.singles = L.singles;
    a.dq = at(L.dq);
    a.dk = at(L.dk);
    a.ends = at(L.ends);
    a.g = g;
    a.gs = w0.gs;
    a.dg = dg;
    a.part = head ? at(L.dg) : nullptr;
    a.H = w0.H;
    a.tokens = L.tokens;
    a.stream = w0.stream;
    e = gdn::launch_decay_gate(a);
    if (e == hipSuccess && head) {
        gdn::RowSumLaunch r{at(L.dg), L.tiles + L.singles, w0.H, 1, 1, dg, nullptr, reinterpret_cast<double*>(ws + L.sums),
                            w0.stream};
        e = gdn::launch_row_sum(r);
    }
    if (e == hipSuccess && shared) {
        gdn::GvaSumLaunch r;
        r.rows = L.tokens;
        r.H = w0.H;
        r.Hq = d->num_heads;
        r.K = (int)d->key_dim;
        r.bf16 = d->dtype == GDN_DTYPE_BF16;
        r.stream = w0.stream;
        r.part = at(L.dq32);
        r.out = dq;
        r.part2 = at(L.dk32);
        r.out2 = dk;
        e = gdn::launch_gva_sum(r);
    }
    return e == hipSuccess ? api_ok() : hip_fail(e, "decay attention gradient launch");
}

gdn_status gdn_decay_attn_step(const gdn_decay_desc* d, const void* q, const void* k, const void* v, const float* g,
                               float* state, void* o, void* stream) {
    gdn_decay_desc one;
    const bool none = d && d->batch == 0;   // no sequences: the sizes are still checked
    if (none) {
        one = *d;
        one.batch = 1;
        d = &one;
    }
    gdn_status s = check_decay(d, false);
    if (s != GDN_OK) return s;
    if (d->seq_len != 1) return api_fail(GDN_ERR_BAD_SHAPE, "a step takes seq_len 1");
    if (none) return api_ok();
    const void* p16[4] = {q, k, v, o};
    if ((s = check_decay_args(d, p16, 4, g, state, nullptr, nullptr, nullptr)) != GDN_OK) return s;
    if (!state) return api_fail(GDN_ERR_NULL_ARG, "state is required");
    if ((s = check_grid((double)d->batch * (double)v_heads(d), 256)) != GDN_OK) return s;
    gdn::DecayStep a;
    a.q = rows_of(d, q, false, d->q_stride, d->q_head_stride);
    a.k = rows_of(d, k, false, d->k_stride, d->k_head_stride);
    a.v = rows_of(d, v, true, d->v_stride, d->v_head_stride);
    a.g = g;
    a.H = v_heads(d);
    a.gs = d->flags & GDN_DECAY_PER_HEAD ? 0 : a.H;
    a.state = state;
    a.o = o;
    a.scale = d->scale;
    a.N = d->batch;
    a.K = (int)d->key_dim;
    a.V = (int)d->value_dim;
    a.bf16 = d->dtype == GDN_DTYPE_BF16;
    a.stream = static_cast<hipStream_t>(stream);
    const hipError_t e = gdn::launch_decay_step(a);
    return e == hipSuccess ? api_ok() : hip_fail(e, "decay attention step launch");
}

gdn_status gdn_paged_append(const gdn_qk_desc* d, const gdn_pages* c, const void* q, const void* k, const void* v,
                            int64_t v_stride, int64_t v_head_stride, const float* q_weight, const float* k_weight,
                            const double* inv_freq, const int64_t* positions, const int64_t* cu_seqlens,
                            const int32_t* page_table, const int64_t* lens, void* q_out, void* k_cache, void* v_cache,
                            void* stream) {
    gdn_status s = check_qk(d);
    if (s != GDN_OK) return s;
    if ((s = check_pages(c, d->k_heads, d->head_dim, k_cache, v_cache, page_table, lens)) != GDN_OK) return s;
    if (cu_seqlens ? d->batch != 1 || c->num_seqs <= 0 : d->batch != c->num_seqs)
        return api_fail(GDN_ERR_BAD_SHAPE, "num_seqs must be the batch, or packed sequences need batch == 1 and num_seqs > 0");
    const int64_t vh = v_head_stride ? v_head_stride : d->head_dim;
    const int64_t vt = v_stride ? v_stride : d->k_heads * vh;
    if (vh < d->head_dim || vt < (d->k_heads - 1) * vh + d->head_dim)
        return api_fail(GDN_ERR_BAD_SHAPE, "v strides %lld, %lld: rows overlap", (long long)v_stride,
                        (long long)v_head_stride);
    if (vh % 8 || vt % 8) return api_fail(GDN_ERR_MISALIGNED, "strides must be multiples of 8 elements");
    if ((q == nullptr) != (q_out == nullptr)) return api_fail(GDN_ERR_NULL_ARG, "q and q_out come together");
    if (!aligned(cu_seqlens, 8)) return api_fail(GDN_ERR_MISALIGNED, "cu_seqlens needs 8-byte alignment");
    if (d->batch * d->seq_len == 0) return api_ok();
    const void* p[4] = {k, v, q, q_out};
    if ((s = check_qk_args(d, p, q ? 4 : 2, q_weight, k_weight, inv_freq, positions)) != GDN_OK) return s;
    gdn::PagedAppend a;
    a.qk = qk_launch(d, q, k, q_weight, k_weight, inv_freq, positions, q_out, nullptr, stream);
    if (!q) a.qk.Hq = 0;
    a.v = v;
    a.vs = vt;
    a.vhs = vh;
    a.kc = pages_of(k_cache, c->k_page_stride, c->k_token_stride, c->k_head_stride);
    a.vc = pages_of(v_cache, c->v_page_stride, c->v_token_stride, c->v_head_stride);
    a.table = page_table;
    a.lens = lens;
    a.cu = cu_seqlens;
    a.N = c->num_seqs;
    a.M = c->max_pages;
    a.pages = c->pages;
    a.page = c->page_size;
    const hipError_t e = gdn::launch_paged_append(a);
    return e == hipSuccess ? api_ok() : hip_fail(e, "paged append launch");
}

gdn_status gdn_paged_attn_workspace(const gdn_paged_attn_desc* d, size_t* bytes) {
    gdn_status s = check_attn(d);
    if (s != GDN_OK) return s;
    if (!bytes) return api_fail(GDN_ERR_NULL_ARG, "bytes is NULL");
    *bytes = attn_bytes(d);
    return api_ok();
}

gdn_status gdn_paged_attn(const gdn_paged_attn_desc* d, const gdn_pages* c, const void* q, const void* k_cache,
                          const void* v_cache, const int32_t* page_table, const int64_t* lens, void* o,
                          void* workspace, size_t workspace_bytes, void* stream) {
    gdn_status s = check_attn(d);
    if (s != GDN_OK) return s;
    if ((s = check_pages(c, d->k_heads, d->head_dim, k_cache, v_cache, page_table, lens)) != GDN_OK) return s;
    if (d->num_seqs != c->num_seqs) return api_fail(GDN_ERR_BAD_SHAPE, "num_seqs of desc and pages differ");
    if (d->num_seqs == 0) return api_ok();
    if (!q || !o) return api_fail(GDN_ERR_NULL_ARG, "q and o are required");
    if (!aligned(q, 16) || !aligned(o, 16)) return api_fail(GDN_ERR_MISALIGNED, "q and o need 16-byte alignment");
    if ((s = check_workspace(workspace, workspace_bytes, attn_bytes(d))) != GDN_OK) return s;
    gdn::PagedAttn a;
    a.q = q;
    a.Hq = (int)d->q_heads;
    a.qhs = d->q_head_stride ? d->q_head_stride : d->head_dim;
    a.qs = d->q_stride ? d->q_stride : a.Hq * a.qhs;
    a.kc = pages_of(const_cast<void*>(k_cache), c->k_page_stride, c->k_token_stride, c->k_head_stride);
    a.vc = pages_of(const_cast<void*>(v_cache), c->v_page_stride, c->v_token_stride, c->v_head_stride);
    a.table = page_table;
    a.lens = lens;
    a.N = d->num_seqs;
    a.M = c->max_pages;
    a.pages = c->pages;
    a.page = c->page_size;
    a.window = d->window;
    a.Hk = (int)d->k_heads;
    a.D = (int)d->head_dim;
    a.scale = d->scale * 1.4426950408889634f;
    a.o = o;
    a.share = gdn::paged_attn_share(d->q_heads, d->k_heads);
    a.part = static_cast<float*>(workspace);
    a.ml = reinterpret_cast<float*>(static_cast<char*>(workspace) + align256(attn_rows(d) * d->head_dim * 4));
    a.bf16 = d->dtype == GDN_DTYPE_BF16;
    a.stream = static_cast<hipStream_t>(stream);
    const hipError_t e = gdn::launch_paged_attn(a);
    return e == hipSuccess ? api_ok() : hip_fail(e, "paged attention launch");
}

}  // extern "C"
