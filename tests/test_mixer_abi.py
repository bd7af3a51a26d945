"""The C ABI of the token mixers on the CPU: sizes, and refusals before anything
is launched (every call below fails validation, so no GPU is touched)."""
import ctypes

import pytest
import torch

import gated_delta_rule_14_amd as gdn

P = ctypes.c_void_p
FAKE, ODD = P(1 << 20), P((1 << 20) + 8)
BIG = 1 << 60


@pytest.fixture(scope="module")
def lib():
    return gdn.load()


def decay(**kw):
    d = dict(batch=2, seq_len=300, num_heads=2, num_v_heads=4, key_dim=128, value_dim=64, num_seqs=0, dtype=1, flags=0,
             scale=0.1)
    d.update(kw)
    return gdn.DecayDesc(**d)


def pages(**kw):
    d = dict(num_seqs=2, max_pages=10, pages=50, page_size=16, k_page_stride=4096, k_token_stride=256, k_head_stride=128,
             v_page_stride=4096, v_token_stride=256, v_head_stride=128)
    d.update(kw)
    return gdn.PagesDesc(**d)


def qk(**kw):
    d = dict(batch=2, seq_len=3, q_heads=4, k_heads=2, head_dim=128, rot_dim=64, dtype=1, norm=2, flags=0, eps=1e-6,
             weight_offset=0.0)
    d.update(kw)
    return gdn.QkDesc(**d)


def attn(**kw):
    d = dict(num_seqs=2, q_heads=4, k_heads=2, head_dim=128, q_stride=0, q_head_stride=0, window=0, dtype=1, scale=0.1)
    d.update(kw)
    return gdn.PagedAttnDesc(**d)


def fwd(lib, d, q=FAKE, g=FAKE, h0=None, cu=None, o=FAKE, ht=None, ws=FAKE, n=BIG):
    return lib.gdn_decay_attn_fwd(d, q, FAKE, FAKE, g, h0, cu, o, ht, ws, n, None)


def bwd(lib, d, do=FAKE, dq=FAKE, dg=FAKE, dh0=None, cu=None, ws=FAKE, n=BIG):
    return lib.gdn_decay_attn_bwd(d, FAKE, FAKE, FAKE, FAKE, None, cu, do, None, dq, FAKE, FAKE, dg, dh0, ws, n, None)


@pytest.mark.parametrize("kw,code", [
    (dict(dtype=2), 3), (dict(flags=2), 4), (dict(key_dim=96), 4), (dict(value_dim=256), 4), (dict(num_heads=0), 2),
    (dict(num_v_heads=3), 2), (dict(num_v_heads=-2), 2), (dict(num_heads=65536, num_v_heads=0), 2), (dict(batch=0), 2),
    (dict(seq_len=-1), 2), (dict(seq_len=1 << 31), 2), (dict(num_seqs=-1), 2), (dict(q_stride=255), 2),
    (dict(k_head_stride=120), 2), (dict(v_head_stride=68), 6), (dict(v_stride=260), 6), (dict(q_stride=-256), 2)])
def test_decay_descriptor(lib, kw, code):
    n, d = ctypes.c_size_t(), decay(**kw)
    assert lib.gdn_decay_attn_workspace(d, 0, n) == code and lib.gdn_last_error().decode() != ""
    assert fwd(lib, d) == code and bwd(lib, d) == code
    assert lib.gdn_decay_attn_step(d, *[FAKE] * 6, None) == code


def test_decay_arguments(lib):
    d, n = decay(), ctypes.c_size_t()
    assert lib.gdn_decay_attn_workspace(None, 0, n) == 1 and lib.gdn_decay_attn_workspace(d, 0, None) == 1
    assert lib.gdn_decay_attn_workspace(d, 0, n) == 0
    f = n.value
    assert f >= 4 * 4 * 128 * 64 * 4                                   # 2 sequences of 2 segments, 4 heads
    assert lib.gdn_decay_attn_workspace(d, 1, n) == 0 and n.value > 2 * f
    one = decay(seq_len=60)
    assert lib.gdn_decay_attn_workspace(one, 0, n) == 0 and n.value == 0   # no segments: no workspace
    assert fwd(lib, d, q=None) == 1 and fwd(lib, d, g=None) == 1 and fwd(lib, d, o=None) == 1
    assert fwd(lib, d, q=ODD) == 6 and fwd(lib, d, h0=ODD) == 6 and fwd(lib, d, ht=ODD) == 6
    assert fwd(lib, d, g=P((1 << 20) + 2)) == 6
    assert fwd(lib, d, cu=FAKE) == 2                                   # packed needs batch 1 and num_seqs
    p = decay(batch=1, num_seqs=5)
    assert fwd(lib, p) == 2 and fwd(lib, p, cu=P((1 << 20) + 4)) == 6
    assert fwd(lib, p, cu=FAKE, ws=None) == 1 and fwd(lib, p, cu=FAKE, ws=P((1 << 20) + 128)) == 6
    assert fwd(lib, p, cu=FAKE, n=64) == 5 and fwd(lib, d, n=f - 1) == 5
    assert bwd(lib, d, do=None) == 1 and bwd(lib, d, dq=ODD) == 6 and bwd(lib, d, dg=None) == 1
    assert bwd(lib, d, dh0=ODD) == 6 and bwd(lib, d, n=100) == 5 and bwd(lib, d, ws=None) == 1
    # many sequences, and sizes past a launch's limits
    assert fwd(lib, decay(batch=1 << 22, seq_len=8, num_v_heads=64)) == 2
    assert bwd(lib, decay(batch=1 << 10, seq_len=1 << 20, num_heads=1 << 12, num_v_heads=1 << 12)) == 2


def test_decay_step_arguments(lib):
    def step(d, q=FAKE, state=FAKE, o=FAKE):
        return lib.gdn_decay_attn_step(d, q, FAKE, FAKE, FAKE, state, o, None)
    d = decay(seq_len=1)
    assert step(decay()) == 2 and step(decay(seq_len=1, num_seqs=2)) == 2
    assert step(d, q=None) == 1 and step(d, state=None) == 1 and step(d, o=None) == 1
    assert step(d, q=ODD) == 6 and step(d, state=ODD) == 6
    assert step(decay(batch=0, seq_len=1), None, None, None) == 0      # no sequences: nothing to do
    assert step(decay(batch=0, seq_len=1, dtype=5)) == 3
    assert step(decay(batch=1 << 23, seq_len=1)) == 2


BAD_PAGES = [
    (dict(pages=0), 2), (dict(page_size=0), 2), (dict(max_pages=0), 2), (dict(max_pages=1 << 28), 2), (dict(pages=1 << 31), 2),
    (dict(k_page_stride=4088), 2), (dict(v_token_stride=248), 2), (dict(k_head_stride=0), 2), (dict(v_page_stride=-4096), 2),
    (dict(k_token_stride=260, k_page_stride=8192), 6), (dict(v_head_stride=132, v_token_stride=264, v_page_stride=8192), 6)]


@pytest.mark.parametrize("kw,code", BAD_PAGES)
def test_pages(lib, kw, code):
    a = [FAKE, FAKE, FAKE, 0, 0, None, None, FAKE, None, None, FAKE, FAKE, FAKE, FAKE, FAKE, None]
    assert lib.gdn_paged_append(qk(), pages(**kw), *a) == code and lib.gdn_last_error().decode() != ""
    assert lib.gdn_paged_attn(attn(), pages(**kw), *[FAKE] * 7, BIG, None) == code


def test_paged_append_arguments(lib):
    def call(d=None, c=None, **kw):
        a = dict(q=FAKE, k=FAKE, v=FAKE, vs=0, vh=0, qw=None, kw=None, f=FAKE, pos=None, cu=None, table=FAKE, lens=FAKE,
                 qo=FAKE, kc=FAKE, vc=FAKE)
        a.update(kw)
        return lib.gdn_paged_append(d or qk(), c or pages(), *a.values(), None)
    assert lib.gdn_paged_append(None, pages(), *[None] * 3, 0, 0, *[None] * 11) == 1
    assert lib.gdn_paged_append(qk(), None, *[None] * 3, 0, 0, *[None] * 11) == 1
    for name in ("k", "v", "f", "table", "lens", "kc", "vc"):
        assert call(**{name: None}) == 1, name
    assert call(q=None) == 1 and call(qo=None) == 1                    # q and q_out come together
    for name in ("q", "k", "v", "qo", "kc", "vc"):
        assert call(**{name: ODD}) == 6, name
    for name, off in (("f", 4), ("pos", 4), ("cu", 4), ("lens", 4), ("table", 2), ("qw", 2)):
        d = dict(d=qk(batch=1), c=pages(num_seqs=3)) if name == "cu" else {}
        assert call(**d, **{name: P((1 << 20) + off)}) == 6, name
    assert call(vs=200) == 2 and call(vh=64) == 2 and call(vh=132) == 6 and call(vs=260) == 6
    assert call(c=pages(num_seqs=3)) == 2 and call(cu=FAKE) == 2 and call(d=qk(batch=1), cu=FAKE, c=pages(num_seqs=0)) == 2
    assert call(d=qk(head_dim=100)) == 4 and call(d=qk(dtype=3)) == 3
    assert call(d=qk(seq_len=0), q=None, k=None, v=None, qo=None) == 0  # no tokens
    assert call(d=qk(batch=0), c=pages(num_seqs=0), q=None, k=None, v=None, qo=None, table=None, lens=None, kc=None,
                vc=None) == 0


@pytest.mark.parametrize("kw,code", [
    (dict(dtype=4), 3), (dict(q_heads=3), 2), (dict(k_heads=0), 2), (dict(q_heads=0), 2), (dict(head_dim=264), 4),
    (dict(head_dim=12), 4), (dict(window=-1), 2), (dict(q_head_stride=64), 2), (dict(q_stride=500), 2),
    (dict(q_stride=516), 6), (dict(num_seqs=-1), 2), (dict(num_seqs=1 << 26), 2), (dict(q_heads=65536, k_heads=1), 2)])
def test_attn_descriptor(lib, kw, code):
    n, d = ctypes.c_size_t(), attn(**kw)
    assert lib.gdn_paged_attn_workspace(d, n) == code
    assert lib.gdn_paged_attn(d, pages(), *[FAKE] * 7, BIG, None) == code


def test_attn_arguments(lib):
    n = ctypes.c_size_t()
    assert lib.gdn_paged_attn_workspace(attn(), None) == 1 and lib.gdn_paged_attn_workspace(None, n) == 1
    assert lib.gdn_paged_attn_workspace(attn(), n) == 0 and n.value > 0

    def call(i=None, v=None, nb=BIG, d=None, c=None):
        a = [FAKE] * 7
        if i is not None:
            a[i] = v
        return lib.gdn_paged_attn(d or attn(), c or pages(), *a, nb, None)
    for i in range(7):
        assert call(i, None) == 1, i
    for i in (0, 1, 2, 5, 6):
        assert call(i, ODD) == 6, i
    assert call(3, P((1 << 20) + 2)) == 6 and call(4, P((1 << 20) + 4)) == 6
    assert call(nb=n.value - 1) == 5 and call(c=pages(num_seqs=3)) == 2
    assert lib.gdn_paged_attn(attn(num_seqs=0), pages(num_seqs=0), *[None] * 7, 0, None) == 0


def test_binding_needs_device_tensors():
    x, g, s = torch.zeros(1, 4, 1, 64), torch.zeros(1, 4, 1), torch.zeros(1, 1, 64, 64)
    kc, table, lens = torch.zeros(3, 8, 1, 64), torch.zeros(1, 3, dtype=torch.int32), torch.zeros(1, dtype=torch.int64)
    for f in (lambda: gdn.decay_attn_fwd(x, x, x, g), lambda: gdn.decay_attn_bwd(x, x, x, g, x),
              lambda: gdn.decay_attn_step(x[0], x[0], x[0], g[0], s), lambda: gdn.paged_append(x, x, x, kc, kc, table, lens),
              lambda: gdn.paged_attn(x[0], kc, kc, table, lens), lambda: gdn.paged_attn_workspace(x[0], kc, kc, table, lens)):
        with pytest.raises(ValueError, match="device tensor"):
            f()
