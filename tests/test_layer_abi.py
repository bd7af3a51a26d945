"""The layer operators' C ABI on the CPU: sizes, and refusals before anything
is launched (every call below fails validation, so no GPU is touched)."""
import ctypes

import pytest
import torch

import gated_delta_rule_14_amd as gdn

P = ctypes.c_void_p
FAKE, ODD = P(1 << 20), P((1 << 20) + 1)
BIG = 1 << 50


@pytest.fixture(scope="module")
def lib():
    return gdn.load()


def linrec(**kw):
    d = dict(batch=2, seq_len=300, channels=64, num_seqs=0, x_stride=0, g_stride=0, y_stride=0, x_dtype=1,
             g_dtype=0, flags=0)
    d.update(kw)
    return gdn.LinrecDesc(**d)


def qk(**kw):
    d = dict(batch=2, seq_len=30, q_heads=4, k_heads=2, head_dim=128, rot_dim=64, q_stride=0, k_stride=0,
             q_head_stride=0, k_head_stride=0, dtype=1, norm=2, flags=0, eps=1e-6, weight_offset=0.0)
    d.update(kw)
    return gdn.QkDesc(**d)


def conv(**kw):
    d = dict(batch=2, seq_len=300, channels=64, num_seqs=0, x_stride=0, y_stride=0, dtype=1, width=4, flags=1)
    d.update(kw)
    return gdn.ConvDesc(**d)


def fwd(lib, d, act=None, x=FAKE, h0=None, cu=None, y=FAKE, ws=FAKE, n=BIG):
    return lib.gdn_linrec_fwd(d, act, x, FAKE, h0, cu, y, None, None, ws, n, None)


def bwd(lib, d, act=None, dy=FAKE, dx=FAKE, dA=None, cu=None, ws=FAKE, n=BIG):
    return lib.gdn_linrec_bwd(d, act, FAKE, FAKE, None, cu, dy, None, None, dx, FAKE, None, dA, dA, ws, n, None)


BAD_ROWS = [(dict(batch=0), 2), (dict(seq_len=-1), 2), (dict(channels=0), 2), (dict(x_stride=63), 2),
            (dict(y_stride=-64), 2), (dict(num_seqs=-1), 2), (dict(seq_len=1 << 31), 2),
            (dict(batch=1 << 20, seq_len=1 << 20), 2), (dict(channels=1 << 31), 2), (dict(flags=2), 4)]


@pytest.mark.parametrize("kw,code", BAD_ROWS + [(dict(x_dtype=2), 3), (dict(g_dtype=-1), 3), (dict(g_stride=5), 2)])
def test_linrec_descriptor(lib, kw, code):
    n = ctypes.c_size_t()
    assert lib.gdn_linrec_workspace(linrec(**kw), 0, n, None) == code
    assert lib.gdn_last_error().decode() != ""
    assert fwd(lib, linrec(**kw)) == code
    assert bwd(lib, linrec(**kw)) == code


def test_linrec_arguments(lib):
    d, n, rows = linrec(), ctypes.c_size_t(), ctypes.c_int64()
    assert lib.gdn_linrec_workspace(None, 0, n, rows) == 1
    assert lib.gdn_linrec_workspace(d, 0, n, rows) == 0 and rows.value >= 2
    f = n.value
    assert lib.gdn_linrec_workspace(d, 1, n, None) == 0 and n.value >= f
    p = linrec(batch=1, num_seqs=5)
    assert lib.gdn_linrec_workspace(p, 0, n, rows) == 0 and n.value >= 5 * 16 and rows.value >= 5
    assert fwd(lib, d, x=None) == 1
    assert fwd(lib, d, x=ODD) == 6
    assert fwd(lib, d, h0=P((1 << 20) + 2)) == 6
    assert fwd(lib, d, cu=FAKE) == 2                                   # packed needs batch 1 and num_seqs
    assert fwd(lib, linrec(batch=1), cu=FAKE) == 2
    assert fwd(lib, p) == 2                                            # num_seqs without offsets
    assert fwd(lib, p, cu=P((1 << 20) + 4)) == 6
    assert fwd(lib, p, cu=FAKE, ws=None) == 1
    assert fwd(lib, p, cu=FAKE, ws=P((1 << 20) + 128)) == 6
    assert fwd(lib, p, cu=FAKE, n=64) == 5
    assert bwd(lib, d, dy=None) == 1 and bwd(lib, d, dx=None) == 1 and bwd(lib, d, dx=ODD) == 6
    assert bwd(lib, d, n=16) == 5 and bwd(lib, d, ws=None) == 1
    for flags, code in ((1, 1), (2, 4), (8, 4), (3, 4)):               # only the gate activation applies
        assert fwd(lib, d, act=gdn.Activation(flags, None, None)) == code
    act = gdn.Activation(1, 1 << 20, 1 << 20)
    assert bwd(lib, d, act=act) == 1                                   # dA_log, ddt_bias required
    assert fwd(lib, d, act=gdn.Activation(1, (1 << 20) + 2, 1 << 20)) == 6


def test_linrec_step_arguments(lib):
    def step(d, x=FAKE, state=FAKE, y=FAKE):
        return lib.gdn_linrec_step(d, None, x, FAKE, state, y, None)
    d = linrec(seq_len=1)
    assert step(linrec()) == 2 and step(linrec(seq_len=1, num_seqs=2)) == 2
    assert step(d, x=None) == 1 and step(d, state=None) == 1 and step(d, y=None) == 1
    assert step(d, x=ODD) == 6 and step(d, state=P((1 << 20) + 2)) == 6
    assert step(linrec(batch=0, seq_len=1), None, None, None) == 0     # no sequences: nothing to do
    assert step(linrec(batch=0, seq_len=1, x_dtype=5)) == 3


@pytest.mark.parametrize("kw,code", [
    (dict(dtype=2), 3), (dict(norm=3), 4), (dict(norm=-1), 4), (dict(flags=2), 4), (dict(batch=-1), 2),
    (dict(seq_len=-1), 2), (dict(q_heads=0), 2), (dict(k_heads=0), 2), (dict(head_dim=100), 4),
    (dict(head_dim=264), 4), (dict(head_dim=0), 4), (dict(rot_dim=24), 4), (dict(rot_dim=144), 4),
    (dict(rot_dim=-16), 4), (dict(q_stride=504), 2), (dict(k_head_stride=120), 2), (dict(q_head_stride=132), 6),
    (dict(q_stride=516), 6), (dict(batch=1 << 16, seq_len=1 << 16), 2)])
def test_qk_descriptor(lib, kw, code):
    n, d = ctypes.c_size_t(), qk(**kw)
    assert lib.gdn_qk_norm_rope_bwd_workspace(d, n) == code
    assert lib.gdn_qk_norm_rope(d, *[FAKE] * 8, None) == code
    assert lib.gdn_qk_norm_rope_bwd(d, *[FAKE] * 13, BIG, None) == code


def test_qk_arguments(lib):
    d = qk()

    def call(i, v):
        a = [FAKE, FAKE, None, None, FAKE, None, FAKE, FAKE]
        a[i] = v
        return lib.gdn_qk_norm_rope(d, *a, None)
    for i in (0, 1, 6, 7):
        assert call(i, None) == 1 and call(i, P((1 << 20) + 8)) == 6
    assert call(4, None) == 1 and call(4, P((1 << 20) + 4)) == 6       # inv_freq
    assert call(5, P((1 << 20) + 4)) == 6 and call(2, P((1 << 20) + 2)) == 6
    assert lib.gdn_qk_norm_rope(qk(batch=0), *[None] * 8, None) == 0   # no tokens
    assert lib.gdn_qk_norm_rope(None, *[FAKE] * 8, None) == 1
    assert lib.gdn_qk_norm_rope_bwd_workspace(d, None) == 1

    def back(i, v, n=BIG):
        a = [FAKE, FAKE, FAKE, FAKE, FAKE, None, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE]
        a[i] = v
        return lib.gdn_qk_norm_rope_bwd(d, *a, n, None)
    for i in (0, 1, 6, 7, 8, 9):
        assert back(i, None) == 1 and back(i, P((1 << 20) + 8)) == 6
    assert back(2, None) == 1                                          # a weight's gradient without the weight
    assert back(10, P((1 << 20) + 2)) == 6
    assert back(12, None) == 1 and back(12, P((1 << 20) + 128)) == 6 and back(0, FAKE, n=0) == 5


@pytest.mark.parametrize("kw,code", BAD_ROWS + [(dict(dtype=2), 3), (dict(width=1), 4), (dict(width=5), 4)])
def test_conv_descriptor(lib, kw, code):
    n, d = ctypes.c_size_t(), conv(**kw)
    assert lib.gdn_short_conv_workspace(d, 0, n) == code
    assert lib.gdn_short_conv_fwd(d, FAKE, FAKE, None, None, None, FAKE, None, FAKE, BIG, None) == code
    assert lib.gdn_short_conv_bwd(d, FAKE, FAKE, None, None, None, FAKE, None, FAKE, FAKE, None, None, FAKE, BIG,
                                  None) == code


def test_conv_arguments(lib):
    def f(d=None, x=FAKE, w=FAKE, s0=None, cu=None, y=FAKE, st=None, ws=FAKE, n=BIG):
        return lib.gdn_short_conv_fwd(d or conv(), x, w, None, s0, cu, y, st, ws, n, None)
    assert f(x=None) == 1 and f(w=None) == 1 and f(y=None) == 1
    assert f(x=ODD) == 6 and f(s0=ODD) == 6 and f(w=P((1 << 20) + 2)) == 6
    assert f(s0=FAKE, st=FAKE) == 4                                    # the carried window is read to the end
    p = conv(batch=1, num_seqs=4)
    assert f(p) == 2 and f(cu=FAKE) == 2 and f(p, cu=P((1 << 20) + 4)) == 6
    assert f(p, cu=FAKE, n=100) == 5 and f(p, cu=FAKE, ws=None) == 1 and f(p, cu=FAKE, ws=P((1 << 20) + 8)) == 6

    def b(bias=None, db=None, dy=FAKE, dw=FAKE, n=BIG):
        return lib.gdn_short_conv_bwd(conv(), FAKE, FAKE, bias, None, None, dy, None, FAKE, dw, db, None, FAKE, n,
                                      None)
    assert b(dy=None) == 1 and b(dw=None) == 1 and b(bias=FAKE) == 1 and b(db=FAKE) == 1 and b(dy=ODD) == 6
    assert b(n=8) == 5
    one = conv(seq_len=1)
    assert lib.gdn_short_conv_step(conv(), FAKE, FAKE, None, FAKE, FAKE, None) == 2
    assert lib.gdn_short_conv_step(one, FAKE, FAKE, None, None, FAKE, None) == 1
    assert lib.gdn_short_conv_step(one, FAKE, FAKE, None, ODD, FAKE, None) == 6
    assert lib.gdn_short_conv_step(conv(batch=0, seq_len=1), None, None, None, None, None, None) == 0


def test_binding_needs_device_tensors():
    x, s = torch.zeros(1, 4, 8), torch.zeros(1, 8)
    for f in (lambda: gdn.linrec_fwd(x, x), lambda: gdn.linrec_bwd(x, x, x), lambda: gdn.linrec_step(s, s, s),
              lambda: gdn.linrec_states(x), lambda: gdn.qk_norm_rope(x[None], x[None]),
              lambda: gdn.qk_norm_rope_bwd(x[None], x[None], x[None], x[None]),
              lambda: gdn.short_conv_fwd(x, torch.zeros(8, 4)), lambda: gdn.short_conv_bwd(x, torch.zeros(8, 4), x),
              lambda: gdn.short_conv_step(s, torch.zeros(8, 4), torch.zeros(1, 3, 8))):
        with pytest.raises(ValueError, match="device tensor"):
            f()
