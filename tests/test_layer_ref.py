"""The 64-bit references of the layer operators against central differences
(CPU), so that the GPU tests rest on gradients of the formulas themselves."""
import pytest
import torch

import layer_ref as ref

F64 = torch.float64


def differ(f, t, cot, grad, eps=1e-5):
    """<cot, f(t)> along three random directions against <grad, direction>."""
    for k in range(3):
        g = torch.Generator().manual_seed(k)
        d = torch.randn(t.shape, dtype=F64, generator=g)
        hi, lo = f(t + eps * d), f(t - eps * d)
        slope = sum(((a - b) * c).sum() for a, b, c in zip(hi, lo, cot)) / (2 * eps)
        want = (grad * d).sum()
        assert abs(slope - want) <= 1e-6 * (1 + (grad.abs() * d.abs()).sum()), (float(slope), float(want))


@pytest.mark.parametrize("normalize", [False, True])
@pytest.mark.parametrize("logits", [False, True])
def test_linrec_reference(normalize, logits):
    torch.manual_seed(3)
    D, cu = 3, torch.tensor([0, 4, 4, 11])
    x, dy = torch.randn(1, 11, D, dtype=F64), torch.randn(1, 11, D, dtype=F64)
    g = torch.randn(1, 11, D, dtype=F64) if logits else -torch.rand(1, 11, D, dtype=F64) - 0.05
    h0, dht = torch.randn(3, D, dtype=F64), torch.randn(3, D, dtype=F64)
    A, b = (torch.randn(D, dtype=F64), torch.randn(D, dtype=F64)) if logits else (None, None)

    def f(**kw):
        a = dict(x=x, g=g, h0=h0, A_log=A, dt_bias=b)
        a.update(kw)
        w, _ = ref.linrec(a["x"], a["g"], a["h0"], cu, normalize, a["A_log"], a["dt_bias"])
        return w["y"], w["ht"]
    w, _ = ref.linrec(x, g, h0, cu, normalize, A, b, dy, dht)
    for name, t, gr in (("x", x, "dx"), ("g", g, "dg"), ("h0", h0, "dh0"), ("A_log", A, "dA_log"),
                        ("dt_bias", b, "ddt_bias")):
        if t is not None:
            differ(lambda v: f(**{name: v}), t, (dy, dht), w[gr])


@pytest.mark.parametrize("norm", ["none", "l2", "rms"])
@pytest.mark.parametrize("inter", [False, True])
def test_qk_reference(norm, inter):
    torch.manual_seed(4)
    x, d = torch.randn(2, 3, 2, 24, dtype=F64), torch.randn(2, 3, 2, 24, dtype=F64)
    w, f = torch.randn(24, dtype=F64), 100.0 ** (-torch.arange(8, dtype=F64) / 8)
    pos = torch.randint(0, 1000, (2, 3))
    want, _ = ref.qk(x, f, pos, norm, 1e-6, w, 1.0, inter, d)
    differ(lambda v: (ref.qk(v, f, pos, norm, 1e-6, w, 1.0, inter)[0]["out"],), x, (d,), want["dx"])
    differ(lambda v: (ref.qk(x, f, pos, norm, 1e-6, v, 1.0, inter)[0]["out"],), w, (d,), want["dw"])


@pytest.mark.parametrize("W", [2, 3, 4])
@pytest.mark.parametrize("silu", [False, True])
def test_conv_reference(W, silu):
    torch.manual_seed(5)
    D, cu = 3, torch.tensor([0, 1, 1, 3, 9])
    x, dy = torch.randn(1, 9, D, dtype=F64), torch.randn(1, 9, D, dtype=F64)
    w, b = torch.randn(D, W, dtype=F64), torch.randn(D, dtype=F64)
    s0, dst = torch.randn(4, W - 1, D, dtype=F64), torch.randn(4, W - 1, D, dtype=F64)

    def f(**kw):
        a = dict(x=x, w=w, b=b, s0=s0)
        a.update(kw)
        r, _ = ref.conv(a["x"], a["w"], a["b"], a["s0"], cu, silu)
        return r["y"], r["st"]
    r, _ = ref.conv(x, w, b, s0, cu, silu, dy, dst)
    for name, t, gr in (("x", x, "dx"), ("w", w, "dweight"), ("b", b, "dbias"), ("s0", s0, "ds0")):
        differ(lambda v: f(**{name: v}), t, (dy, dst), r[gr])
