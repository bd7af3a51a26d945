"""The 64-bit reference of the decayed linear attention against central
differences and against its definition as a sum over pairs (CPU)."""
import pytest
import torch

import mixer_ref as ref
from test_layer_ref import differ

F64 = torch.float64
NAMES = (("q", "dq"), ("k", "dk"), ("v", "dv"), ("g", "dg"), ("h0", "dh0"))


def problem(per_head, seed=3):
    r = torch.Generator().manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=r, dtype=torch.float32)  # noqa: E731
    T, H, HV, K, V = 11, 2, 4, 3, 5
    g = -0.3 * torch.rand(HV, generator=r) if per_head else -torch.rand(1, T, HV, generator=r)
    return dict(q=n(1, T, H, K), k=n(1, T, H, K), v=n(1, T, HV, V), g=g, h0=n(3, HV, K, V)), \
        dict(do=n(1, T, HV, V), dht=n(3, HV, K, V)), torch.tensor([0, 4, 4, 11])


@pytest.mark.parametrize("per_head", [False, True])
def test_gradients(per_head, monkeypatch):
    x, d, cu = problem(per_head)
    monkeypatch.setitem(ref.HALF, F64, 0.0)
    x, d = {n: t.to(F64) for n, t in x.items()}, {n: t.to(F64) for n, t in d.items()}

    def f(**kw):
        a = dict(x, **kw)
        w, _ = ref.decay(a["q"], a["k"], a["v"], a["g"], None, a["h0"], cu)
        return w["o"], w["ht"]
    w, e = ref.decay(x["q"], x["k"], x["v"], x["g"], None, x["h0"], cu, d["do"], d["dht"])
    for name, gr in NAMES:
        differ(lambda t: f(**{name: t}), x[name], (d["do"], d["dht"]), w[gr])
        assert e[gr].shape == w[gr].shape and bool((e[gr] >= 0).all())


def test_pairs():
    """o_i = scale sum_{j <= i} exp(g_{j+1} + ... + g_i) (q_i k_j) v_j."""
    x, _, cu = problem(False, 4)
    w, _ = ref.decay(x["q"], x["k"], x["v"], x["g"], 0.7, None, cu)
    q, k = (x[n].to(F64).repeat_interleave(2, 2) for n in "qk")
    v, g = x["v"].to(F64), x["g"].to(F64)
    for i in range(11):
        first = 0 if i < 4 else 4
        want = sum(0.7 * torch.exp(g[0, j + 1:i + 1].sum(0))[:, None] * (q[0, i] * k[0, j]).sum(-1, keepdim=True) * v[0, j]
                   for j in range(first, i + 1))
        assert torch.allclose(w["o"][0, i], want, rtol=1e-12, atol=1e-12)
