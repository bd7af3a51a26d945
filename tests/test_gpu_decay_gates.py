"""Gates that are not finite: what a token's gate does not enter stays as it is."""
import pytest
import torch

import layer_ref
import mixer_ref as ref
from test_gpu_decay import inputs

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("T,at", [(50, 30), (64, 0), (130, 129), (300, 290), (700, 200)])
def test_gates_that_are_not_finite(gpu_lib, dt, bad, T, at):
    """A gate stands between the tokens before its own and the rest.  Outputs before it, and dk and dv from its
    token on, do not contain it; nor do the other head and the other sequence."""
    gdn = gpu_lib
    d = inputs(21, 2, T, 2, 2, 64, 128, dt)
    want, err = ref.decay(d["q"], d["k"], d["v"], d["g"], None, d["h0"], None, d["do"], d["dht"])
    d["g"][1, at, 1] = bad
    c = {n: t.cuda() for n, t in d.items()}
    o, ht = gdn.decay_attn_fwd(c["q"], c["k"], c["v"], c["g"], h0=c["h0"])
    got = dict(gdn.decay_attn_bwd(c["q"], c["k"], c["v"], c["g"], c["do"], h0=c["h0"], dht=c["dht"]), o=o, ht=ht)
    torch.cuda.synchronize()
    tokens = ("o", "dq", "dk", "dv", "dg")
    for n in want:
        for part in ((0,), (1, slice(None), 0) if n in tokens else (1, 0)):
            layer_ref.check(got[n][part], want[n][part], err[n][part], n)
    before, after = (1, slice(0, at), 1), (1, slice(at, T), 1)
    for n, clean, hit in (("o", before, after), ("dq", before, after), ("dk", after, before), ("dv", after, before)):
        layer_ref.check(got[n][clean], want[n][clean], err[n][clean], n)
        assert not bool(torch.isfinite(got[n][hit]).any()), n
    for n in ("ht", "dh0"):
        assert not bool(torch.isfinite(got[n][1, 1]).any()), n


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("T,HV,K,V", [(1, 1, 64, 64), (60, 1, 64, 64), (64, 2, 128, 64), (330, 1, 64, 64), (330, 2, 128, 128)])
def test_strong_gates_and_a_final_gradient(gpu_lib, dt, T, HV, K, V):
    """The final state's gradient meets the last token's k v^T undecayed, in no token's dg: 150 times the terms
    that dg has.  Its relative error is 32-bit all the same: K products with V terms, 64 pairs, a chunk each."""
    d = inputs(22, 2, T, 1, HV, K, V, dt)
    d["g"] = -5 - torch.rand(2, T, HV, generator=torch.Generator().manual_seed(3))
    c = {n: t.cuda() for n, t in d.items()}
    got = gpu_lib.decay_attn_bwd(c["q"], c["k"], c["v"], c["g"], c["do"], h0=c["h0"], dht=c["dht"])["dg"].cpu().double()
    torch.cuda.synchronize()
    want = ref.decay(d["q"], d["k"], d["v"], d["g"], None, d["h0"], None, d["do"], d["dht"])[0]["dg"]
    e = (got - want).norm() / want.norm()
    assert e <= (K + V + 64 + -(-T // 64)) * 2.0 ** -24, float(e)
