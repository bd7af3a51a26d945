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
