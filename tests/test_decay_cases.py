"""The bound on the gates' gradient rejects wrong ones at every shape that it is used at (CPU): mistakes
are planted in the 64-bit reference's values."""
import pytest
import torch

import decay_cases as dc


def without_pairs(d, per_token):
    """dg without each token's pair with the one before it, one of those that its chunk's sums are made of."""
    m = d["v"].shape[2] // d["q"].shape[2]
    q, k = (d[n].double().repeat_interleave(m, 2) for n in "qk")
    g = d["g"].double().expand(d["v"].shape[:3])
    out = per_token.clone()
    x = (q * torch.roll(k, 1, 1)).sum(-1) * (d["do"].double() * torch.roll(d["v"].double(), 1, 1)).sum(-1) * torch.exp(g)
    out[:, 1:] -= x[:, 1:] * d["q"].shape[3] ** -0.5
    return out


def rejected(got, want, per_token, *sizes):
    try:
        dc.check_dg(got.float(), want, per_token, *sizes)
    except AssertionError:
        return True
    return False


def run(d, o, name):
    K, V = d["q"].shape[3], d["v"].shape[3]
    n = o.get("lengths", (d["v"].shape[1],))
    want, _, per_token = dc.reference(d, o)
    want, sizes = want["dg"], (K, V, max(n))
    dc.check_dg(want.float(), want, per_token, *sizes)                 # the right one, rounded, passes
    total = (lambda x: x.flatten(0, -2).sum(0)) if want.dim() == 1 else (lambda x: x)
    if bool((want != 0).any()):
        wrong = dict(zero=0 * want, sign=-want, half=0.5 * want, more=1.01 * want)
        if max(n) > 2 and o.get("gates") != "strong":
            wrong["pairs"] = total(without_pairs(d, per_token))
        for what, w in wrong.items():
            assert rejected(w, want, per_token, *sizes), (name, what)


@pytest.mark.parametrize("name", dc.SHORT)
def test_wrong_gate_gradients_are_rejected(name):
    run(*dc.problem(name, "f32"), name)


@pytest.mark.parametrize("name", dc.LONG)
def test_wrong_gate_gradients_of_long_walks_are_rejected(name):
    d, o = dc.problem(name, "bf16")
    for seq, head in o["see"][:2]:
        one, _ = dc.seen(d, o, seq, head)
        if one["v"].shape[1] > 0:
            run(one, {}, name)
