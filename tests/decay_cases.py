"""Shapes at which the gates' gradient of the decayed linear attention is held to its norm, and walks of
many chunks, with what of them is compared; and that norm's bound."""
from __future__ import annotations

import torch

import mixer_ref as ref
from layer_ref import U
from test_gpu_decay import inputs, offsets

CHUNK = 64


def _gates(kind, T):
    r = torch.Generator().manual_seed(9)
    u = torch.rand(1, T, 2, generator=r)
    return {"none": 0 * u, "strong": -5 - 20 * u, "cut": torch.where(u < 0.1, -float("inf"), -0.1 * u),
            "mixed": torch.where(u < 0.2, -torch.exp(12 * u / 0.2), -0.01 * u), "growing": 0.1 * (u - 0.3)}[kind]


def _short():
    """Short sequences and segments of a chunk or two, as test_gpu_decay.py has them."""
    for K, V in ((64, 64), (64, 128), (128, 64), (128, 128)):
        for T in (63, 65, 130):
            yield "head%dx%d-%d" % (K, V, T), dict(B=2, T=T, H=1, HV=1, K=K, V=V), {}
    for T in (2, 256, 257, 700):
        yield "length-%d" % T, dict(B=1, T=T, H=2, HV=2, K=64, V=64, gate=0.1), {}
    for name, n in (("few", (5, 0, 70, 1)), ("segments", (0, 300, 0, 600, 256, 1, 0)), ("ones", (1,) * 40)):
        yield "packed-" + name, dict(B=1, T=sum(n), H=1, HV=2, K=64, V=64, N=len(n)), dict(lengths=n)
    for H, HV in ((1, 3), (2, 4)):
        for per in (False, True):
            yield "shared%d-%d%s" % (H, HV, "-head" if per else ""), \
                dict(B=2, T=300, H=H, HV=HV, K=64, V=128, per_head=per), dict(scale=0.3)
            yield "shared%d-%d%s-packed" % (H, HV, "-head" if per else ""), \
                dict(B=1, T=75, H=H, HV=HV, K=128, V=64, N=3, per_head=per), dict(lengths=(33, 0, 42), ends=False)
    yield "slices", dict(B=1, T=400, H=1, HV=1, K=128, V=128, N=2, gap=True), dict(lengths=(390, 10))
    for kind in ("none", "strong", "cut", "mixed", "growing"):
        yield "gates-" + kind, dict(B=1, T=330, H=2, HV=2, K=64, V=64), dict(gates=kind)
    for name, n in (("few", (0, 5, 0)), ("many", (3,) * 600), ("segments", (700, 0, 40))):
        yield "head-over-" + name, dict(B=1, T=sum(n), H=1, HV=2, K=64, V=64, N=len(n), per_head=True), dict(lengths=n)


def _long():
    """Walks of several chunks in a segment, or of a whole sequence, the last one short: `tile` tokens to a
    segment; `see`: the (sequence, state head) pairs that are compared."""
    # sequences walked whole, of five chunks and ten tokens
    yield "whole-330", dict(B=512, T=330, H=1, HV=1, K=64, V=64), dict(tile=384, see=((0, 0), (511, 0)))
    yield "whole-330-head", dict(B=256, T=330, H=1, HV=2, K=64, V=128, per_head=True), dict(tile=384, see=((0, 1), (255, 0)))
    # segments of six chunks, the last of 348 tokens
    yield "segments-384", dict(B=1, T=1500, H=64, HV=128, K=64, V=64), dict(tile=384, see=((0, 0), (0, 127)))
    yield "segments-384-wide", dict(B=1, T=1500, H=128, HV=128, K=128, V=128), dict(tile=384, see=((0, 70),))
    yield "segments-448-slices", dict(B=2, T=900, H=60, HV=120, K=128, V=64, gap=True), dict(tile=448, see=((0, 3), (1, 119)))
    # packed: a sequence as long as a segment, one a token longer, one of ten segments
    yield "packed-320", dict(B=1, T=2560, H=32, HV=64, K=64, V=64, N=6), \
        dict(tile=320, lengths=(320, 321, 1, 0, 1900, 18), see=((0, 0), (1, 63), (2, 5), (3, 5), (4, 31), (5, 0)))
    yield "packed-192", dict(B=1, T=2900, H=32, HV=32, K=64, V=128, N=4), \
        dict(tile=192, lengths=(2000, 192, 193, 515), see=((0, 31), (1, 0), (2, 1), (3, 2)))
    yield "packed-192-head", dict(B=1, T=2900, H=32, HV=32, K=64, V=64, N=4, per_head=True), \
        dict(tile=192, lengths=(2000, 192, 193, 515), see=((0, 31), (1, 0), (2, 1), (3, 2)))


SHORT = {n: (a, o) for n, a, o in _short()}
LONG = {n: (a, o) for n, a, o in _long()}


def problem(name, dt):
    """CPU inputs of a case and its options."""
    a, o = (SHORT.get(name) or LONG[name])
    d = inputs(sum(map(ord, name)), dt=dt, **a)
    if "gates" in o:
        d["g"] = _gates(o["gates"], a["T"])
    return d, o


def reference(d, o):
    """Values, bounds, and dg of each token [B, T, H_V] also where a gate serves a head, with what the 64-bit
    reference takes for it."""
    cu = offsets(o["lengths"]) if "lengths" in o else None
    ends = o.get("ends", True)
    args = (o.get("scale"), d["h0"] if ends else None, cu, d["do"], d["dht"] if ends else None)
    want, err = ref.decay(d["q"], d["k"], d["v"], d["g"], *args)
    per_token = want["dg"]
    if d["g"].dim() == 1:
        per_token = ref.decay(d["q"], d["k"], d["v"], d["g"].expand(d["v"].shape[:3]).contiguous(), *args)[0]["dg"]
    return want, err, per_token


def seen(d, o, seq, head):
    """The inputs of one sequence and state head of a case, alone: a problem of its own."""
    m = d["v"].shape[2] // d["q"].shape[2]
    if "lengths" in o:
        a = sum(o["lengths"][:seq])
        row, tok = 0, slice(a, a + o["lengths"][seq])
    else:
        row, tok = seq, slice(None)
    one = {n: d[n][row:row + 1, tok, head // m:head // m + 1] for n in "qk"}
    one.update({n: d[n][row:row + 1, tok, head:head + 1] for n in ("v", "do")})
    one["g"] = d["g"][head:head + 1] if d["g"].dim() == 1 else d["g"][row:row + 1, tok, head:head + 1]
    one.update({n: d[n][seq:seq + 1, head:head + 1] for n in ("h0", "dht")})
    return {n: t.contiguous() for n, t in one.items()}, (row, tok)


def dg_bound(per_token, K, V, longest):
    """Bound on the norm of dg's error, for each state head.

    A sum in 32 bits of n terms of either sign is off by at most n half units, 2^-24, of what it comes to on
    the way, and that is as large as dg itself: every sum on the way to dg_t is dg of another token, or the
    change from one to the next.  Terms: K and V of the products with the state, 64 pairs of a chunk,
    and one more for each chunk that the states pass."""
    return (K + V + CHUNK + longest / CHUNK) * U * per_token.flatten(0, -2).norm(dim=0)


def check_dg(got, want, per_token, K, V, longest, what="dg"):
    """got within dg_bound of want; for a gate of each head, whose error is the sum of its tokens', within
    sqrt(tokens) times it (Cauchy and Schwarz) and its own last rounding."""
    lim = dg_bound(per_token, K, V, longest)
    e = got.detach().cpu().double() - want
    if want.dim() == 1:
        lim = lim * per_token.flatten(0, -2).shape[0] ** 0.5 + U * want.abs()
    else:
        e = e.flatten(0, -2).norm(dim=0)
    assert bool((e.abs() <= lim).all()), "%s: off by %s, bound %s" % (what, e.tolist(), lim.tolist())
