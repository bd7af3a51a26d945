"""Linear attention with a decay for each head on the GPU: the gates' gradient held to its norm, and walks of
many chunks, by sequence and state head against the 64-bit token recurrence."""
import ctypes

import pytest
import torch

import decay_cases as dc
import layer_ref
from test_gpu_decay import cuda, offsets

pytestmark = pytest.mark.gpu
TOKENS = ("o", "dq", "dk", "dv", "dg")


def call(gdn, d, o):
    """Outputs and gradients of a case, on the CPU."""
    c, ends = cuda(d), o.get("ends", True)
    kw = dict(scale=o.get("scale"), h0=c["h0"] if ends else None,
              cu_seqlens=offsets(o["lengths"]).cuda() if "lengths" in o else None)
    y, ht = gdn.decay_attn_fwd(c["q"], c["k"], c["v"], c["g"], **kw)
    got = gdn.decay_attn_bwd(c["q"], c["k"], c["v"], c["g"], c["do"], dht=c["dht"] if ends else None, **kw)
    torch.cuda.synchronize()
    return {n: t.cpu() for n, t in dict(got, o=y, ht=ht).items()}


def sizes(d, longest):
    return d["q"].shape[3], d["v"].shape[3], longest


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("name", dc.SHORT)
def test_gate_gradients(gpu_lib, dt, name):
    """dg is made in 32 bits from both types' inputs."""
    d, o = dc.problem(name, dt)
    got = call(gpu_lib, d, o)
    want, _, per_token = dc.reference(d, o)
    dc.check_dg(got["dg"], want["dg"], per_token, *sizes(d, max(o.get("lengths", (d["v"].shape[1],)))), what=name)


def aligned(n):
    return (n + 255) // 256 * 256


def workspace_of(d, o):
    """Bytes of the forward's workspace with segments of o["tile"] tokens: a table of packed sequences, and the
    segments' states and decays."""
    B, T, HV = d["g"].shape if d["g"].dim() > 1 else (*d["v"].shape[:2], d["g"].numel())
    N, tile = len(o.get("lengths", ())), o["tile"]
    rows = -(-T // tile) + min(N, T // (tile + 1)) if N else B * -(-T // tile)
    table = 256 + aligned(16 * N) + aligned(32 * rows) if N else 0
    if T <= tile:
        rows = 0
    return table + aligned(rows * HV * d["q"].shape[3] * d["v"].shape[3] * 4) + aligned(rows * HV * 4)


def needs(gdn, d, o):
    B, T, H, K = d["q"].shape
    n, HV, V = ctypes.c_size_t(), d["v"].shape[2], d["v"].shape[3]
    desc = gdn.DecayDesc(batch=B, seq_len=T, num_heads=H, num_v_heads=HV, key_dim=K, value_dim=V,
                         num_seqs=len(o.get("lengths", ())), dtype=1, flags=int(d["g"].dim() == 1), scale=1.0)
    assert gdn.load().gdn_decay_attn_workspace(desc, 0, n) == 0
    return n.value


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("name", dc.LONG)
def test_walks_of_many_chunks(gpu_lib, dt, name):
    """Segments, and sequences without them, of three chunks or more: their states, the gates of the chunk after
    next, the rest at a walk's end and the sums of more than 256 tokens."""
    gdn = gpu_lib
    d, o = dc.problem(name, dt)
    assert o["tile"] >= 3 * dc.CHUNK and needs(gdn, d, o) == workspace_of(d, o)
    got = call(gdn, d, o)
    shared, per_head = d["v"].shape[2] != d["q"].shape[2], d["g"].dim() == 1
    for seq, head in o["see"]:
        one, (row, tok) = dc.seen(d, o, seq, head)
        want, err, per_token = dc.reference(one, {})
        what = "%s %d/%d " % (name, seq, head)
        for n in ("ht", "dh0"):
            layer_ref.check(got[n][seq, head], want[n][0, 0], err[n][0, 0], what + n)
        for n in ("o", "dv"):
            layer_ref.check(got[n][row, tok, head], want[n][0, :, 0], err[n][0, :, 0], what + n)
        if not shared:
            for n in ("dq", "dk"):
                layer_ref.check(got[n][row, tok, head], want[n][0, :, 0], err[n][0, :, 0], what + n)
        if not per_head and one["v"].shape[1] > 0:
            dc.check_dg(got["dg"][row, tok, head][None, :, None], want["dg"], per_token,
                        *sizes(d, one["v"].shape[1]), what=what + "dg")


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_shared_heads_of_many_chunks(gpu_lib, dt):
    """dq and dk of a head sum the terms of the state heads that use it; dg of a gate for each head sums
    every token of every sequence."""
    d, o = dc.problem("segments-384", dt)
    got = call(gpu_lib, d, o)
    sums, errs = {}, {}
    for head in (62, 63):                                  # the state heads of q's and k's head 31
        one, _ = dc.seen(d, o, 0, head)
        want, err, _ = dc.reference(one, {})
        for n in ("dq", "dk"):
            sums[n] = sums.get(n, 0) + want[n][0, :, 0]
            errs[n] = errs.get(n, 0) + err[n][0, :, 0] + 2 * layer_ref.U * want[n][0, :, 0].abs()
    for n in sums:
        layer_ref.check(got[n][0, :, 31], sums[n], errs[n], n)
    for name, (args, o) in dc.LONG.items():
        if not args.get("per_head") or "lengths" not in o:
            continue
        d, o = dc.problem(name, dt)
        got = call(gpu_lib, d, o)
        for head in (0, d["g"].numel() - 1):
            parts = [dc.reference(dc.seen(d, o, s, head)[0], {}) for s, n in enumerate(o["lengths"]) if n]
            per_token = torch.cat([p[2] for p in parts], 1)
            dc.check_dg(got["dg"][head:head + 1], sum(p[0]["dg"] for p in parts), per_token,
                        *sizes(d, max(o["lengths"])), what="%s head %d" % (name, head))


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("name", ["whole-330", "segments-384", "packed-192"])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_not_finite_in_walks_of_many_chunks(gpu_lib, dt, name, bad):
    """A value or gate that is not finite, in the middle of a walk: what does not see it is as without it."""
    gdn = gpu_lib
    d, o = dc.problem(name, dt)
    seq, head = o["see"][0]
    m = d["v"].shape[2] // d["q"].shape[2]
    one, (row, tok) = dc.seen(d, o, seq, head)
    T, at = one["v"].shape[1], one["v"].shape[1] * 5 // 9
    want, err, _ = dc.reference(one, {})
    for name in ("q", "k", "v", "do", "g"):
        x = dict(d, **{name: d[name].clone()})
        x[name][(row, (tok.start or 0) + at, head // m if name in "qk" else head) + ((7,) if name != "g" else ())] = bad
        got = call(gdn, x, o)
        before, after = slice(0, at), slice(at + 1, T)
        clean = dict(q=[("o", before), ("o", after), ("dq", before), ("dq", after), ("dk", after), ("dv", after)],
                     k=[("o", before), ("dq", before), ("dk", before), ("dk", after), ("dv", before), ("dv", after)],
                     v=[("o", before), ("dq", before), ("dk", before), ("dk", after), ("dv", before), ("dv", after)],
                     do=[("o", slice(0, T)), ("dq", before), ("dq", after), ("dk", after), ("dv", after)],
                     g=[("o", before), ("dq", before), ("dk", slice(at, T)), ("dv", slice(at, T))])[name]
        for n, part in clean:
            if n in ("dq", "dk") and m > 1:                # sums over the heads that share it
                assert bool(torch.isfinite(got[n][row, tok, head // m][part]).all()), (n, name)
            else:
                layer_ref.check(got[n][row, tok, head][part], want[n][0, part, 0], err[n][0, part, 0], "%s of bad %s" % (n, name))
        seen = dict(q=[("dv", slice(0, at + 1), slice(None))], k=[("o", slice(at, at + 1), slice(None))],
                    v=[("o", slice(at, T), 7)], do=[("dv", slice(0, at + 1), 7)],
                    g=[("o", slice(at, T), slice(None)), ("dv", before, slice(None))])[name]
        for n, part, col in seen:
            assert not bool(torch.isfinite(got[n][row, tok, head][part, col]).any()), (n, name)
