"""Linear attention with a decay for each head on the GPU against the 64-bit
token recurrence, within bounds on the rounding of every step."""
import pytest
import torch

import layer_ref
import mixer_ref as ref

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def inputs(seed, B, T, H, HV, K, V, dt="bf16", N=None, per_head=False, gate=0.3, gap=False):
    """CPU inputs; gap: q, k, v between NaNs of wider rows."""
    r = torch.Generator().manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=r)  # noqa: E731
    N = B if N is None else N
    d = dict(q=n(B, T, H, K), k=n(B, T, H, K), v=n(B, T, HV, V), do=n(B, T, HV, V))
    d = {k_: t.to(DT[dt]) for k_, t in d.items()}
    g = torch.rand(HV, generator=r) if per_head else torch.rand(B, T, HV, generator=r)
    d.update(g=-gate * g * g, h0=n(N, HV, K, V), dht=n(N, HV, K, V))
    if gap:
        for name in "qkv":
            t = d[name]
            wide = torch.full((B, T, t.shape[2] + 1, t.shape[3] + 8), float("nan"), dtype=t.dtype)
            d[name] = wide[:, :, :-1, 8:] if t.shape[3] % 8 == 0 else t
            d[name].copy_(t)
    return d


def cuda(d):
    out = {}
    for n, t in d.items():
        if t.is_contiguous():
            out[n] = t.cuda()
        else:                      # keep the strides and what lies between the rows
            base = torch.empty(0, dtype=t.dtype).set_(t.untyped_storage()).cuda()
            out[n] = base.as_strided(t.shape, t.stride(), t.storage_offset())
    return out


def both(gdn, d, cu=None, scale=None, h0=True, dht=True):
    c = cuda(d)
    cud = None if cu is None else cu.cuda()
    kw = dict(scale=scale, h0=c["h0"] if h0 else None, cu_seqlens=cud)
    o, ht = gdn.decay_attn_fwd(c["q"], c["k"], c["v"], c["g"], **kw)
    out = gdn.decay_attn_bwd(c["q"], c["k"], c["v"], c["g"], c["do"], dht=c["dht"] if dht else None, **kw)
    torch.cuda.synchronize()
    want, err = ref.decay(d["q"], d["k"], d["v"], d["g"], scale, d["h0"] if h0 else None, cu, d["do"],
                          d["dht"] if dht else None)
    got = dict(out, o=o, ht=ht)
    layer_ref.check_all(got, want, err)
    return got


def offsets(lengths):
    return torch.tensor([sum(lengths[:i]) for i in range(len(lengths) + 1)])


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("K,V", [(64, 64), (64, 128), (128, 64), (128, 128)])
@pytest.mark.parametrize("T", [1, 63, 65, 130])
def test_head_sizes(gpu_lib, dt, K, V, T):
    both(gpu_lib, inputs(1, 2, T, 1, 1, K, V, dt))


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("T", [0, 2, 64, 256, 257, 700])
def test_lengths(gpu_lib, dt, T):
    both(gpu_lib, inputs(2, 1, T, 2, 2, 64, 64, dt, gate=0.1))


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("lengths", [(5, 0, 70, 1), (0,), (0, 300, 0, 600, 256, 1, 0), (1,) * 40])
def test_packed(gpu_lib, dt, lengths):
    both(gpu_lib, inputs(3, 1, sum(lengths), 1, 2, 64, 64, dt, N=len(lengths)), offsets(lengths))


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("H,HV", [(1, 3), (2, 4)])
@pytest.mark.parametrize("per_head", [False, True])
def test_shared_heads_and_gates(gpu_lib, dt, H, HV, per_head):
    both(gpu_lib, inputs(4, 2, 300, H, HV, 64, 128, dt, per_head=per_head), scale=0.3)
    both(gpu_lib, inputs(5, 1, 75, H, HV, 128, 64, dt, N=3, per_head=per_head), offsets((33, 0, 42)), h0=False, dht=False)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_rows_in_wider_tensors(gpu_lib, dt):
    both(gpu_lib, inputs(6, 2, 90, 2, 4, 64, 64, dt, gap=True))
    both(gpu_lib, inputs(7, 1, 400, 1, 1, 128, 128, dt, gap=True, N=2), offsets((390, 10)))


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("kind", ["none", "strong", "cut", "mixed", "growing"])
def test_gates(gpu_lib, dt, kind):
    d = inputs(8, 1, 330, 2, 2, 64, 64, dt)
    r = torch.Generator().manual_seed(9)
    u = torch.rand(1, 330, 2, generator=r)
    d["g"] = {"none": 0 * u, "strong": -5 - 20 * u, "cut": torch.where(u < 0.1, -float("inf"), -0.1 * u),
              "mixed": torch.where(u < 0.2, -torch.exp(12 * u / 0.2), -0.01 * u), "growing": 0.1 * (u - 0.3)}[kind]
    got = both(gpu_lib, d)
    if kind == "cut":
        at = torch.isinf(d["g"])
        assert at.any() and bool((got["dg"].cpu()[at] == 0).all())


def test_strong_gates_keep_their_digits(gpu_lib):
    """dg of gates around -5 is 1/150 of the undecayed products; its relative error is 32-bit all the
    same: 64 products of 64 + 64 terms, sums over a chunk and over the segment's five, in 2^-24 each."""
    d = inputs(10, 1, 330, 1, 1, 64, 64, "f32")
    d["g"] = -5 - torch.rand(1, 330, 1, generator=torch.Generator().manual_seed(1))
    got = both(gpu_lib, d, dht=False)
    want, _ = ref.decay(d["q"], d["k"], d["v"], d["g"], None, d["h0"], None, d["do"], None)
    e = (got["dg"].cpu().double() - want["dg"]).norm() / want["dg"].norm()
    assert e <= (64 + 64 + 64 + 5) * 2.0 ** -24, float(e)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("N,H,HV,K,V", [(1, 1, 1, 64, 64), (3, 2, 6, 64, 128), (5, 1, 2, 128, 64), (300, 1, 2, 128, 128)])
@pytest.mark.parametrize("per_head", [False, True])
def test_step(gpu_lib, dt, N, H, HV, K, V, per_head):
    gdn = gpu_lib
    d = inputs(11, N, 1, H, HV, K, V, dt, per_head=per_head, gap=N == 3)
    c = cuda(d)
    state = c["h0"].clone()
    o = gdn.decay_attn_step(c["q"][:, 0], c["k"][:, 0], c["v"][:, 0], c["g"] if per_head else c["g"][:, 0], state)
    torch.cuda.synchronize()
    want, err = ref.step(d["q"][:, 0], d["k"][:, 0], d["v"][:, 0], d["g"] if per_head else d["g"][:, 0], d["h0"])
    layer_ref.check_all(dict(o=o, state=state), want, err)


def test_prefill_then_steps(gpu_lib):
    """Two prompts carrying the state, then tokens one by one, in the state's own buffer."""
    gdn = gpu_lib
    d = inputs(12, 2, 300, 2, 4, 64, 64, "f32")
    want, err = ref.decay(d["q"], d["k"], d["v"], d["g"], None, d["h0"])
    c, outs, h = cuda(d), [], d["h0"].cuda()
    for a, e in ((0, 130), (130, 290)):
        part = [c[n][:, a:e].contiguous() for n in ("q", "k", "v", "g")]
        o, h2 = gdn.decay_attn_fwd(*part, h0=h, ht=h)
        assert h2 is h
        outs.append(o)
    for t in range(290, 300):
        outs.append(gdn.decay_attn_step(*(c[n][:, t] for n in ("q", "k", "v")), c["g"][:, t].contiguous(), h)[:, None])
    torch.cuda.synchronize()
    layer_ref.check(torch.cat(outs, 1), want["o"], err["o"], "o")
    layer_ref.check(h, want["ht"], err["ht"], "state")


def test_same_bits_streams_and_graphs(gpu_lib, monkeypatch):
    gdn = gpu_lib
    cu = offsets((700, 0, 300, 20)).cuda()
    c = cuda(inputs(13, 1, 1020, 2, 4, 128, 64, "bf16", N=4))

    def call(stream=None):
        kw = dict(h0=c["h0"], cu_seqlens=cu, stream=stream)
        o, ht = gdn.decay_attn_fwd(c["q"], c["k"], c["v"], c["g"], **kw)
        st = c["h0"][:1].clone() if stream is None else None
        b = gdn.decay_attn_bwd(c["q"], c["k"], c["v"], c["g"], c["do"], dht=c["dht"], **kw)
        if st is not None:
            b["step"] = gdn.decay_attn_step(c["q"][:, 0], c["k"][:, 0], c["v"][:, 0], c["g"][:, 0].contiguous(), st)
            b["st"] = st
        return dict(b, o=o, ht=ht)
    first = call()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    again, other = call(s), call()               # two at once, workspaces of their own
    torch.cuda.synchronize()
    assert all(torch.equal(first[n], again[n]) for n in again)
    assert all(torch.equal(first[n], other[n]) for n in first)
    monkeypatch.setenv("GDN_DEBUG", "0")         # reading the check of the offsets would wait inside the capture
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = call()
    q0 = c["q"].clone()
    for k in range(3):
        c["q"].copy_(q0 * (1 + k))
        want = call()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(want[n], out[n]) for n in want), k


def test_supplied_outputs_and_workspace(gpu_lib):
    gdn = gpu_lib
    c = cuda(inputs(14, 1, 600, 1, 2, 64, 64, "bf16"))
    args = [c[n] for n in ("q", "k", "v", "g")]
    o, ht = gdn.decay_attn_fwd(*args, h0=c["h0"])
    b = gdn.decay_attn_bwd(*args, c["do"], h0=c["h0"], dht=c["dht"])
    ws = torch.full((1 << 24,), 255, dtype=torch.uint8, device="cuda")      # NaNs
    o2, ht2 = torch.full_like(o, float("nan")), torch.full_like(ht, float("nan"))
    gdn.decay_attn_fwd(*args, h0=c["h0"], o=o2, ht=ht2, workspace=ws)
    into = {n: torch.full_like(t, float("nan")) for n, t in b.items()}
    b2 = gdn.decay_attn_bwd(*args, c["do"], h0=c["h0"], dht=c["dht"], out=into, workspace=ws)
    assert all(b2[n] is into[n] for n in b)
    torch.cuda.synchronize()
    assert torch.equal(o, o2) and torch.equal(ht, ht2) and all(torch.equal(b[n], b2[n]) for n in b)
    o3, none = gdn.decay_attn_fwd(*args, h0=c["h0"], output_final_state=False)
    b3 = gdn.decay_attn_bwd(*args, c["do"], h0=c["h0"], dht=c["dht"], want_dh0=False)
    assert none is None and b3["dh0"] is None and torch.equal(o3, o) and torch.equal(b3["dg"], b["dg"])


def test_long_sequence(gpu_lib):
    """Many segments: two heads' outputs of 20000 tokens against the 64-bit sums over pairs of the last
    2000 tokens (what lies before is decayed by exp(-40) at least)."""
    gdn = gpu_lib
    d = inputs(15, 1, 20000, 2, 2, 64, 64, "f32", gate=0.0)
    d["g"] = -0.02 - 0.01 * torch.rand(1, 20000, 2, generator=torch.Generator().manual_seed(2))
    c = cuda(d)
    o, ht = gdn.decay_attn_fwd(c["q"], c["k"], c["v"], c["g"], h0=c["h0"])
    b = gdn.decay_attn_bwd(c["q"], c["k"], c["v"], c["g"], c["do"], h0=c["h0"], dht=c["dht"])
    torch.cuda.synchronize()
    tail = {n: d[n][:, -4000:] for n in ("q", "k", "v", "g", "do")}
    want, err = ref.decay(tail["q"], tail["k"], tail["v"], tail["g"], None, None, None, tail["do"], d["dht"])
    far = 1e-14          # exp(-40) times what 16000 tokens add up to
    for n, t in dict(o=o, dq=b["dq"], dk=b["dk"], dv=b["dv"], dg=b["dg"]).items():
        layer_ref.check(t[:, -1900:], want[n][:, -1900:], err[n][:, -1900:] + far, n)
    layer_ref.check(ht, want["ht"], err["ht"] + far, "ht")


def test_bad_offsets_are_reported(gpu_lib):
    gdn = gpu_lib
    c = cuda(inputs(16, 1, 600, 1, 1, 64, 64, "bf16", N=2))
    for cu in ([0, 700, 600], [1, 5, 600], [0, 300, 500], [0, -5, 600], [300, 0, 600]):
        with pytest.raises(gdn.GdnError) as e:
            gdn.decay_attn_fwd(c["q"], c["k"], c["v"], c["g"], cu_seqlens=torch.tensor(cu, device="cuda"))
        assert e.value.status == 8
        with pytest.raises(gdn.GdnError) as e:
            gdn.decay_attn_bwd(c["q"], c["k"], c["v"], c["g"], c["do"], cu_seqlens=torch.tensor(cu, device="cuda"))
        assert e.value.status == 8


def test_refusals(gpu_lib):
    gdn = gpu_lib
    c = cuda(inputs(17, 2, 8, 1, 2, 64, 64, "bf16"))
    q, k, v, g, do, h = (c[n] for n in ("q", "k", "v", "g", "do", "h0"))
    cu = torch.tensor([0, 8], device="cuda")
    bad = [lambda: gdn.decay_attn_fwd(q[0], k, v, g), lambda: gdn.decay_attn_fwd(q, k[:, :4], v, g),
           lambda: gdn.decay_attn_fwd(q, k.float(), v, g), lambda: gdn.decay_attn_fwd(q.half(), k.half(), v.half(), g),
           lambda: gdn.decay_attn_fwd(q, k, v[:1], g), lambda: gdn.decay_attn_fwd(q, k, v, g.bfloat16()),
           lambda: gdn.decay_attn_fwd(q, k, v, g[:, :, :1]), lambda: gdn.decay_attn_fwd(q, k, v, g, h0=h[:1]),
           lambda: gdn.decay_attn_fwd(q, k, v, g, h0=h.bfloat16()), lambda: gdn.decay_attn_fwd(q, k, v, g, cu_seqlens=cu.int()),
           lambda: gdn.decay_attn_fwd(q, k, v, g, o=do.float()), lambda: gdn.decay_attn_fwd(q, k, v, g.cpu()),
           lambda: gdn.decay_attn_fwd(q.expand(2, 8, 1, 64)[:, :, :, ::2], k[..., ::2], v, g),
           lambda: gdn.decay_attn_bwd(q, k, v, g, do[:, :4]), lambda: gdn.decay_attn_bwd(q, k, v, g, do, dht=h[0]),
           lambda: gdn.decay_attn_bwd(q, k, v, g, do, out=dict(dq=do)),
           lambda: gdn.decay_attn_step(q[:, 0], k[:, 0], v[:, 0], g[:, 0].contiguous(), h[:1]),
           lambda: gdn.decay_attn_step(q, k, v, g, h), lambda: gdn.decay_attn_step(q[:, 0], k[:, 0], v[:, 0], g[0, 0], h.cpu()),
           lambda: gdn.decay_attn_step(q[:, 0], k[:, 0], v[:, 0], g[0, 0], None)]
    for i, f in enumerate(bad):
        with pytest.raises((ValueError, TypeError)):
            f()
            print("accepted", i, flush=True)
    wide = torch.zeros(2, 8, 1, 66, dtype=torch.bfloat16, device="cuda")
    three = torch.zeros(2, 8, 3, 64, dtype=torch.bfloat16, device="cuda")
    for f, code in ((lambda: gdn.decay_attn_fwd(q[..., :32].contiguous(), k[..., :32].contiguous(), v, g), 4),
                    (lambda: gdn.decay_attn_fwd(q, k, v, g, cu_seqlens=cu), 2),
                    (lambda: gdn.decay_attn_fwd(wide[..., :64], k, v, g), 6),
                    (lambda: gdn.decay_attn_fwd(torch.cat([q, q], 2), torch.cat([k, k], 2), three,
                                                torch.zeros(2, 8, 3, device="cuda")), 2),
                    (lambda: gdn.decay_attn_bwd(q, k, v, g, do, workspace=torch.zeros(256, dtype=torch.uint8, device="cuda")), 5)):
        with pytest.raises(gdn.GdnError) as e:
            f()
        assert e.value.status == code, e.value


def test_no_sequences_step(gpu_lib):
    z = lambda *s: torch.zeros(*s, device="cuda")  # noqa: E731
    assert gpu_lib.decay_attn_step(z(0, 1, 64), z(0, 1, 64), z(0, 2, 64), z(0, 2), z(0, 2, 64, 64)).shape == (0, 2, 64)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("T,at", [(50, 30), (300, 290), (700, 200)])
def test_values_that_are_not_finite(gpu_lib, dt, bad, T, at):
    """A value that is not finite, in one head of one sequence, reaches what sees it and nothing else."""
    gdn = gpu_lib
    d = inputs(11, 2, T, 2, 2, 64, 128, dt)
    want, err = ref.decay(d["q"], d["k"], d["v"], d["g"], None, d["h0"], None, d["do"], d["dht"])
    for name in ("q", "k", "v", "do"):
        x = dict(d, **{name: d[name].clone()})
        x[name][1, at, 1, 7] = bad
        c = {n: t.cuda() if torch.is_tensor(t) else t for n, t in x.items()}
        o, ht = gdn.decay_attn_fwd(c["q"], c["k"], c["v"], c["g"], h0=c["h0"])
        b = gdn.decay_attn_bwd(c["q"], c["k"], c["v"], c["g"], c["do"], h0=c["h0"], dht=c["dht"])
        torch.cuda.synchronize()
        got = dict(b, o=o, ht=ht)
        for n in want:                     # the other sequence and the other head
            for part in ((0, slice(None)), (1, slice(None), 0) if n[0] in "od" and n != "dh0" else (1, 0)):
                layer_ref.check(got[n][part], want[n][part], err[n][part], "%s of bad %s" % (n, name))
        before, after = (1, slice(0, at), 1), (1, slice(at + 1, T), 1)
        clean = dict(q=[("o", before), ("o", after), ("dq", before), ("dq", after), ("dk", after), ("dv", after)],
                     k=[("o", before), ("dq", before), ("dk", before), ("dk", after), ("dv", before), ("dv", after)],
                     v=[("o", before), ("dq", before), ("dk", before), ("dk", after), ("dv", before), ("dv", after)],
                     do=[("o", (1, slice(None), 1)), ("dq", before), ("dq", after), ("dk", after), ("dv", after)])[name]
        for n, part in clean:
            layer_ref.check(got[n][part], want[n][part], err[n][part], "%s of bad %s" % (n, name))
        seen = dict(q=[("o", (1, at, 1)), ("dv", (1, slice(0, at + 1), 1))], k=[("o", (1, at, 1)), ("ht", (1, 1, 7))],
                    v=[("o", (1, slice(at, T), 1, 7)), ("ht", (1, 1, slice(None), 7))],
                    do=[("dq", (1, at, 1)), ("dv", (1, slice(0, at + 1), 1, 7))])[name]
        for n, part in seen:
            assert not bool(torch.isfinite(got[n][part]).any()), (n, name)


@pytest.mark.parametrize("T", [500, 1000, 2500])
def test_state_carried_in_place(gpu_lib, T):
    """ht in h0's place: the bits of a call with its own, of sequences of a few segments and of many."""
    gdn = gpu_lib
    c = cuda(inputs(12, 2, T, 2, 2, 64, 128))
    o, ht = gdn.decay_attn_fwd(c["q"], c["k"], c["v"], c["g"], h0=c["h0"])
    h = c["h0"].clone()
    o2, _ = gdn.decay_attn_fwd(c["q"], c["k"], c["v"], c["g"], h0=h, ht=h)
    torch.cuda.synchronize()
    assert torch.equal(o, o2) and torch.equal(ht, h)


@pytest.mark.parametrize("lengths", [(0,), (0, 5, 0), (3,) * 600, (700, 0, 40)])
def test_gate_per_head_over_sequences(gpu_lib, lengths):
    """dg of a gate for each head sums over all tokens: none, few, many sequences, segments."""
    d = inputs(13, 1, sum(lengths), 1, 2, 64, 64, "f32", N=len(lengths), per_head=True)
    both(gpu_lib, d, offsets(lengths))
