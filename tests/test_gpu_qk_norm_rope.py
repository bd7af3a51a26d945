"""Per-head norm of q and k with the rotation on the GPU against the 64-bit definition."""
import pytest
import torch

import layer_ref as ref

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


def inputs(seed, B, T, Hq, Hk, D, dt=BF, gap=False, weights=True, far=0):
    r = torch.Generator().manual_seed(seed)
    q, k = torch.randn(B, T, Hq, 2 * D if gap else D, generator=r), torch.randn(B, T, Hk * (2 if gap else 1), D, generator=r)
    q, k = q.to(dt).cuda(), k.to(dt).cuda()
    if gap:
        q, k = q[..., :D], k[:, :, :Hk]
    d = dict(q=q, k=k, dq=torch.randn(B, T, Hq, D, generator=r).to(dt).cuda(),
             dk=torch.randn(B, T, Hk, D, generator=r).to(dt).cuda(),
             positions=torch.randint(0, far, (B, T), generator=r).cuda() if far else None)
    d["qw"], d["kw"] = ((1 + 0.2 * torch.randn(D, generator=r)).cuda() for _ in range(2)) if weights else (None, None)
    return d


def freqs(R):
    return (10000.0 ** (-torch.arange(0, R, 2, dtype=torch.float64) / R)).cuda() if R else None


def both(gdn, d, R, norm="rms", eps=1e-6, offset=0.0, inter=False):
    f = freqs(R)
    kw = dict(positions=d["positions"], norm=norm, eps=eps, q_weight=d["qw"], k_weight=d["kw"], weight_offset=offset,
              interleaved=inter)
    qo, ko = gdn.qk_norm_rope(d["q"], d["k"], f, **kw)
    got = gdn.qk_norm_rope_bwd(d["q"], d["k"], d["dq"], d["dk"], f, **kw)
    torch.cuda.synchronize()
    for name, out, t, w, do in (("q", qo, d["q"], d["qw"], d["dq"]), ("k", ko, d["k"], d["kw"], d["dk"])):
        want, err = ref.qk(t, f, d["positions"], norm, eps, w, offset, inter, do)
        ref.check(out, want["out"], err["out"], name)
        ref.check(got["d" + name], want["dx"], err["dx"], "d" + name)
        if w is not None:
            ref.check(got["d%s_weight" % name], want["dw"], err["dw"], "d%s_weight" % name)
        else:
            assert "d%s_weight" % name not in got
    return qo, ko, got


@pytest.mark.parametrize("norm", ["none", "l2", "rms"])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("dt", [BF, F32])
def test_norms_and_pairs(gpu_lib, norm, inter, dt):
    print("case: qk", norm, inter, dt, flush=True)
    both(gpu_lib, inputs(1, 2, 9, 4, 2, 128, dt, far=5000), 128, norm, inter=inter)
    both(gpu_lib, inputs(2, 1, 5, 3, 5, 64, dt, weights=False), 32, norm, inter=inter)


@pytest.mark.parametrize("D,R", [(8, 0), (16, 16), (24, 16), (64, 64), (72, 48), (80, 80), (96, 32), (128, 0),
                                 (128, 16), (192, 128), (256, 64), (256, 256), (248, 240)])
@pytest.mark.parametrize("inter", [False, True])
def test_sizes(gpu_lib, D, R, inter):
    print("case: qk sizes", D, R, inter, flush=True)
    both(gpu_lib, inputs(D + R, 2, 7, 3, 2, D, BF, gap=True, far=1000), R, "rms", offset=1.0, inter=inter)
    both(gpu_lib, inputs(D + R, 1, 4, 1, 1, D, F32, far=1000), R, "l2", inter=inter)


@pytest.mark.parametrize("B,T", [(1, 1), (64, 1), (1, 63), (3, 129), (2, 1000)])
@pytest.mark.parametrize("Hq,Hk", [(1, 1), (16, 2), (5, 3), (40, 8)])
def test_tokens_and_heads(gpu_lib, B, T, Hq, Hk):
    if B * T * Hq > 20000:
        T //= 4
    print("case: qk tokens", B, T, Hq, Hk, flush=True)
    both(gpu_lib, inputs(B + T + Hq, B, T, Hq, Hk, 64, BF, gap=T % 2 == 1, far=100000), 64)


def test_far_positions(gpu_lib):
    """Angles keep their accuracy far out and for negative positions."""
    d = inputs(5, 1, 6, 2, 2, 64, F32, weights=False)
    d["positions"] = torch.tensor([[0, -1, 1000003, (1 << 31) - 1, -(1 << 30), 123456789]], device="cuda")
    # a position p times a frequency is off by p 2^-53 in 64 bits, under 2^-22 here: 4 U more
    q, k = gpu_lib.qk_norm_rope(d["q"], d["k"], freqs(64), d["positions"], norm="none")
    want, err = ref.qk(d["q"], freqs(64), d["positions"], "none", 0.0, None, 0.0, False)
    ref.check(q, want["out"], 2 * err["out"], "q")


def test_zero_rows_and_large_values(gpu_lib):
    d = inputs(6, 1, 4, 2, 2, 128, F32)
    d["q"][0, 0] = 0
    d["k"][0, 1] = 0
    d["q"][0, 2] *= 1e15
    d["k"][0, 3] *= 1e-15
    for norm in ("l2", "rms"):
        qo, ko, got = both(gpu_lib, d, 64, norm)
        assert all(torch.isfinite(t).all() for t in (qo, ko, *got.values()))


def test_non_finite_stays_in_its_row(gpu_lib):
    d = inputs(7, 1, 6, 4, 2, 64)
    q0, k0 = gpu_lib.qk_norm_rope(d["q"], d["k"], freqs(64))
    d["q"][0, 2, 1, 5], d["k"][0, 3, 0, 60] = float("nan"), float("inf")
    q, k = gpu_lib.qk_norm_rope(d["q"], d["k"], freqs(64))
    torch.cuda.synchronize()
    mq, mk = torch.ones_like(q, dtype=torch.bool), torch.ones_like(k, dtype=torch.bool)
    mq[0, 2, 1], mk[0, 3, 0] = False, False
    assert torch.equal(q[mq], q0[mq]) and torch.equal(k[mk], k0[mk]) and torch.isnan(q[0, 2, 1]).all()


def test_no_tokens(gpu_lib):
    q, k = torch.empty(2, 0, 4, 64, device="cuda"), torch.empty(2, 0, 2, 64, device="cuda")
    w = torch.ones(64, device="cuda")
    qo, ko = gpu_lib.qk_norm_rope(q, k, freqs(64))
    got = gpu_lib.qk_norm_rope_bwd(q, k, q, k, freqs(64), q_weight=w, k_weight=w)
    torch.cuda.synchronize()
    assert qo.shape == q.shape and ko.shape == k.shape and got["dq"].shape == q.shape
    assert (got["dq_weight"] == 0).all() and (got["dk_weight"] == 0).all()


def test_one_weight(gpu_lib):
    d = inputs(8, 1, 20, 4, 2, 64)
    d["kw"] = None
    both(gpu_lib, d, 32)
    d = inputs(9, 1, 20, 4, 2, 64)
    d["qw"] = None
    both(gpu_lib, d, 32, "l2", offset=0.5)


def test_same_bits_streams_and_graphs(gpu_lib):
    d = inputs(10, 1, 1500, 8, 2, 128, BF, gap=True, far=4096)
    f, kw = freqs(128), dict(positions=d["positions"], norm="rms", q_weight=d["qw"], k_weight=d["kw"])

    def call(stream=None):
        q, k = gpu_lib.qk_norm_rope(d["q"], d["k"], f, stream=stream, **kw)
        return dict(gpu_lib.qk_norm_rope_bwd(d["q"], d["k"], d["dq"], d["dk"], f, stream=stream, **kw), q=q, k=k)
    first = call()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    again = call(s)
    s.synchronize()
    assert all(torch.equal(first[n], again[n]) for n in first)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = call()
    q0 = d["q"].clone()
    for i in range(3):
        d["q"].copy_(q0 * (1 + i))
        want = call()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(want[n], out[n]) for n in want), i


def test_options_are_read_at_every_call(gpu_lib):
    """eps and weight_offset as scalars that change between two calls."""
    d = inputs(61, 1, 5, 2, 2, 64)
    eps, offset = torch.tensor(1e-6), torch.tensor(0.0)
    kw = dict(norm="rms", q_weight=d["qw"])
    for e, o in ((1e-6, 0.0), (0.5, 1.0)):
        eps.fill_(e)
        offset.fill_(o)
        got = gpu_lib.qk_norm_rope(d["q"], d["k"], eps=eps, weight_offset=offset, **kw)
        want = gpu_lib.qk_norm_rope(d["q"], d["k"], eps=e, weight_offset=o, **kw)
        torch.cuda.synchronize()
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]), (e, o)


def test_refusals(gpu_lib):
    gdn = gpu_lib
    q, k, f = torch.zeros(1, 4, 4, 64, device="cuda"), torch.zeros(1, 4, 2, 64, device="cuda"), freqs(64)
    w = torch.ones(64, device="cuda")
    bad = [lambda: gdn.qk_norm_rope(q[0], k[0], f), lambda: gdn.qk_norm_rope(q, k[:, :2], f),
           lambda: gdn.qk_norm_rope(q, k[..., :32], f), lambda: gdn.qk_norm_rope(q, k.bfloat16(), f),
           lambda: gdn.qk_norm_rope(q.half(), k.half(), f), lambda: gdn.qk_norm_rope(q, k, f.float()),
           lambda: gdn.qk_norm_rope(q, k, f.cpu()), lambda: gdn.qk_norm_rope(q, k, f, norm="layer"),
           lambda: gdn.qk_norm_rope(q, k, f, positions=torch.zeros(1, 4, device="cuda", dtype=torch.int32)),
           lambda: gdn.qk_norm_rope(q, k, f, positions=torch.zeros(4, device="cuda", dtype=torch.int64)),
           lambda: gdn.qk_norm_rope(q, k, f, q_weight=w[:32]), lambda: gdn.qk_norm_rope(q, k, f, q_weight=w.bfloat16()),
           lambda: gdn.qk_norm_rope(q[..., ::2], k[..., ::2]), lambda: gdn.qk_norm_rope(q.transpose(1, 2), k.transpose(1, 2)[:, :, :2]),
           lambda: gdn.qk_norm_rope(q, k, f, q_out=k), lambda: gdn.qk_norm_rope_bwd(q, k, k, k, f),
           lambda: gdn.qk_norm_rope_bwd(q, k, q, k.bfloat16(), f)]
    for i, g in enumerate(bad):
        with pytest.raises((ValueError, TypeError)):
            g()
            print("accepted", i, flush=True)
    for kk, ff in ((dict(), freqs(80)), (dict(), freqs(24))):
        with pytest.raises(gdn.GdnError) as e:
            gdn.qk_norm_rope(q, k, ff, **kk)
        assert e.value.status == 4
    wide = torch.zeros(1, 4, 4, 68, device="cuda", dtype=BF)[..., :64]        # heads 136 bytes apart
    with pytest.raises(gdn.GdnError) as e:
        gdn.qk_norm_rope(wide, k.bfloat16(), f)
    assert e.value.status == 6
