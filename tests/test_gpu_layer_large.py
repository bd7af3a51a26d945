"""The layer operators where element offsets pass 32 bits, and two calls at
once.  A tensor of repeated 64-channel columns has to give the columns' own
result everywhere, bit for bit: every channel is computed alike whatever
their number."""
import pytest
import torch

pytestmark = pytest.mark.gpu
BF = torch.bfloat16
T, R = 540000, 64          # 540000 x 64 x 64 elements: above 2^31


def wide(t):
    return t.repeat(1, 1, R)


def same(big, small):
    """big [1, T, 64 R] equals small [1, T, 64] in every column."""
    for a in range(0, big.shape[1], 65536):
        assert torch.equal(big[:, a:a + 65536], small[:, a:a + 65536].repeat(1, 1, R)), a


@pytest.fixture(scope="module")
def columns():
    g = torch.Generator(device="cuda").manual_seed(1)
    return [torch.randn(1, T, 64, device="cuda", generator=g).to(BF) for _ in range(3)]


def test_linrec_offsets_past_32_bits(gpu_lib, columns):
    x, g, dy = columns
    g = -torch.nn.functional.softplus(g.float()).to(BF)
    cu = torch.tensor([0, 3, 400000, T], device="cuda")
    print("case: linrec", T, 64 * R, flush=True)
    want = gpu_lib.linrec_fwd(x, g, cu_seqlens=cu)
    X, G = wide(x), wide(g)
    assert X.numel() > 1 << 31
    keep = gpu_lib.linrec_states(X, cu)
    y, ht = gpu_lib.linrec_fwd(X, G, cu_seqlens=cu, states=keep)
    same(y, want[0])
    assert torch.equal(ht, want[1].repeat(1, R))
    del y
    back = gpu_lib.linrec_bwd(x, g, dy, cu_seqlens=cu)
    got = gpu_lib.linrec_bwd(X, G, wide(dy), cu_seqlens=cu, states=keep)
    same(got["dx"], back["dx"])
    same(got["dg"], back["dg"])
    assert torch.equal(got["dh0"], back["dh0"].repeat(1, R))


def test_conv_offsets_past_32_bits(gpu_lib, columns):
    x, _, dy = columns
    cu = torch.tensor([0, 3, 400000, T], device="cuda")
    w = torch.randn(64, 4, device="cuda", generator=torch.Generator(device="cuda").manual_seed(2))
    print("case: conv", T, 64 * R, flush=True)
    want = gpu_lib.short_conv_fwd(x, w, cu_seqlens=cu, output_final_state=True)
    X, W = wide(x), w.repeat(R, 1)
    y, st = gpu_lib.short_conv_fwd(X, W, cu_seqlens=cu, output_final_state=True)
    same(y, want[0])
    assert torch.equal(st, want[1].repeat(1, 1, R))
    del y
    back = gpu_lib.short_conv_bwd(x, w, dy, cu_seqlens=cu)
    got = gpu_lib.short_conv_bwd(X, W, wide(dy), cu_seqlens=cu)
    same(got["dx"], back["dx"])
    assert torch.equal(got["dweight"], back["dweight"].repeat(R, 1))
    assert torch.equal(got["ds0"], back["ds0"].repeat(1, 1, R))


def test_qk_offsets_past_32_bits(gpu_lib, columns):
    x, y, _ = columns
    print("case: qk", T, 64, 64, flush=True)
    q = wide(x).view(1, T, R, 64)
    k = y.view(1, T, 1, 64)
    f = 10000.0 ** (-torch.arange(0, 64, 2, device="cuda", dtype=torch.float64) / 64)
    w = torch.linspace(0.5, 1.5, 64, device="cuda")
    qo, ko = gpu_lib.qk_norm_rope(q, k, f, q_weight=w)
    one, k1 = gpu_lib.qk_norm_rope(x.view(1, T, 1, 64), k, f, q_weight=w)
    same(qo.flatten(2), one.flatten(2))
    assert torch.equal(ko, k1)
    got = gpu_lib.qk_norm_rope_bwd(q, k, qo, ko, f, q_weight=w)
    ref = gpu_lib.qk_norm_rope_bwd(x.view(1, T, 1, 64), k, one, ko, f, q_weight=w)
    same(got["dq"].flatten(2), ref["dq"].flatten(2))
    assert torch.equal(got["dk"], ref["dk"])


def test_two_calls_at_once(gpu_lib):
    """Calls on two streams, each with what it allocates: the results of calls in turn."""
    gdn = gpu_lib
    d = [[torch.randn(2, 3000, 192, device="cuda", generator=torch.Generator(device="cuda").manual_seed(s + i))
          for i in range(3)] for s in (10, 20)]
    for t in d:
        t[1] = -t[1].abs()

    def call(t, stream=None):
        y, ht = gdn.linrec_fwd(t[0], t[1], stream=stream)
        b = gdn.linrec_bwd(t[0], t[1], t[2], dht=ht, stream=stream)
        return y, ht, b["dx"], b["dg"], b["dh0"]
    want = [call(t) for t in d]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [[call(t, s) for t, s in zip(d, streams)] for _ in range(4)]
    torch.cuda.synchronize()
    for r in got:
        for a, b in zip(r, want):
            assert all(torch.equal(u, v) for u, v in zip(a, b))


def test_many_single_tokens(gpu_lib):
    """More sequences of one token than a launch has tiles of a whole workgroup."""
    N, D = 70000, 4096
    x = torch.randn(N, 1, D, device="cuda", dtype=torch.bfloat16)
    g = torch.full((N, 1, D), -0.5, device="cuda")
    h0 = torch.randn(N, D, device="cuda")
    print("case: linrec", N, 1, D, flush=True)
    y, ht = gpu_lib.linrec_fwd(x, g, h0=h0)
    out = gpu_lib.linrec_bwd(x, g, x, h0=h0, dht=h0)
    step = h0.clone()
    gpu_lib.linrec_step(x[:, 0], g[:, 0], step)
    torch.cuda.synchronize()
    assert torch.equal(ht, step)                    # the same product and sum, rounded once each or fused in both
    for n in (0, N // 2, N - 1):
        a, h, v = torch.exp(torch.tensor(-0.5, dtype=torch.float64)), h0[n].double().cpu(), x[n, 0].double().cpu()
        want = a * h + v
        # two products or sums of 2^-23 and an a off by a few of them, then the output's half step
        tol = 2.0 ** -20 * (a * h).abs() + 2.0 ** -22 * want.abs() + 1e-30
        assert ((ht[n].double().cpu() - want).abs() <= tol).all()
        assert ((y[n, 0].double().cpu() - want).abs() <= tol + 2.0 ** -8 * want.abs()).all()
        dh = v + h
        assert ((out["dh0"][n].double().cpu() - a * dh).abs() <= 2.0 ** -20 * (v.abs() + h.abs())).all()
