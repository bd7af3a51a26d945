"""Short causal convolution on the GPU against the 64-bit definition."""
import pytest
import torch

import layer_ref as ref

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


def inputs(seed, B, T, D, W, dt=BF, N=None, pad=0):
    r = torch.Generator().manual_seed(seed)
    N = B if N is None else N

    def rows(t):
        wide = torch.full((B, T, D + pad), float("nan"), dtype=dt)
        wide[..., pad // 2:pad // 2 + D] = t.to(dt)
        return wide.cuda()[..., pad // 2:pad // 2 + D]
    return dict(x=rows(torch.randn(B, T, D, generator=r)), dy=rows(torch.randn(B, T, D, generator=r)),
                w=(torch.randn(D, W, generator=r) * W ** -0.5).cuda(), b=torch.randn(D, generator=r).cuda(),
                s0=torch.randn(N, W - 1, D, generator=r).to(dt).cuda(),
                dst=torch.randn(N, W - 1, D, generator=r).to(dt).cuda())


def both(gdn, d, cu=None, silu=True, bias=True, s0=True, dst=True):
    dev = None if cu is None else cu.cuda()
    kw = dict(bias=d["b"] if bias else None, s0=d["s0"] if s0 else None, cu_seqlens=dev, silu=silu)
    y, st = gdn.short_conv_fwd(d["x"], d["w"], output_final_state=True, **kw)
    got = gdn.short_conv_bwd(d["x"], d["w"], d["dy"], dst=d["dst"] if dst else None, **kw)
    torch.cuda.synchronize()
    got.update(y=y, st=st)
    want, err = ref.conv(d["x"], d["w"], kw["bias"], kw["s0"], cu, silu, d["dy"], d["dst"] if dst else None)
    ref.check_all(got, want, err)
    assert "dbias" in got or not bias
    return got


@pytest.mark.parametrize("T", [1, 2, 3, 4, 5, 15, 16, 17, 63, 64, 65, 128, 200])
@pytest.mark.parametrize("W", [2, 3, 4])
def test_lengths(gpu_lib, T, W):
    print("case: conv", T, W, flush=True)
    both(gpu_lib, inputs(T + W, 2, T, 72, W))
    both(gpu_lib, inputs(T + W, 1, T, 9, W, F32), silu=False, bias=False)


@pytest.mark.parametrize("D", [1, 7, 63, 64, 65, 128, 520, 1030])
@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("silu", [False, True])
def test_channels(gpu_lib, D, dt, silu):
    print("case: conv channels", D, dt, silu, flush=True)
    both(gpu_lib, inputs(D, 2, 70, D, 4, dt), silu=silu, bias=silu)
    both(gpu_lib, inputs(D, 1, 33, D, 3, dt), silu=silu, s0=False, dst=False)


@pytest.mark.parametrize("lengths", [(5,), (0, 3, 0), (64, 64), (1, 1, 1, 1, 2, 2), (0, 0), (300, 0, 129, 64, 1, 3, 65)])
@pytest.mark.parametrize("W", [2, 3, 4])
def test_packed(gpu_lib, lengths, W):
    print("case: conv packed", lengths, W, flush=True)
    T, N = sum(lengths), len(lengths)
    cu = torch.tensor([sum(lengths[:i]) for i in range(N + 1)])
    d = inputs(11, 1, T, 66, W, N=N)
    both(gpu_lib, d, cu)
    both(gpu_lib, d, cu, s0=False, dst=False, bias=False)


def test_many_short_sequences(gpu_lib):
    r = torch.Generator().manual_seed(2)
    n = torch.randint(0, 6, (2100,), generator=r)
    cu = torch.cat([torch.zeros(1, dtype=torch.int64), n.cumsum(0)])
    print("case: conv many", int(cu[-1]), flush=True)
    both(gpu_lib, inputs(12, 1, int(cu[-1]), 16, 4, N=2100), cu)


@pytest.mark.parametrize("pad", [2, 8, 13])
def test_strided_rows(gpu_lib, pad):
    d = inputs(15, 2, 140, 64, 4, pad=pad)
    both(gpu_lib, d)
    wide = torch.full((2, 140, 64 + pad), 7.0, dtype=BF, device="cuda")
    y, st = gpu_lib.short_conv_fwd(d["x"], d["w"], y=wide[..., :64])
    plain, _ = gpu_lib.short_conv_fwd(d["x"].contiguous(), d["w"])
    torch.cuda.synchronize()
    assert st is None and y.data_ptr() == wide.data_ptr() and torch.equal(wide[..., :64], plain)
    assert (wide[..., 64:] == 7).all()


@pytest.mark.parametrize("W", [2, 3, 4])
@pytest.mark.parametrize("dt", [BF, F32])
def test_step_continues_prefill(gpu_lib, W, dt):
    gdn = gpu_lib
    for D, N in ((77, 3), (512, 1), (64, 40)):
        d = inputs(16, N, 20, D, W, dt)
        want, err = ref.conv(d["x"], d["w"], d["b"], d["s0"])
        _, st = gdn.short_conv_fwd(d["x"][:, :2].contiguous(), d["w"], d["b"], d["s0"], output_final_state=True)
        for t in range(2, 20):
            y = gdn.short_conv_step(d["x"][:, t], d["w"], st, d["b"])
            ref.check(y, want["y"][:, t], err["y"][:, t], "step %d" % t)
        assert torch.equal(st.cpu().double(), want["st"])
    e = torch.empty(0, 8, device="cuda")
    assert gdn.short_conv_step(e, torch.zeros(8, W, device="cuda"), torch.empty(0, W - 1, 8, device="cuda")).shape == (0, 8)


def test_no_tokens(gpu_lib):
    d = inputs(17, 2, 0, 24, 4)
    got = both(gpu_lib, d)
    assert torch.equal(got["st"], d["s0"]) and torch.equal(got["ds0"], d["dst"])
    assert (got["dweight"] == 0).all() and (got["dbias"] == 0).all()


def test_extremes(gpu_lib):
    """Pre-activations far out: silu and its slope have no NaN where the definition has none."""
    for sign in (1.0, -1.0):
        d = inputs(18, 1, 40, 16, 4, F32)
        d["b"].fill_(sign * 200.0)
        got = both(gpu_lib, d)
        assert all(torch.isfinite(t).all() for t in got.values())


def test_non_finite_stays_in_its_channel_and_sequence(gpu_lib):
    gdn = gpu_lib
    cu = torch.tensor([0, 70, 150, 200], device="cuda")
    d = inputs(19, 1, 200, 64, 4, N=3)
    y0, st0 = gdn.short_conv_fwd(d["x"], d["w"], d["b"], d["s0"], cu, output_final_state=True)
    b0 = gdn.short_conv_bwd(d["x"], d["w"], d["dy"], d["b"], d["s0"], d["dst"], cu)
    x, dy = d["x"].clone(), d["dy"].clone()
    x[0, 69, 3], dy[0, 70, 4], dy[0, 100, 5] = float("nan"), float("nan"), float("inf")
    y, st = gdn.short_conv_fwd(x, d["w"], d["b"], d["s0"], cu, output_final_state=True)
    b = gdn.short_conv_bwd(d["x"], d["w"], dy, d["b"], d["s0"], d["dst"], cu)
    torch.cuda.synchronize()
    m = torch.zeros_like(y, dtype=torch.bool)
    m[0, 69, 3] = True
    assert torch.equal(y[~m], y0[~m]) and torch.isnan(y[0, 69, 3]) and torch.equal(st[1:], st0[1:])
    m = torch.zeros_like(y, dtype=torch.bool)
    m[0, 70, 4], m[0, 97:101, 5] = True, True
    assert torch.equal(b["dx"][~m], b0["dx"][~m])
    assert torch.equal(b["dweight"][:3], b0["dweight"][:3]) and torch.equal(b["ds0"][0], b0["ds0"][0])


def test_same_bits_streams_and_graphs(gpu_lib, monkeypatch):
    gdn = gpu_lib
    cu = torch.tensor([0, 700, 700, 1500], device="cuda")
    d = inputs(20, 1, 1500, 136, 4, N=3)

    def call(stream=None):
        y, st = gdn.short_conv_fwd(d["x"], d["w"], d["b"], d["s0"], cu, output_final_state=True, stream=stream)
        return dict(gdn.short_conv_bwd(d["x"], d["w"], d["dy"], d["b"], d["s0"], d["dst"], cu, stream=stream), y=y, st=st)
    first = call()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    again = call(s)
    s.synchronize()
    assert all(torch.equal(first[n], again[n]) for n in first)
    monkeypatch.setenv("GDN_DEBUG", "0")     # reading the check of the offsets would wait inside the capture
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = call()
    x0 = d["x"].clone()
    for k in range(3):
        d["x"].copy_(x0 * (1 + k))
        want = call()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(want[n], out[n]) for n in want), k


def test_refusals(gpu_lib):
    gdn = gpu_lib
    x, w = torch.zeros(2, 8, 16, device="cuda"), torch.zeros(16, 4, device="cuda")
    s, cu = torch.zeros(2, 3, 16, device="cuda"), torch.tensor([0, 8], device="cuda")
    bad = [lambda: gdn.short_conv_fwd(x[0], w), lambda: gdn.short_conv_fwd(x, w[:8]), lambda: gdn.short_conv_fwd(x, w[0]),
           lambda: gdn.short_conv_fwd(x, w.bfloat16()), lambda: gdn.short_conv_fwd(x.half(), w),
           lambda: gdn.short_conv_fwd(x, w, bias=w[0]), lambda: gdn.short_conv_fwd(x, w, s0=s[:, :2]),
           lambda: gdn.short_conv_fwd(x, w, s0=s.bfloat16()), lambda: gdn.short_conv_fwd(x.transpose(1, 2), torch.zeros(8, 4, device="cuda")),
           lambda: gdn.short_conv_fwd(x, w, cu_seqlens=cu.int()), lambda: gdn.short_conv_fwd(x, w, y=x[:1]),
           lambda: gdn.short_conv_bwd(x, w, x[:, :4]), lambda: gdn.short_conv_bwd(x, w, x, dst=s[:1]),
           lambda: gdn.short_conv_step(x[:, 0], w, s[:, :2]), lambda: gdn.short_conv_step(x, w, s),
           lambda: gdn.short_conv_step(x[:, 0], w, s.cpu())]
    for i, f in enumerate(bad):
        with pytest.raises((ValueError, TypeError)):
            f()
            print("accepted", i, flush=True)
    for f, code in ((lambda: gdn.short_conv_fwd(x, torch.zeros(16, 5, device="cuda")), 4),
                    (lambda: gdn.short_conv_fwd(x, w, cu_seqlens=cu), 2),
                    (lambda: gdn.short_conv_fwd(x, w, s0=s, st=s, output_final_state=True), 4)):
        with pytest.raises(gdn.GdnError) as e:
            f()
        assert e.value.status == code


def test_offsets_check(gpu_lib):
    gdn = gpu_lib
    d = inputs(24, 1, 300, 16, 4, N=3)
    for cu in ([0, 200, 100, 300], [10, 100, 200, 300], [0, 100, 200, 290], [0, 100, 200, 1 << 40], [-5, 1, 2, 300]):
        cu = torch.tensor(cu, device="cuda")
        for f in (lambda: gdn.short_conv_fwd(d["x"], d["w"], cu_seqlens=cu),
                  lambda: gdn.short_conv_bwd(d["x"], d["w"], d["dy"], cu_seqlens=cu)):
            with pytest.raises(gdn.GdnError) as e:
                f()
            assert e.value.status == 8
