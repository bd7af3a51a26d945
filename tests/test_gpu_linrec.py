"""Gated linear recurrence on the GPU against the 64-bit definition."""
import pytest
import torch

import layer_ref as ref

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


def inputs(seed, B, T, D, xdt=BF, gdt=F32, logits=False, N=None, pad=0):
    """x, g, h0, dy, dht, A_log, dt_bias; x, g, dy as slices of rows `pad` wider."""
    r = torch.Generator().manual_seed(seed)
    N = B if N is None else N

    def rows(dt, t):
        wide = torch.full((B, T, D + pad), float("nan"), dtype=dt)
        wide[..., pad // 2:pad // 2 + D] = t.to(dt)
        return wide.cuda()[..., pad // 2:pad // 2 + D]
    A = 1 + 15 * torch.rand(D, generator=r)
    bias = torch.log(torch.expm1(torch.exp(torch.rand(D, generator=r) * 4.6 - 6.9)))
    raw = torch.randn(B, T, D, generator=r)
    g = raw if logits else -A * torch.nn.functional.softplus(raw + bias)
    return dict(x=rows(xdt, torch.randn(B, T, D, generator=r)), g=rows(gdt, g),
                dy=rows(xdt, torch.randn(B, T, D, generator=r)), h0=torch.randn(N, D, generator=r).cuda(),
                dht=torch.randn(N, D, generator=r).cuda(), A_log=torch.log(A).cuda() if logits else None,
                dt_bias=bias.cuda() if logits else None)


def both(gdn, d, cu=None, normalize=False, h0=True, dht=True, keep=True):
    """Forward and backward against the reference."""
    kw = dict(h0=d["h0"] if h0 else None, normalize=normalize, A_log=d["A_log"], dt_bias=d["dt_bias"])
    dev = None if cu is None else cu.cuda()
    states = gdn.linrec_states(d["x"], dev) if keep else None
    y, ht = gdn.linrec_fwd(d["x"], d["g"], cu_seqlens=dev, states=states, **kw)
    got = gdn.linrec_bwd(d["x"], d["g"], d["dy"], cu_seqlens=dev, dht=d["dht"] if dht else None, states=states, **kw)
    torch.cuda.synchronize()
    got.update(y=y, ht=ht)
    want, err = ref.linrec(d["x"], d["g"], cu=cu, dy=d["dy"], dht=d["dht"] if dht else None, **kw)
    ref.check_all(got, want, err)
    return got


@pytest.mark.parametrize("T", [1, 2, 15, 16, 17, 63, 64, 65, 127, 128, 129, 257, 700])
@pytest.mark.parametrize("D", [1, 64, 130])
def test_lengths(gpu_lib, T, D):
    print("case: linrec", T, D, flush=True)
    both(gpu_lib, inputs(T + D, 2, T, D))


@pytest.mark.parametrize("xdt", [BF, F32])
@pytest.mark.parametrize("gdt", [BF, F32])
@pytest.mark.parametrize("logits", [False, True])
@pytest.mark.parametrize("normalize", [False, True])
def test_types_and_options(gpu_lib, xdt, gdt, logits, normalize):
    print("case: linrec types", xdt, gdt, logits, normalize, flush=True)
    both(gpu_lib, inputs(7, 3, 150, 72, xdt, gdt, logits), normalize=normalize)
    both(gpu_lib, inputs(8, 1, 290, 35, xdt, gdt, logits), normalize=normalize, h0=False, dht=False, keep=False)


@pytest.mark.parametrize("lengths", [(5,), (0, 3, 0), (128, 128), (1, 1, 1, 1), (0, 0), (300, 0, 129, 64, 1, 700, 65)])
@pytest.mark.parametrize("logits", [False, True])
def test_packed(gpu_lib, lengths, logits):
    print("case: linrec packed", lengths, flush=True)
    T, N = sum(lengths), len(lengths)
    cu = torch.tensor([sum(lengths[:i]) for i in range(N + 1)])
    d = inputs(11, 1, T, 66, BF, BF if logits else F32, logits, N=N)
    both(gpu_lib, d, cu, normalize=logits)
    both(gpu_lib, d, cu, h0=False, dht=False, keep=False)


def test_many_short_sequences(gpu_lib):
    """More sequences than one pass of the tile table's prefix sum."""
    r = torch.Generator().manual_seed(2)
    n = torch.randint(0, 4, (2500,), generator=r)
    cu = torch.cat([torch.zeros(1, dtype=torch.int64), n.cumsum(0)])
    print("case: linrec many", int(cu[-1]), flush=True)
    both(gpu_lib, inputs(12, 1, int(cu[-1]), 8, N=2500), cu)


@pytest.mark.parametrize("D", [8, 129, 200])
def test_short_among_long_sequences(gpu_lib, D):
    """Packed input whose mean length is short: sequences on either side of 16 and of 64 tokens."""
    for more in (0, 50):
        short_among_long(gpu_lib, D, (1, 2, 15, 16, 17, 18, 0, 63, 64, 65, 200, 16, 0, 300, 3, 16, 17, 128, 1, 1)
                         + (3,) * more)


def short_among_long(gpu_lib, D, lengths):
    T, N = sum(lengths), len(lengths)
    cu = torch.tensor([sum(lengths[:i]) for i in range(N + 1)])
    print("case: linrec short among long", T, N, D, flush=True)
    d = inputs(25, 1, T, D, BF, BF, True, N=N)
    both(gpu_lib, d, cu, normalize=True)
    both(gpu_lib, d, cu, h0=False, dht=False, keep=False)
    both(gpu_lib, inputs(26, 1, T, D, F32, F32, N=N), cu)


def test_many_tiles_among_short_sequences(gpu_lib):
    """More tiles and channel blocks in use than workgroups that take them in turn: repeated columns
    have to give the columns' own result."""
    lengths = [2] * 3000 + [2500] * 10 + [3] * 500 + [129] * 10
    T, N, R = sum(lengths), len(lengths), 16
    cu = torch.tensor([0] + lengths).cumsum(0).cuda()
    print("case: linrec tiles in turn", T, N, 64 * R, flush=True)
    d = inputs(71, 1, T, 64, BF, BF, True, N=N)

    def call(r):
        w = {k: v.repeat(*([1] * (v.dim() - 1)), r) for k, v in d.items()}
        gate = dict(h0=w["h0"], cu_seqlens=cu, normalize=True, A_log=w["A_log"], dt_bias=w["dt_bias"])
        y, ht = gpu_lib.linrec_fwd(w["x"], w["g"], **gate)
        out = gpu_lib.linrec_bwd(w["x"], w["g"], w["dy"], dht=w["dht"], **gate)
        torch.cuda.synchronize()
        return dict(out, y=y, ht=ht)
    one, many = call(1), call(R)
    for n, v in one.items():
        assert torch.equal(v.repeat(*([1] * (v.dim() - 1)), R), many[n]), n
    for i in (0, 2999, 3000, 3009, 3010, 3519):        # first and last of each kind, by the call of it alone
        a, b = int(cu[i]), int(cu[i + 1])
        y, ht = gpu_lib.linrec_fwd(d["x"][:, a:b].contiguous(), d["g"][:, a:b].contiguous(), h0=d["h0"][i:i + 1].contiguous(),
                                   normalize=True, A_log=d["A_log"], dt_bias=d["dt_bias"])
        torch.cuda.synchronize()
        assert torch.equal(y, one["y"][:, a:b]) and torch.equal(ht, one["ht"][i:i + 1]), i


def test_long_sequence(gpu_lib):
    """More tiles than one group of the look-back."""
    print("case: linrec long", flush=True)
    both(gpu_lib, inputs(13, 1, 128 * 40 + 5, 9, F32, F32))
    both(gpu_lib, inputs(14, 2, 128 * 18, 24, BF, BF, True), normalize=True, keep=False)


@pytest.mark.parametrize("pad", [2, 8, 13])
def test_strided_rows(gpu_lib, pad):
    print("case: linrec strided", pad, flush=True)
    d = inputs(15, 2, 140, 64, pad=pad)
    both(gpu_lib, d)
    wide = torch.full((2, 140, 64 + pad), 7.0, dtype=BF, device="cuda")
    y, _ = gpu_lib.linrec_fwd(d["x"], d["g"], y=wide[..., :64])
    plain, _ = gpu_lib.linrec_fwd(d["x"].contiguous(), d["g"].contiguous())
    torch.cuda.synchronize()
    assert y.data_ptr() == wide.data_ptr() and torch.equal(wide[..., :64], plain)
    assert (wide[..., 64:] == 7).all()


def test_step_continues_prefill(gpu_lib):
    gdn = gpu_lib
    for logits, normalize in ((True, True), (False, False)):
        d = inputs(16, 3, 40, 77, BF, BF if logits else F32, logits)
        kw = dict(normalize=normalize, A_log=d["A_log"], dt_bias=d["dt_bias"])
        want, err = ref.linrec(d["x"], d["g"], d["h0"], **kw)
        _, state = gdn.linrec_fwd(d["x"][:, :30].contiguous(), d["g"][:, :30].contiguous(), h0=d["h0"], **kw)
        for t in range(30, 40):
            y = gdn.linrec_step(d["x"][:, t], d["g"][:, t], state, **kw)
            ref.check(y, want["y"][:, t], err["y"][:, t], "step %d" % t)
        ref.check(state, want["ht"], err["ht"], "state")
    empty = torch.empty(0, 8, device="cuda")
    assert gdn.linrec_step(empty, empty, empty).shape == (0, 8)


@pytest.mark.parametrize("D", [1, 63, 64, 256, 515])
@pytest.mark.parametrize("dt", [BF, F32])
def test_step_sizes(gpu_lib, D, dt):
    for N in (1, 5, 33):
        d = inputs(N + D, N, 1, D, dt, F32)
        want, err = ref.linrec(d["x"], d["g"], d["h0"])
        y = gpu_lib.linrec_step(d["x"][:, 0], d["g"][:, 0], d["h0"])
        ref.check(y, want["y"][:, 0], err["y"][:, 0], "y")
        ref.check(d["h0"], want["ht"], err["ht"], "state")


@pytest.mark.parametrize("T", [3, 16, 40, 64, 100, 300])
@pytest.mark.parametrize("packed", [False, True])
def test_final_state_over_the_initial_one(gpu_lib, T, packed):
    """ht may be h0: sequences of one wave, of several, of several tiles; the waves of a sequence all read
    h0, one of them writes ht, and with many sequences they do not run in step."""
    print("case: linrec ht = h0", T, packed, flush=True)
    N, D = 200, 130
    d = inputs(51 + T, 1 if packed else N, N * T if packed else T, D, N=N)
    cu = torch.arange(0, N * T + 1, T).cuda() if packed else None
    y, ht = gpu_lib.linrec_fwd(d["x"], d["g"], h0=d["h0"], cu_seqlens=cu)
    state = d["h0"].clone()
    y2, ht2 = gpu_lib.linrec_fwd(d["x"], d["g"], h0=state, cu_seqlens=cu, ht=state)
    assert ht2 is state and torch.equal(ht, state) and torch.equal(y, y2)


def test_state_in_place_and_empty(gpu_lib):
    """ht may be h0; sequences without tokens keep their state, also with T = 0."""
    gdn = gpu_lib
    d = inputs(17, 2, 300, 40)
    want, ht = gdn.linrec_fwd(d["x"], d["g"], h0=d["h0"])
    y, got = gdn.linrec_fwd(d["x"], d["g"], h0=d["h0"], ht=d["h0"])
    torch.cuda.synchronize()
    assert torch.equal(y, want) and torch.equal(got, ht) and got.data_ptr() == d["h0"].data_ptr()
    z = torch.empty(2, 0, 40, dtype=BF, device="cuda")
    gz = torch.empty(2, 0, 40, device="cuda")
    y, ht = gdn.linrec_fwd(z, gz, h0=d["h0"])
    out = gdn.linrec_bwd(z, gz, z, dht=d["dht"], A_log=torch.zeros(40, device="cuda"),
                         dt_bias=torch.zeros(40, device="cuda"))
    torch.cuda.synchronize()
    assert y.shape == (2, 0, 40) and torch.equal(ht, d["h0"]) and torch.equal(out["dh0"], d["dht"])
    assert (out["dA_log"] == 0).all() and (out["ddt_bias"] == 0).all()
    _, ht = gdn.linrec_fwd(z, gz)
    assert (ht == 0).all()


def test_gate_extremes(gpu_lib):
    """Gates of 0 and minus infinity, and raw logits far out: no NaN where the definition has none."""
    gdn = gpu_lib
    d = inputs(18, 1, 200, 64)
    g = d["g"].clone()
    g[:, ::3] = 0.0
    g[:, 1::7] = float("-inf")
    g[:, 2::11] = -1e-30
    for normalize in (False, True):
        y, ht = gdn.linrec_fwd(d["x"], g, h0=d["h0"], normalize=normalize)
        got = gdn.linrec_bwd(d["x"], g, d["dy"], h0=d["h0"], dht=d["dht"], normalize=normalize)
        want, err = ref.linrec(d["x"], g, d["h0"], normalize=normalize)
        ref.check(y, want["y"], err["y"].nan_to_num(1e-6), "y")
        ref.check(ht, want["ht"], err["ht"].nan_to_num(1e-6), "ht")
        for t in ("dx", "dg", "dh0"):
            assert torch.isfinite(got[t]).all(), t
        if normalize:
            assert (got["dx"][:, ::3][g[:, ::3] == 0] == 0).all()      # m = 0 there
    e = inputs(19, 1, 130, 64, BF, F32, True)
    e["g"][:, ::2] = 100.0
    e["g"][:, 1::4] = -100.0
    got = both(gdn, e)
    assert all(torch.isfinite(t).all() for t in got.values())


def test_non_finite_stays_in_its_channel_and_sequence(gpu_lib):
    gdn = gpu_lib
    cu = torch.tensor([0, 200, 470, 600], device="cuda")
    d = inputs(20, 1, 600, 64, N=3)
    clean = gdn.linrec_fwd(d["x"], d["g"], h0=d["h0"], cu_seqlens=cu)
    back = gdn.linrec_bwd(d["x"], d["g"], d["dy"], h0=d["h0"], dht=d["dht"], cu_seqlens=cu)
    x = d["x"].clone()
    x[0, 250, 5], x[0, 199, 6], x[0, 300, 7] = float("nan"), float("inf"), float("-inf")
    y, ht = gdn.linrec_fwd(x, d["g"], h0=d["h0"], cu_seqlens=cu)
    dy = d["dy"].clone()
    dy[0, 250, 5], dy[0, 200, 6], dy[0, 469, 7] = float("nan"), float("inf"), float("inf")
    got = gdn.linrec_bwd(d["x"], d["g"], dy, h0=d["h0"], dht=d["dht"], cu_seqlens=cu)
    torch.cuda.synchronize()
    mask = torch.zeros_like(y, dtype=torch.bool)
    mask[0, 250:470, 5], mask[0, 199:200, 6], mask[0, 300:470, 7] = True, True, True
    assert torch.equal(y[~mask], clean[0][~mask])
    assert torch.isnan(y[0, 250, 5]) and torch.isinf(y[0, 199, 6]) and torch.equal(ht[2], clean[1][2])
    mask = torch.zeros_like(y, dtype=torch.bool)
    mask[0, 200:251, 5], mask[0, 200:201, 6], mask[0, 200:470, 7] = True, True, True
    assert torch.equal(got["dx"][~mask], back["dx"][~mask]) and torch.equal(got["dg"][~mask], back["dg"][~mask])


def test_same_bits_streams_and_graphs(gpu_lib, monkeypatch):
    """Equal bits from equal calls: again, on another stream, and out of replayed graphs with
    eager calls between the replays."""
    gdn = gpu_lib
    d = inputs(21, 1, 128 * 20 + 3, 136, BF, BF, True, N=3)
    cu = torch.tensor([0, 1500, 1500, 128 * 20 + 3], device="cuda")
    kw = dict(h0=d["h0"], cu_seqlens=cu, normalize=True, A_log=d["A_log"], dt_bias=d["dt_bias"])

    def call(stream=None):
        keep = gdn.linrec_states(d["x"], cu)
        y, ht = gdn.linrec_fwd(d["x"], d["g"], states=keep, stream=stream, **kw)
        got = gdn.linrec_bwd(d["x"], d["g"], d["dy"], dht=d["dht"], states=keep, stream=stream, **kw)
        return dict(got, y=y, ht=ht)
    first = call()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    again = call(s)
    s.synchronize()
    assert all(torch.equal(first[k], again[k]) for k in first)
    monkeypatch.setenv("GDN_DEBUG", "0")     # reading the words would wait inside the capture
    graphs = []
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = call()
        graphs.append((graph, out))
    x0 = d["x"].clone()
    for k in range(3):
        d["x"].copy_(x0 * (1 + k))
        want = call()
        torch.cuda.synchronize()
        for graph, out in graphs:
            for t in out.values():
                t.zero_()
            graph.replay()
        torch.cuda.synchronize()
        for _, out in graphs:
            assert all(torch.equal(want[n], out[n]) for n in want), k


def test_packed_short_sequences_in_a_graph(gpu_lib, monkeypatch):
    """Captured and replayed on other inputs, with eager calls between the replays, and on two streams at once."""
    monkeypatch.setenv("GDN_DEBUG", "0")        # its check of the words synchronises
    lengths = [2] * 300 + [700, 0, 2500, 64] * 3
    T, N = sum(lengths), len(lengths)
    cu = torch.tensor([0] + lengths).cumsum(0).cuda()
    print("case: linrec short packed graph", T, N, flush=True)
    d = inputs(81, 1, T, 130, BF, BF, True, N=N)
    kw = dict(h0=d["h0"], cu_seqlens=cu, normalize=True, A_log=d["A_log"], dt_bias=d["dt_bias"])

    def call(stream=None):
        y, ht = gpu_lib.linrec_fwd(d["x"], d["g"], stream=stream, **kw)
        return dict(gpu_lib.linrec_bwd(d["x"], d["g"], d["dy"], dht=d["dht"], stream=stream, **kw), y=y, ht=ht)
    first = call()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = [call(s) for _ in range(3) for s in streams]
    torch.cuda.synchronize()
    assert all(torch.equal(first[n], o[n]) for o in outs for n in first)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = call()
    x0 = d["x"].clone()
    for i in range(4):
        d["x"].copy_(x0 * (1 + i))
        want = call()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(want[n], out[n]) for n in want), i


def test_supplied_outputs_and_workspace(gpu_lib):
    gdn = gpu_lib
    d = inputs(22, 2, 150, 40)
    y0, h0 = gdn.linrec_fwd(d["x"], d["g"])
    ws = torch.full((1 << 22,), 255, dtype=torch.uint8, device="cuda")
    y, ht = torch.empty_like(y0), torch.empty_like(h0)
    r = gdn.linrec_fwd(d["x"], d["g"], y=y, ht=ht, workspace=ws)
    assert r[0] is y and r[1] is ht
    dx = torch.empty_like(y0)
    b0 = gdn.linrec_bwd(d["x"], d["g"], d["dy"], want_dh0=False)
    b = gdn.linrec_bwd(d["x"], d["g"], d["dy"], out=dict(dx=dx), workspace=ws, want_dh0=False)
    torch.cuda.synchronize()
    assert torch.equal(y, y0) and torch.equal(ht, h0) and b["dx"] is dx and torch.equal(dx, b0["dx"])
    assert b["dh0"] is None and gdn.linrec_fwd(d["x"], d["g"], output_final_state=False)[1] is None


@pytest.mark.parametrize("keep", [False, True])
@pytest.mark.parametrize("packed", [False, True])
def test_status_words(gpu_lib, keep, packed):
    """The two status words are this call's, whatever the workspace held."""
    print("case: linrec status words", keep, packed, flush=True)
    d = inputs(23, 1 if packed else 2, 2300, 40)
    cu = torch.tensor([0, 300, 2300]).cuda() if packed else None
    h0 = torch.zeros(2, 40, device="cuda")
    states = gpu_lib.linrec_states(d["x"], cu) if keep else None
    ws = torch.full((1 << 22,), 255, dtype=torch.uint8, device="cuda")
    gpu_lib.linrec_fwd(d["x"], d["g"], h0=h0, cu_seqlens=cu, states=states, workspace=ws)
    torch.cuda.synchronize()
    assert ws[:8].view(torch.int32).tolist() == [0, 0]
    ws.fill_(255)
    gpu_lib.linrec_bwd(d["x"], d["g"], d["dy"], h0=h0, cu_seqlens=cu, states=states, workspace=ws)
    torch.cuda.synchronize()
    assert ws[:8].view(torch.int32).tolist() == [0, 0]


def test_gradient_against_differences(gpu_lib):
    """A directional difference of the kernel's own float32 forward."""
    gdn = gpu_lib
    d = inputs(23, 1, 200, 48, F32, F32, True)
    kw = dict(normalize=True, dt_bias=d["dt_bias"])

    def loss(x, g, h0, A):
        y, ht = gdn.linrec_fwd(x, g, h0=h0, A_log=A, **kw)
        return (y.double() * d["dy"].double()).sum() + (ht.double() * d["dht"].double()).sum()
    at = (d["x"], d["g"], d["h0"], d["A_log"])
    got = gdn.linrec_bwd(d["x"], d["g"], d["dy"], h0=d["h0"], dht=d["dht"], A_log=d["A_log"], **kw)
    for i, name in enumerate(("dx", "dg", "dh0", "dA_log")):
        r = torch.randn(at[i].shape, generator=torch.Generator().manual_seed(i)).cuda()
        e = 1e-2
        hi, lo = (loss(*(t + s * e * r if j == i else t for j, t in enumerate(at))) for s in (1, -1))
        want = (got[name].double() * r.double()).sum()
        # second-order rest of the centred difference, and 32-bit noise over 2e
        tol = 2e-3 * (got[name].double() * r.double()).norm() + 1e-3 * want.abs() + 1e-2
        assert abs((hi - lo) / (2 * e) - want) <= tol, (name, float((hi - lo) / (2 * e)), float(want))


def test_refusals(gpu_lib):
    gdn = gpu_lib
    x = torch.zeros(2, 8, 16, device="cuda")
    h = torch.zeros(2, 16, device="cuda")
    cu = torch.tensor([0, 8], device="cuda")
    bad = [lambda: gdn.linrec_fwd(x, x[:, :4]), lambda: gdn.linrec_fwd(x[0], x[0]),
           lambda: gdn.linrec_fwd(x.half(), x), lambda: gdn.linrec_fwd(x, x, h0=h.double()),
           lambda: gdn.linrec_fwd(x, x, h0=h[:1]), lambda: gdn.linrec_fwd(x, x, h0=h.cpu()),
           lambda: gdn.linrec_fwd(x, x.cpu()), lambda: gdn.linrec_fwd(x, x, A_log=h[0]),
           lambda: gdn.linrec_fwd(x, x, A_log=h[0], dt_bias=h), lambda: gdn.linrec_fwd(x, x, cu_seqlens=cu.int()),
           lambda: gdn.linrec_fwd(x, x, cu_seqlens=cu.cpu()), lambda: gdn.linrec_fwd(x.transpose(1, 2), x.transpose(1, 2)),
           lambda: gdn.linrec_fwd(x[:, ::2][:, :1].expand(2, 8, 16), x), lambda: gdn.linrec_fwd(x, x, y=x[:, :4]),
           lambda: gdn.linrec_fwd(x, x, states=h[:1]), lambda: gdn.linrec_bwd(x, x, x.bfloat16()),
           lambda: gdn.linrec_bwd(x, x, x, dht=h[:1]), lambda: gdn.linrec_bwd(x, x, x, out=dict(dx=x[:, :, :8])),
           lambda: gdn.linrec_step(x[:, 0], x[:, 0], h[:1]), lambda: gdn.linrec_step(x[:, 0], x[:, 0], None),
           lambda: gdn.linrec_step(x, x, h)]
    for i, f in enumerate(bad):
        with pytest.raises((ValueError, TypeError)):
            f()
            print("accepted", i, flush=True)
    with pytest.raises(gdn.GdnError) as e:
        gdn.linrec_fwd(x, x, cu_seqlens=cu)           # packed input has batch 1
    assert e.value.status == 2
    with pytest.raises(gdn.GdnError) as e:
        long = torch.zeros(1, 500, 16, device="cuda")   # several tiles: hand-offs in the workspace
        gdn.linrec_fwd(long, long, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    assert e.value.status == 5


def test_offsets_check(gpu_lib):
    gdn = gpu_lib
    d = inputs(24, 1, 300, 16, N=3)
    for cu in ([0, 200, 100, 300], [10, 100, 200, 300], [0, 100, 200, 290], [0, 100, 200, 1 << 40], [-5, 1, 2, 300]):
        cu = torch.tensor(cu, device="cuda")
        for f in (lambda: gdn.linrec_fwd(d["x"], d["g"], cu_seqlens=cu),
                  lambda: gdn.linrec_bwd(d["x"], d["g"], d["dy"], cu_seqlens=cu)):
            with pytest.raises(gdn.GdnError) as e:
                f()
            assert e.value.status == 8


@pytest.mark.parametrize("first", [0, 100])
def test_growing_gates(gpu_lib, first):
    """Gates above 0 whose products are finite over 2048 tokens (4e3) but not over the sequence: zero states
    stay zero, and states that start late, or gradients that start early, are the definition's."""
    T, D = 65536, 5
    print("case: linrec growing", first, flush=True)
    r = torch.Generator().manual_seed(91)
    g = torch.tensor([0.004, 0.004, 0.003, 0.0008, -0.01]).repeat(1, first + T, 1)
    x, dy = (torch.rand(1, first + T, D, generator=r) + 0.5 for _ in range(2))
    late, early = first + 52000, first + 13000
    x[:, :, 0] = 0.0
    dy[:, :, 0] = 0.0
    x[:, :late, 1:3] = 0.0
    dy[:, early:, 1:3] = 0.0
    cu = torch.tensor([0, first, first + T]) if first else None
    x, g, dy = x.cuda(), g.cuda(), dy.cuda()
    dev = None if cu is None else cu.cuda()
    states = gpu_lib.linrec_states(x, dev)
    y, ht = gpu_lib.linrec_fwd(x, g, cu_seqlens=dev, states=states)
    got = gpu_lib.linrec_bwd(x, g, dy, cu_seqlens=dev, states=states)
    torch.cuda.synchronize()
    want, err = ref.linrec(x, g, cu=cu, dy=dy)
    ref.check_all(dict(got, y=y, ht=ht), want, err)


def whole_numbers(seed, lengths, D, resets):
    """x, g, h0, dy, dht whose recurrence is exact in 32 bits (gates of 0, some of minus infinity, whole numbers),
    and its results: sums between resets."""
    r = torch.Generator().manual_seed(seed)
    T, N = sum(lengths), len(lengths)
    x, dy = (torch.randint(1, 100, (T, D), generator=r) for _ in range(2))
    h0, dht = (torch.randint(-99, 100, (N, D), generator=r) for _ in range(2))
    cut = torch.rand(T, D, generator=r) < resets
    want = dict(y=torch.zeros(T, D), dx=torch.zeros(T, D), dg=torch.zeros(T, D), ht=h0.double(), dh0=dht.double())
    want = {k: v.double() for k, v in want.items()}
    at = 0
    for n, length in enumerate(lengths):
        if length == 0:
            continue
        s = slice(at, at + length)
        at += length
        i = torch.arange(length)[:, None]

        def sums(v, first, reset):      # of v since the last reset, `first` in front
            c = v.cumsum(0)
            last = torch.where(reset, i, -1).cummax(0).values
            base = torch.where(last > 0, c.gather(0, (last - 1).clamp(min=0)), torch.zeros_like(c))
            return c - base + torch.where(last < 0, first, torch.zeros_like(first))
        h = sums(x[s], h0[n], cut[s])
        # dh_t = dy_t + a_{t+1} dh_{t+1}: from the end, a reset at t + 1 comes before token t
        back = torch.cat([torch.zeros(1, D, dtype=torch.bool), cut[s].flip(0)[:-1]])
        dh = sums(dy[s].flip(0), dht[n], back).flip(0)
        a = (~cut[s]).long()
        before = torch.cat([h0[n][None], h[:-1]])
        want["y"][s], want["dx"][s], want["dg"][s] = h.double(), dh.double(), (a * dh * before).double()
        want["ht"][n], want["dh0"][n] = h[-1].double(), (a * dh)[0].double()
    assert all(want[k].abs().max() < 2 ** 24 for k in ("y", "dx", "ht", "dh0")) and want["dg"].abs().max() < 2 ** 53
    g = torch.where(cut, float("-inf"), 0.0)
    return dict(x=x.float()[None], dy=dy.float()[None], g=g[None], h0=h0.float(), dht=dht.float()), want


@pytest.mark.parametrize("lengths", [(40037,), (70001, 0, 128 * 16 * 9, 128 * 16 * 9 + 1), (2,) * 4000 + (45000, 3, 0, 20000),
                                     (150000,)])
@pytest.mark.parametrize("D", [3, 6])
@pytest.mark.parametrize("resets", [0.0, 1e-4])
def test_many_groups_exactly(gpu_lib, lengths, D, resets):
    """Sequences of many groups of tiles, packed ones among short ones too: every pair once and in order."""
    print("case: linrec groups", len(lengths), sum(lengths), D, resets, flush=True)
    d, want = whole_numbers(92, lengths, D, resets)
    d = {k: v.cuda() for k, v in d.items()}
    cu = torch.tensor([0] + list(lengths)).cumsum(0).cuda() if len(lengths) > 1 else None
    for keep in (False, True):
        states = gpu_lib.linrec_states(d["x"], cu) if keep else None
        y, ht = gpu_lib.linrec_fwd(d["x"], d["g"], h0=d["h0"], cu_seqlens=cu, states=states)
        got = gpu_lib.linrec_bwd(d["x"], d["g"], d["dy"], h0=d["h0"], dht=d["dht"], cu_seqlens=cu, states=states)
        torch.cuda.synchronize()
        got.update(y=y, ht=ht)
        for k, w in want.items():
            assert torch.equal(got[k].cpu().view(w.shape), w.float()), (k, keep)


@pytest.mark.parametrize("lengths", [(40037,), (2,) * 3500 + (40000, 5)])
def test_many_groups_of_slow_gates(gpu_lib, lengths):
    """Decays slow enough for far groups to count, inputs above 0 so that none is lost in the bound."""
    T, N, D = sum(lengths), len(lengths), 6
    print("case: linrec slow", N, T, flush=True)
    r = torch.Generator().manual_seed(93)
    g = -torch.rand(1, T, D, generator=r) * torch.tensor([2e-5, 2e-4, 2e-3, 2e-4, 2e-5, 2e-2])
    x, dy = (torch.rand(1, T, D, generator=r).cuda() + 0.5 for _ in range(2))
    h0, dht = (torch.rand(N, D, generator=r).cuda() for _ in range(2))
    cu = torch.tensor([0] + list(lengths)).cumsum(0) if N > 1 else None
    both(gpu_lib, dict(x=x, g=g.cuda(), dy=dy, h0=h0, dht=dht, A_log=None, dt_bias=None), cu, normalize=True)


def test_same_bits_of_a_long_sequence(gpu_lib):
    """Where a tile starts among the groups before it depends on timing; the bits do not."""
    T, D = 100000, 130
    print("case: linrec long bits", T, D, flush=True)
    r = torch.Generator().manual_seed(94)
    x, dy = (torch.randn(1, T, D, generator=r).cuda() for _ in range(2))
    g = (-torch.rand(1, T, D, generator=r) * 1e-3).cuda()

    def call():
        y, ht = gpu_lib.linrec_fwd(x, g)
        return dict(gpu_lib.linrec_bwd(x, g, dy), y=y, ht=ht)
    first = call()
    for _ in range(5):
        again = call()
        assert all(torch.equal(first[n], again[n]) for n in first)


def test_states_belong_to_their_stream(gpu_lib):
    """The buffer of the tiles' states comes from the memory of the stream whose kernels use it, and goes back there."""
    s = torch.cuda.Stream()
    x = torch.zeros(1, 8192, 4096, dtype=BF, device="cuda")
    print("case: linrec states on a stream", flush=True)
    for stream, other in ((s, torch.cuda.current_stream()), (None, s)):
        own = torch.cuda.current_stream() if stream is None else stream
        keep = gpu_lib.linrec_states(x, stream=stream)
        shape, at = keep.shape, keep.data_ptr()
        del keep
        with torch.cuda.stream(other):
            there = torch.empty(shape, device="cuda")
        with torch.cuda.stream(own):
            here = torch.empty(shape, device="cuda")
        assert here.data_ptr() == at and there.data_ptr() != at
        del here, there     # or the next pass finds a block that it frees itself
    x, g = x + 1, x.float() - 0.5
    want, _ = gpu_lib.linrec_fwd(x, g)
    torch.cuda.synchronize()
    keep = gpu_lib.linrec_states(x, stream=s)
    got, _ = gpu_lib.linrec_fwd(x, g, states=keep, stream=s)
    torch.cuda.synchronize()
    assert torch.equal(got, want)


@pytest.mark.parametrize("normalize", [False, True])
@pytest.mark.parametrize("T", [1, 16, 64, 200, 2500])
def test_gradients_at_gate_extremes(gpu_lib, normalize, T):
    """Gates of 0, minus infinity and just below 0: the gradients are the definition's, the slope of
    sqrt(1 - a^2) being taken as 0 where a = 1."""
    print("case: linrec gate extremes", T, normalize, flush=True)
    d = inputs(95, 1, T, 10, F32, F32)
    d["g"][:, ::3] = 0.0
    d["g"][:, 1::7] = float("-inf")
    d["g"][:, 2::11] = -1e-30
    both(gpu_lib, d, normalize=normalize)
    both(gpu_lib, d, normalize=normalize, h0=False, dht=False, keep=False)


@pytest.mark.parametrize("shape", [(1, 1 << 20), (1 << 10, 1 << 10), (64, 64, 64)])
def test_workspace_of_any_shape_and_type(gpu_lib, shape):
    """A supplied workspace counts by its bytes, also where the status words are read from it."""
    print("case: linrec workspace", shape, flush=True)
    d = inputs(96, 1, 300, 24, N=2)
    cu = torch.tensor([0, 100, 300], device="cuda")
    want = gpu_lib.linrec_fwd(d["x"], d["g"], cu_seqlens=cu)
    for dt in (torch.uint8, F32):
        ws = torch.zeros(shape, dtype=dt, device="cuda")
        got = gpu_lib.linrec_fwd(d["x"], d["g"], cu_seqlens=cu, workspace=ws)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        with pytest.raises(gpu_lib.GdnError) as e:
            gpu_lib.linrec_fwd(d["x"], d["g"], cu_seqlens=cu + 1, workspace=ws)
        assert e.value.status == 8
