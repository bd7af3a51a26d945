"""The append to a paged cache and the attention of one new token over it, on
the GPU against 64-bit definitions, within bounds on the rounding of every step."""
import pytest
import torch

import layer_ref
import mixer_ref as ref

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
NAN = float("nan")


def pool(seed, lens, P, Hk, D, dt, layout="dense", spare=2, width=None):
    """A cache with the pages of `lens` tokens in random order: (k, v, table), values random, NaN
    where no sequence has a token."""
    r = torch.Generator().manual_seed(seed)
    need = [-(-max(n, 0) // P) for n in lens]
    total, M = sum(need) + spare, width or max(1, max(need, default=1))
    order = torch.randperm(total, generator=r)
    table = torch.full((len(lens), M), -1, dtype=torch.int32)
    shape = {"dense": (total, P, Hk, D), "heads": (total, Hk, P, D), "pairs": (total, 2, P, Hk, D)}[layout]
    kv = [torch.full(shape, NAN, dtype=DT[dt]) for _ in range(1 if layout == "pairs" else 2)]
    k, v = (kv[0][:, 0], kv[0][:, 1]) if layout == "pairs" else (t.transpose(1, 2) if layout == "heads" else t for t in kv)
    at = 0
    for n, (L, c) in enumerate(zip(lens, need)):
        table[n, :c] = order[at:at + c].to(torch.int32)
        at += c
        for t in range(L):
            for cache in (k, v):
                cache[table[n, t // P], t % P] = torch.randn(Hk, D, generator=r).to(DT[dt])
    return k, v, table


def cuda(t):
    base = torch.empty(0, dtype=t.dtype).set_(t.untyped_storage()).cuda()
    return base.as_strided(t.shape, t.stride(), t.storage_offset())


def run_attn(gdn, seed, lens, P, Hk, m, D, dt, layout="dense", scale=None, window=0, width=None, spread=1.0):
    k, v, table = pool(seed, lens, P, Hk, D, dt, layout, width=width)
    q = (spread * torch.randn(len(lens), Hk * m, D, generator=torch.Generator().manual_seed(seed + 1))).to(DT[dt])
    n = torch.tensor(lens)
    o = gdn.paged_attn(q.cuda(), cuda(k), cuda(v), table.cuda(), n.cuda(), scale=scale, window=window)
    torch.cuda.synchronize()
    want, err = ref.attn(q, k, v, table, n, scale, window)
    layer_ref.check(o, want, err, "o")
    return o


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("D", [8, 24, 64, 96, 128, 200, 256])
def test_attn_head_sizes(gpu_lib, dt, D):
    run_attn(gpu_lib, 1, (37, 1, 0, 200), 16, 2, 3, D, dt)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("Hk,m", [(1, 1), (5, 1), (1, 16), (2, 20), (1, 33)])
def test_attn_groups(gpu_lib, dt, Hk, m):
    run_attn(gpu_lib, 2, (70, 129), 8, Hk, m, 64, dt)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("P,layout", [(1, "dense"), (7, "heads"), (16, "pairs"), (24, "heads"), (64, "dense"), (256, "pairs")])
def test_attn_pages_and_lengths(gpu_lib, dt, P, layout):
    """Lengths at the borders of waves, pieces and pages; 2000 tokens run in several pieces."""
    run_attn(gpu_lib, 3, (0, 1, 2, 31, 32, 33, 127, 128, 129, 257, 600, 2000), P, 1, 2, 64, dt, layout)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("window", [1, 5, 32, 100, 129, 5000])
def test_attn_window(gpu_lib, dt, window):
    run_attn(gpu_lib, 4, (0, 1, 40, 300, 1001, 1000), 16, 2, 2, 64, dt, window=window)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("N", [1, 64, 65, 200])
def test_attn_many_sequences(gpu_lib, dt, N):
    run_attn(gpu_lib, 5, tuple((37 * i * i) % 71 for i in range(N)), 16, 1, 2, 64, dt)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_attn_peaked_scores(gpu_lib, dt):
    """Scores of some hundred: one token takes all, and its maximum may come late; and a scale of its own."""
    run_attn(gpu_lib, 6, (500, 130, 3), 16, 1, 4, 128, dt, spread=60.0)
    run_attn(gpu_lib, 7, (500, 130, 3), 16, 1, 4, 128, dt, scale=-0.7)


def test_attn_lowest_and_infinite_keys(gpu_lib):
    """Keys of the type's lowest value next to others, infinite ones behind the last token."""
    gdn = gpu_lib
    k, v, table = pool(8, (90, 5), 16, 1, 64, "f32")
    k[table[0, 1], :] = torch.finfo(torch.float32).min
    k[k.isnan()] = float("inf")
    v[v.isnan()] = -float("inf")
    q, n = torch.rand(2, 2, 64) + 0.5, torch.tensor([90, 5])
    o = gdn.paged_attn(q.cuda(), k.cuda(), v.cuda(), table.cuda(), n.cuda())
    keep = [t for t in range(90) if t // 16 != 1]                 # scores of -inf: weight 0
    kk, vv = ref.rows(k, table, 0, 0, 90)[keep], ref.rows(v, table, 0, 0, 90)[keep]
    x = torch.softmax((q[0].double() * kk).sum(-1) / 8, 0)
    want = (x[..., None] * vv).sum(0)
    # 64 products and 74 weights in 32 bits: scores of up to some tens
    assert torch.allclose(o[0].cpu().double(), want, rtol=0, atol=(64 + 74 + 100) * 2.0 ** -24 * float(vv.abs().max()))


def test_attn_bad_pages_and_lengths_are_left_out(gpu_lib, monkeypatch):
    """Without GDN_DEBUG what has no page is not there; with it the call raises."""
    gdn = gpu_lib
    k, v, table = pool(9, (100, 64, 40, 20), 16, 2, 64, "f32", width=7)
    table[0, 2], table[1, 0], table[2, 1] = -5, 10 ** 6, k.shape[0]
    table[3] = -1
    n = torch.tensor([100, 10 ** 12, -3, 20])
    q = torch.randn(4, 4, 64)
    args = (q.cuda(), k.cuda(), v.cuda(), table.cuda(), n.cuda())
    with pytest.raises(ValueError):
        gdn.paged_attn(*args)
    with pytest.raises(ValueError, match="page_table"):
        gdn.paged_attn(*args[:4], n.clamp(0, 100).cuda())
    monkeypatch.setenv("GDN_DEBUG", "0")
    for window in (0, 37):
        o = gdn.paged_attn(*args, window=window)
        # (sequence 1 counts up to the table's end; its pages there are -1)
        want, err = ref.attn(q, k, v, table, n.clamp(max=112), None, window)
        layer_ref.check(o, want, err, "o")
        assert bool((o[2:] == 0).all())


def test_attn_far_page(gpu_lib):
    """A page behind 2^31 elements of the pool."""
    gdn = gpu_lib
    step = (1 << 31) + 64 * 1024
    base = torch.zeros(step + 4096, dtype=torch.bfloat16, device="cuda")
    kc, vc = (base[i:].as_strided((2, 16, 2, 64), (step, 128, 64, 1)) for i in (0, 2048))
    q = torch.randn(1, 4, 64, device="cuda").bfloat16()
    new = torch.randn(1, 20, 2, 64, device="cuda").bfloat16()
    table, n = torch.tensor([[1, 0]], dtype=torch.int32, device="cuda"), torch.zeros(1, dtype=torch.int64, device="cuda")
    gdn.paged_append(None, new, -new, kc, vc, table, n)
    n += 20
    o = gdn.paged_attn(q, kc, vc, table, n)
    torch.cuda.synchronize()
    assert torch.equal(kc[1], new[0, :16]) and torch.equal(kc[0, :4], new[0, 16:]) and torch.equal(vc[1], -new[0, :16])
    want, err = ref.attn(q, kc.cpu(), vc.cpu(), table, n)
    layer_ref.check(o, want, err, "o")


def append_ref(d, lens, pos, cu, kw):
    """The rotated q and the rows that go to the cache, with bounds."""
    f, w = kw["inv_freq"], (kw["q_weight"], kw["k_weight"])
    out = []
    for t, wt in ((d["q"], w[0]), (d["k"], w[1])):
        v, e = layer_ref.qk(t, f, pos, kw["norm"], kw["eps"], wt, kw["weight_offset"], kw["interleaved"])
        out.append((v["out"], e["out"]))
    return out


def run_append(gdn, seed, held, news, P, Hq, Hk, D, dt, R=None, layout="dense", norm="rms", w=True, off=0.0, inter=False,
               packed=False, with_q=True, given=False, gap=True):
    r = torch.Generator().manual_seed(seed)
    N = len(held)
    k, v, table = pool(seed, [a + b for a, b in zip(held, news)], P, Hk, D, dt, layout)
    lead = (1, sum(news)) if packed else (N, news[0])
    wide = 2 if gap else 1
    d = dict(q=torch.randn(*lead, Hq, wide * D, generator=r).to(DT[dt])[..., :D])
    u = torch.randn(*lead, 2 * Hk, D, generator=r).to(DT[dt])
    d["k"], d["v"] = u[:, :, :Hk], u[:, :, Hk:]
    if not gap:
        d = {n: t.contiguous() for n, t in d.items()}
    R = D // 16 * 16 if R is None else R
    kw = dict(inv_freq=10000.0 ** (-torch.arange(0, R, 2, dtype=torch.float64) / R) if R else None, norm=norm, eps=1e-6,
              q_weight=torch.rand(D, generator=r) if w else None, k_weight=torch.rand(D, generator=r) if w else None,
              weight_offset=off, interleaved=inter)
    own = torch.cat([torch.arange(b) + a for a, b in zip(held, news)])
    seq = torch.cat([torch.full((b,), n) for n, b in enumerate(news)])
    pos = torch.randint(0, 10 ** 6, own.shape, generator=r) if given else own
    cu = torch.tensor([sum(news[:i]) for i in range(N + 1)]) if packed else None
    kc, vc = cuda(k), cuda(v)
    before = [x.clone() for x in (k, v)]
    dev = lambda x: x.cuda() if isinstance(x, torch.Tensor) else x  # noqa: E731
    got = gdn.paged_append(cuda(d["q"]) if with_q else None, cuda(d["k"]), cuda(d["v"]), kc, vc, table.cuda(),
                           torch.tensor(held).cuda(), positions=pos.view(lead).cuda() if given else None, cu_seqlens=dev(cu),
                           **{n: dev(x) for n, x in kw.items()})
    torch.cuda.synchronize()
    (qo, qe), (ko, ke) = append_ref(d, held, pos.view(lead), cu, kw)
    if with_q:
        layer_ref.check(got, qo, qe, "q")
    else:
        assert got is None
    page, slot = table[seq, own // P].long(), own % P
    layer_ref.check(kc.cpu()[page, slot], ko.flatten(0, 1), ke.flatten(0, 1), "k")
    assert torch.equal(vc.cpu()[page, slot], d["v"].flatten(0, 1))
    for x, old in ((kc, before[0]), (vc, before[1])):                # nothing else was touched
        x, rest = x.cpu().clone(), old.clone()
        x[page, slot], rest[page, slot] = 0, 0
        assert bool(((x == rest) | (x.isnan() & rest.isnan())).all())


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("D,R", [(8, 0), (16, 16), (64, 32), (72, 64), (128, 128), (256, 64)])
def test_append_head_sizes(gpu_lib, dt, D, R):
    run_append(gpu_lib, 20, (0, 15, 16, 33), (1, 1, 1, 1), 16, 4, 2, D, dt, R)
    run_append(gpu_lib, 21, (0, 5), (40, 40), 24, 3, 5, D, dt, R, layout="heads", inter=True, off=1.0, norm="l2")


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("P,layout", [(1, "dense"), (7, "pairs"), (64, "heads")])
def test_append_packed(gpu_lib, dt, P, layout):
    run_append(gpu_lib, 22, (3, 0, 100, 64, 0), (70, 0, 1, 33, 0), P, 4, 2, 64, dt, layout=layout, packed=True)
    run_append(gpu_lib, 23, (3,), (130,), P, 1, 1, 128, dt, layout=layout, packed=True, given=True, with_q=False, w=False,
               norm="none", gap=False)


def test_append_many_sequences(gpu_lib):
    """More packed sequences than one look at the offsets covers, empty ones among them."""
    news = tuple((7 * i) % 4 for i in range(300))
    run_append(gpu_lib, 24, tuple(i % 20 for i in range(300)), news, 16, 2, 1, 64, "bf16", packed=True)


def test_append_outside_is_left_out(gpu_lib, monkeypatch):
    gdn = gpu_lib
    P, Hk, D = 16, 2, 64
    kc, vc = (torch.zeros(6, P, Hk, D, device="cuda") for _ in range(2))
    table = torch.tensor([[0, 1], [2, 9], [-1, 3], [4, 5], [4, 5]], dtype=torch.int32, device="cuda")
    lens = torch.tensor([31, 15, 15, -1, 33], device="cuda")
    x = 1 + torch.rand(5, 3, Hk, D, device="cuda")
    with pytest.raises(ValueError):
        gdn.paged_append(x, x, x, kc, vc, table, lens)
    monkeypatch.setenv("GDN_DEBUG", "0")
    q = gdn.paged_append(x, x, x, kc, vc, table, lens)
    torch.cuda.synchronize()
    assert torch.equal(q, x)
    want = torch.zeros_like(kc)
    want[1, 15], want[2, 15], want[3, 0], want[3, 1] = x[0, 0], x[1, 0], x[2, 1], x[2, 2]
    assert torch.equal(kc, want) and torch.equal(vc, want)
    # offsets that make no sense write no page twice as long as they lie in their sequence, and nothing outside
    kc.zero_(), vc.zero_()
    y = 1 + torch.rand(1, 8, Hk, D, device="cuda")
    for cu in ([0, 100, 8], [5, 2, 8], [-4, 1, 3], [8, 8, 8]):
        gdn.paged_append(y, y, y, kc, vc, table[:2].contiguous(), lens[:2].contiguous() * 0,
                         cu_seqlens=torch.tensor(cu, device="cuda"))
    torch.cuda.synchronize()
    assert bool((kc[3:] == 0).all())


def test_same_bits_streams_and_graphs(gpu_lib, monkeypatch):
    gdn = gpu_lib
    lens = [300, 0, 1500, 64]
    k, v, table = pool(30, [x + 4 for x in lens], 16, 2, 128, "bf16")
    r = torch.Generator().manual_seed(31)
    kc, vc, tb, n = k.cuda(), v.cuda(), table.cuda(), torch.tensor(lens).cuda()
    q, kn, vn = (torch.randn(4, 1, h, 128, generator=r).bfloat16().cuda() for h in (8, 2, 2))
    f = 10000.0 ** (-torch.arange(0, 64, 2, dtype=torch.float64) / 64).cuda()

    def call(stream=None, ws=None):
        x = gdn.paged_append(q, kn, vn, kc, vc, tb, n, f, norm="rms", stream=stream)
        return gdn.paged_attn(x[:, 0], kc, vc, tb, n + 1 if stream is None else more, stream=stream, workspace=ws)
    more = n + 1
    first = call()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    again, other = call(s), call()               # two at once, workspaces of their own
    torch.cuda.synchronize()
    assert torch.equal(first, again) and torch.equal(first, other)
    ws = gdn.paged_attn_workspace(q[:, 0], kc, vc, tb, n)
    ws.fill_(255)
    assert torch.equal(first, call(ws=ws))
    monkeypatch.setenv("GDN_DEBUG", "0")         # looking at the lengths would wait inside the capture
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = call()
    for step in range(4):                        # the lengths grow by themselves between replays
        q.mul_(1.01)
        want = call()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(want, out), step
        n += 1


def test_refusals(gpu_lib):
    gdn = gpu_lib
    z = lambda *s, t=torch.bfloat16: torch.zeros(*s, dtype=t, device="cuda")  # noqa: E731
    kc, vc, table, lens = z(4, 16, 2, 64), z(4, 16, 2, 64), z(3, 2, t=torch.int32), z(3, t=torch.int64)
    q, k, x = z(3, 1, 4, 64), z(3, 1, 2, 64), z(3, 4, 64)
    bad = [lambda: gdn.paged_append(q, k[0], k[0], kc, vc, table, lens), lambda: gdn.paged_append(q[:2], k, k, kc, vc, table, lens),
           lambda: gdn.paged_append(q, k, k[:, :, :1], kc, vc, table, lens), lambda: gdn.paged_append(q.float(), k, k, kc, vc, table, lens),
           lambda: gdn.paged_append(q, k, k.float(), kc, vc, table, lens), lambda: gdn.paged_append(q, k, k, kc.float(), vc, table, lens),
           lambda: gdn.paged_append(q, k, k, kc[:, :, :1], vc, table, lens), lambda: gdn.paged_append(q, k, k, kc, vc, table.long(), lens),
           lambda: gdn.paged_append(q, k, k, kc, vc, table, lens.int()), lambda: gdn.paged_append(q, k, k, kc, vc, table[:2], lens[:2]),
           lambda: gdn.paged_append(q, k, k, kc, vc, table, lens, norm="layer"),
           lambda: gdn.paged_append(q, k, k, kc, vc, table, lens, inv_freq=z(32, t=torch.float32)),
           lambda: gdn.paged_append(q, k, k, kc, vc, table, lens, positions=z(3, t=torch.int64)),
           lambda: gdn.paged_append(q, k, k, kc, vc, table, lens, cu_seqlens=z(4, t=torch.int64)),
           lambda: gdn.paged_append(q, k, k, kc, vc, table, lens, q_out=q[:, :, :2]),
           lambda: gdn.paged_attn(q, kc, vc, table, lens), lambda: gdn.paged_attn(x[:2], kc, vc, table, lens),
           lambda: gdn.paged_attn(x.float(), kc, vc, table, lens), lambda: gdn.paged_attn(x[..., :32], kc, vc, table, lens),
           lambda: gdn.paged_attn(x, kc, vc[:2], table, lens), lambda: gdn.paged_attn(x, kc, vc, table[0], lens),
           lambda: gdn.paged_attn(x, kc.transpose(2, 3), vc.transpose(2, 3), table, lens),
           lambda: gdn.paged_attn(x, kc, vc, table, lens, o=x.float()), lambda: gdn.paged_attn(x, kc[0], vc[0], table, lens)]
    for i, f in enumerate(bad):
        with pytest.raises((ValueError, TypeError)):
            f()
            print("accepted", i, flush=True)
    one = z(4, 16, 1, 64).expand(4, 16, 2, 64)
    for f, code in ((lambda: gdn.paged_attn(z(3, 3, 64), kc, vc, table, lens), 2), (lambda: gdn.paged_attn(x, one, vc, table, lens), 2),
                    (lambda: gdn.paged_attn(x, kc, vc, table, lens, window=-1), 2),
                    (lambda: gdn.paged_attn(x, kc, vc, table, lens, workspace=z(256, t=torch.uint8)), 5),
                    (lambda: gdn.paged_append(q, k, k, kc, one, table, lens), 2)):
        with pytest.raises(gdn.GdnError) as e:
            f()
        assert e.value.status == code, e.value
    assert gdn.paged_attn(x[:0], kc, vc, table[:0], lens[:0]).shape == (0, 4, 64)
