"""The token mixers where element offsets pass 32 bits: rows far apart, and many
tokens; and many sequences at once."""
import pytest
import torch

import layer_ref
import mixer_ref as ref

pytestmark = pytest.mark.gpu


def test_rows_far_apart(gpu_lib):
    """q, k and v as slices of tokens 2^24 - 64 elements apart: 300 tokens span 10 GB."""
    gdn = gpu_lib
    T, step = 300, (1 << 24) - 64
    base = torch.empty(T * step, dtype=torch.bfloat16, device="cuda")
    rows = base.as_strided((1, T, 1, 3 * 64), (T * step, step, 192, 1))
    r = torch.Generator().manual_seed(1)
    x = torch.randn(1, T, 1, 192, generator=r).bfloat16()
    rows.copy_(x)
    q, k, v = rows.split(64, -1)
    g, do = -0.1 * torch.rand(1, T, 1, generator=r), torch.randn(1, T, 1, 64, generator=r).bfloat16()
    o, ht = gdn.decay_attn_fwd(q, k, v, g.cuda())
    b = gdn.decay_attn_bwd(q, k, v, g.cuda(), do.cuda())
    torch.cuda.synchronize()
    xq, xk, xv = x.split(64, -1)
    want, err = ref.decay(xq, xk, xv, g, do=do)
    layer_ref.check_all(dict(b, o=o, ht=ht), want, err)
    with pytest.raises(gdn.GdnError) as e:
        gdn.decay_attn_fwd(*(t[:, ::2] for t in (q, k, v)), g[:, ::2].contiguous().cuda())
    assert e.value.status == 2


def test_many_tokens(gpu_lib):
    """A pack of 2.3e9 elements of v; the last sequence alone is checked, and the first tokens."""
    gdn = gpu_lib
    H, V, lens = 70, 128, (258000, 300)
    T = sum(lens)
    r = torch.Generator(device="cuda").manual_seed(2)
    v = torch.empty(1, T, H, V, dtype=torch.bfloat16, device="cuda").normal_(generator=r)
    assert v.numel() > 1 << 31
    q, k = (torch.empty(1, T, 1, 64, dtype=torch.bfloat16, device="cuda").normal_(generator=r) for _ in range(2))
    g = -0.1 * torch.rand(1, T, H, device="cuda", generator=r)
    cu = torch.tensor([0, lens[0], T], device="cuda")
    o, ht = gdn.decay_attn_fwd(q, k, v, g, cu_seqlens=cu)
    torch.cuda.synchronize()
    heads = [0, 33, 69]
    for at, n in ((slice(0, 200), None), (slice(lens[0], T), 1)):
        want, err = ref.decay(q[:, at].cpu(), k[:, at].cpu(), v[:, at][:, :, heads].cpu(), g[:, at][:, :, heads].cpu())
        layer_ref.check(o[:, at][:, :, heads], want["o"], err["o"], "o")
        if n is not None:
            layer_ref.check(ht[n:n + 1, heads], want["ht"], err["ht"], "ht")


@pytest.mark.parametrize("N", [1500, 5000])
def test_many_sequences(gpu_lib, N):
    """Short ones, empty ones among them, and one of several segments."""
    gdn = gpu_lib
    lens = [(i * 7) % 4 for i in range(N)]
    lens[N // 2] = 900
    T = sum(lens)
    r = torch.Generator().manual_seed(3)
    n = lambda *s: torch.randn(*s, generator=r)  # noqa: E731
    d = dict(q=n(1, T, 1, 64), k=n(1, T, 1, 64), v=n(1, T, 1, 64), g=-0.2 * torch.rand(1, T, 1, generator=r))
    do, h0 = n(1, T, 1, 64), n(N, 1, 64, 64)
    cu = torch.tensor([0] + lens).cumsum(0)
    c = {name: t.cuda() for name, t in d.items()}
    o, ht = gdn.decay_attn_fwd(c["q"], c["k"], c["v"], c["g"], h0=h0.cuda(), cu_seqlens=cu.cuda())
    b = gdn.decay_attn_bwd(c["q"], c["k"], c["v"], c["g"], do.cuda(), h0=h0.cuda(), cu_seqlens=cu.cuda())
    torch.cuda.synchronize()
    pick = [0, 1, 2, N // 2, N - 3, N - 1]
    for i in pick:
        a, e = int(cu[i]), int(cu[i + 1])
        want, err = ref.decay(*(d[x][:, a:e] for x in "qkvg"), None, h0[i:i + 1], None, do[:, a:e])
        got = {x: b[x][:, a:e] for x in ("dq", "dk", "dv", "dg")}
        got.update(o=o[:, a:e], ht=ht[i:i + 1], dh0=b["dh0"][i:i + 1])
        layer_ref.check_all(got, want, err, "sequence %d" % i)
