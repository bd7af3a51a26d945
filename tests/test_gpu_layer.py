"""The layer operators as a layer runs them: convolution, q/k norm with
rotation and the delta rule; convolution and the linear recurrence; prefill,
then steps.  In float32, held to the bar of the float32 delta rule against the
same chain in 64 bits."""
import numpy as np
import pytest
import torch

import layer_ref as ref
import oracle
from oracle.backward import recurrent_backward
from parity_util import TOL, rel_err

pytestmark = pytest.mark.gpu
H, K = 2, 64


def test_delta_rule_layer(gpu_lib):
    """Packed training step of conv -> norm + rotation -> chunk_fwd, forward and backward."""
    gdn = gpu_lib
    r = torch.Generator().manual_seed(1)
    lengths = (70, 0, 130, 3)
    T, N = sum(lengths), len(lengths)
    cu = torch.tensor([sum(lengths[:i]) for i in range(N + 1)])
    pos = torch.cat([torch.arange(n) for n in lengths])[None]
    D = 3 * H * K
    x, w = torch.randn(1, T, D, generator=r), torch.randn(D, 4, generator=r) * 0.5
    beta = torch.sigmoid(torch.randn(1, T, H, generator=r))
    g = -0.1 * torch.rand(1, T, H, generator=r)
    do, dht = torch.randn(1, T, H, K, generator=r), torch.randn(N, H, K, K, generator=r)
    f = 10000.0 ** (-torch.arange(0, 32, 2, dtype=torch.float64) / 32)
    c = {n: t.cuda() for n, t in dict(x=x, w=w, beta=beta, g=g, do=do, dht=dht, f=f, pos=pos, cu=cu).items()}

    u, _ = gdn.short_conv_fwd(c["x"], c["w"], cu_seqlens=c["cu"])
    q, k, v = (t.unflatten(-1, (H, K)) for t in u.split(H * K, -1))      # slices of one projection
    v = v.contiguous()
    qn, kn = gdn.qk_norm_rope(q, k, c["f"], c["pos"], norm="l2")
    o, ht = gdn.chunk_fwd(qn, kn, v, c["beta"], c["g"], cu_seqlens=c["cu"])
    b = gdn.chunk_bwd(qn, kn, v, c["beta"], c["g"], c["do"], dht=c["dht"], cu_seqlens=c["cu"])
    n = gdn.qk_norm_rope_bwd(q, k, b["dq"], b["dk"], c["f"], c["pos"], norm="l2")
    du = torch.cat([t.flatten(2) for t in (n["dq"], n["dk"], b["dv"])], -1)
    cb = gdn.short_conv_bwd(c["x"], c["w"], du, cu_seqlens=c["cu"])
    torch.cuda.synchronize()

    ur, _ = ref.conv(x, w, cu=cu)
    qr, kr, vr = (t.unflatten(-1, (H, K)) for t in ur["y"].split(H * K, -1))
    args = (f, pos, "l2", 1e-6, None, 0.0, False)
    qnr, knr = (ref.qk(t, *args)[0]["out"] for t in (qr, kr))
    s = K ** -0.5
    want_o, want_ht = oracle.recurrent_forward(qnr, knr, vr, beta, g, s, cu_seqlens=cu)
    gr = recurrent_backward(qnr, knr, vr, beta, g, s, do, dht=dht, cu_seqlens=cu)
    gr = {key: torch.as_tensor(np.asarray(t)) for key, t in gr.items() if t is not None}
    dqr, dkr = (ref.qk(t, *args, dout=d)[0]["dx"] for t, d in ((qr, gr["dq"]), (kr, gr["dk"])))
    dur = torch.cat([t.flatten(2) for t in (dqr, dkr, gr["dv"])], -1)
    cr, _ = ref.conv(x, w, cu=cu, dy=dur)
    for name, got, want in (("o", o, want_o), ("ht", ht, want_ht), ("dx", cb["dx"], cr["dx"].numpy()),
                            ("dweight", cb["dweight"], cr["dweight"].numpy())):
        e = rel_err(got, np.asarray(want))
        assert e <= TOL["f32"], (name, e)


def test_recurrent_block_prefill_then_steps(gpu_lib):
    """Chunked prefill (two calls carrying window and state), then single tokens."""
    gdn = gpu_lib
    r = torch.Generator().manual_seed(2)
    B, T, D = 3, 300, 96
    x, w, b = torch.randn(B, T, D, generator=r), torch.randn(D, 4, generator=r) * 0.5, torch.randn(D, generator=r)
    g, A, dt = torch.randn(B, T, D, generator=r), torch.rand(D, generator=r), torch.randn(D, generator=r) - 4
    kw = dict(normalize=True, A_log=A.cuda(), dt_bias=dt.cuda())
    xd, wd, bd, gd = x.cuda(), w.cuda(), b.cuda(), g.cuda()
    outs, st, h = [], None, None
    for a, e in ((0, 200), (200, 290)):
        u, st = gdn.short_conv_fwd(xd[:, a:e].contiguous(), wd, bd, s0=st, output_final_state=True)
        y, h = gdn.linrec_fwd(u, gd[:, a:e].contiguous(), h0=h, **kw)
        outs.append(y)
    for t in range(290, T):
        u = gdn.short_conv_step(xd[:, t], wd, st, bd)
        outs.append(gdn.linrec_step(u, gd[:, t], h, **kw)[:, None])
    torch.cuda.synchronize()
    u, _ = ref.conv(x, w, b)
    want, _ = ref.linrec(u["y"], g, normalize=True, A_log=A, dt_bias=dt)
    assert rel_err(torch.cat(outs, 1), want["y"].numpy()) <= TOL["f32"]
    assert rel_err(h, want["ht"].numpy()) <= TOL["f32"] and torch.equal(st.cpu(), x[:, -3:])


def test_recurrent_block_gradients(gpu_lib):
    gdn = gpu_lib
    r = torch.Generator().manual_seed(3)
    B, T, D = 2, 260, 40
    x, w = torch.randn(B, T, D, generator=r), torch.randn(D, 3, generator=r) * 0.5
    g, dy = -0.2 * torch.rand(B, T, D, generator=r), torch.randn(B, T, D, generator=r)
    u, _ = gdn.short_conv_fwd(x.cuda(), w.cuda())
    keep = gdn.linrec_states(u)
    gdn.linrec_fwd(u, g.cuda(), states=keep)
    d = gdn.linrec_bwd(u, g.cuda(), dy.cuda(), states=keep)
    c = gdn.short_conv_bwd(x.cuda(), w.cuda(), d["dx"])
    torch.cuda.synchronize()
    ur, _ = ref.conv(x, w)
    dr, _ = ref.linrec(ur["y"], g, dy=dy)
    cr, _ = ref.conv(x, w, dy=dr["dx"])
    for name, got, want in (("dg", d["dg"], dr["dg"]), ("dx", c["dx"], cr["dx"]), ("dweight", c["dweight"], cr["dweight"])):
        e = rel_err(got, want.numpy())
        assert e <= TOL["f32"], (name, e)


# offsets over 700 tokens; the invalid ones decrease, so that the sequences' tiles come to more
# than the table holds
OFFSETS = {"valid": [0, 0, 300, 301, 700, 700, 700], "twice": [0, 700, 0, 700, 0, 700],
           "many": [0, 700] * 40, "beyond": [5, 900, -3, 1 << 40, 0, 650], "tail": [0, 1, 0, 2, 0, 700]}


@pytest.mark.parametrize("name", sorted(OFFSETS))
def test_offsets_stay_inside(gpu_lib, monkeypatch, name):
    """Whatever the offsets: nothing is written past a workspace of the size asked for or past
    the last token, no wait gives up, and the check of the offsets says which were invalid."""
    gdn = gpu_lib
    monkeypatch.setenv("GDN_DEBUG", "0")     # the words are read here
    cu = torch.tensor(OFFSETS[name], device="cuda")
    r = torch.Generator().manual_seed(1)
    T, D = 700, 40
    x, dy = (torch.randn(1, T, D, generator=r).cuda() for _ in range(2))
    g, w = -torch.rand(1, T, D, generator=r).cuda(), torch.randn(D, 4, generator=r).cuda()
    N = cu.numel() - 1
    h = torch.zeros(N, D, device="cuda")

    def room(plan_bytes):
        buf = torch.full((plan_bytes + 4096,), 77, dtype=torch.uint8, device="cuda")
        return buf, buf[:plan_bytes]

    def rows():
        buf = torch.full((1, T + 64, D), 7.0, device="cuda")
        return buf, buf[:, :T]
    from gated_delta_rule_14_amd import _layer as L
    lp = L._linrec_plan(1, T, D, N, 0, 0, 0, 0, 0, 0)
    cp = L._conv_plan(1, T, D, N, 0, 0, 0, 4, 1)
    for nbytes, call in (
            (lp.fwd, lambda ws, o: gdn.linrec_fwd(x, g, cu_seqlens=cu, y=o, workspace=ws)),
            (lp.bwd, lambda ws, o: gdn.linrec_bwd(x, g, dy, dht=h, cu_seqlens=cu, out=dict(dx=o), workspace=ws)),
            (cp.fwd, lambda ws, o: gdn.short_conv_fwd(x, w, cu_seqlens=cu, output_final_state=True, y=o, workspace=ws)),
            (cp.bwd, lambda ws, o: gdn.short_conv_bwd(x, w, dy, cu_seqlens=cu, out=dict(dx=o), workspace=ws))):
        print("case: offsets", name, nbytes, flush=True)
        (buf, ws), (big, o) = room(nbytes), rows()
        call(ws, o)
        torch.cuda.synchronize()
        assert (buf[nbytes:] == 77).all() and (big[:, T:] == 7).all()
        bad, wait = ws[:8].view(torch.int32).tolist()
        assert bad == (name != "valid") and wait == 0
