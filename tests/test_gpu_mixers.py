"""The token mixers as a stack runs them: a prompt, then tokens one by one,
through a delta-rule layer, a decayed linear attention layer and an attention
layer over a paged cache; float32, against the same stack in 64 bits over the
whole sequence."""
import numpy as np
import pytest
import torch

import layer_ref
import mixer_ref
import oracle
from parity_util import TOL, rel_err

pytestmark = pytest.mark.gpu
H, K = 2, 64


def weights(seed):
    r = torch.Generator().manual_seed(seed)
    W = H * K
    return {n: torch.randn(*s, generator=r) * s[0] ** -0.5 for n, s in
            dict(delta=(W, 3 * W + 8), decay=(W, 3 * W + 8), attn=(W, 3 * W)).items()}


def split(u, *widths):
    out = u.split(widths, -1)
    return [t.unflatten(-1, (H, K)) if w == H * K else t for t, w in zip(out, widths)]


def stack_in_64_bits(x, w, f):
    """[1, T, H K] through the three layers, every token at once."""
    x, w, W, T = x.double(), {n: t.double() for n, t in w.items()}, H * K, x.shape[1]
    q, k, v, b, g, _ = split(x @ w["delta"], W, W, W, H, H, 8 - 2 * H)
    q, k = (layer_ref.qk(t, None, None, "l2", 1e-6, None, 0.0, False)[0]["out"] for t in (q, k))
    o, _ = oracle.recurrent_forward(q, k, v, torch.sigmoid(b), -torch.sigmoid(g), K ** -0.5)
    x = x + torch.as_tensor(np.asarray(o)).flatten(2)
    q, k, v, g, _ = split(x @ w["decay"], W, W, W, H, 8 - H)
    o, _ = mixer_ref.decay(q.float(), k.float(), v.float(), -torch.sigmoid(g))
    x = x + o["o"].flatten(2)
    q, k, v = split(x @ w["attn"], W, W, W)
    q, k = (layer_ref.qk(t, f, None, "rms", 1e-6, None, 0.0, False)[0]["out"] for t in (q, k))
    s = torch.einsum("bihk,bjhk->bhij", q, k) * K ** -0.5
    s = s.masked_fill(torch.ones(T, T).triu(1).bool(), -float("inf"))
    return x + torch.einsum("bhij,bjhk->bihk", torch.softmax(s, -1), v).flatten(2)


def test_prompt_then_tokens(gpu_lib, monkeypatch):
    """Prompt of 150 tokens of one request, then 10 tokens each out of one captured graph."""
    gdn = gpu_lib
    T, P, pre = 160, 16, 150
    r = torch.Generator().manual_seed(1)
    x, w = torch.randn(1, T, H * K, generator=r), weights(2)
    f = 10000.0 ** (-torch.arange(0, 32, 2, dtype=torch.float64) / 32)
    want = stack_in_64_bits(x, w, f)
    w, f, xd, W = {n: t.cuda() for n, t in w.items()}, f.cuda(), x.cuda(), H * K
    kc, vc = (torch.full((12, P, H, K), float("nan"), device="cuda") for _ in range(2))
    table = torch.randperm(12, generator=r).to(torch.int32)[None, :10].contiguous().cuda()
    lens = torch.zeros(1, dtype=torch.int64, device="cuda")

    def mixers(x, delta, decay, attn):
        q, k, v, b, g, _ = split(x @ w["delta"], W, W, W, H, H, 8 - 2 * H)
        q, k = gdn.qk_norm_rope(q, k, norm="l2")
        x = x + delta(q, k, v.contiguous(), torch.sigmoid(b).contiguous(), -torch.sigmoid(g).contiguous()).flatten(2)
        q, k, v, g, _ = split(x @ w["decay"], W, W, W, H, 8 - H)
        x = x + decay(q, k, v, -torch.sigmoid(g).contiguous()).flatten(2)
        q, k, v = split(x @ w["attn"], W, W, W)
        q = gdn.paged_append(q, k, v, kc, vc, table, lens, f, norm="rms")
        return x + attn(q).flatten(2)

    states = {}

    def first(name, fn):
        def call(*a):
            o, states[name] = fn(*a)
            return o
        return call

    def each(q):           # the prompt's attention, a token at a time
        return torch.stack([gdn.paged_attn(q[:, t].contiguous(), kc, vc, table, lens + t + 1) for t in range(q.shape[1])], 1)
    y = mixers(xd[:, :pre], first("delta", gdn.chunk_fwd), first("decay", gdn.decay_attn_fwd), each)
    lens += pre

    def step(fn, name):
        return lambda *a: fn(*(t[:, 0].contiguous() for t in a), states[name])[:, None]

    def token(x):
        y = mixers(x, step(gdn.recurrent_step, "delta"), step(gdn.decay_attn_step, "decay"),
                   lambda q: gdn.paged_attn(q[:, 0], kc, vc, table, lens + 1)[:, None])
        lens.add_(1)
        return y
    outs = [y, token(xd[:, pre:pre + 1])]
    torch.cuda.synchronize()
    monkeypatch.setenv("GDN_DEBUG", "0")       # looking at lengths would wait inside the capture
    held = {n: t.clone() for n, t in states.items()}
    buf, graph = xd[:, pre + 1:pre + 2].clone(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = token(buf)
    for n, t in states.items():                # (capturing runs nothing)
        assert torch.equal(t, held[n])
    for t in range(pre + 1, T):
        buf.copy_(xd[:, t:t + 1])
        graph.replay()
        outs.append(out.clone())
    torch.cuda.synchronize()
    assert int(lens) == T
    # the bar of the float32 delta rule (the layers' products run in float32 as well)
    e = rel_err(torch.cat(outs, 1), want.numpy())
    assert e <= TOL["f32"], e
