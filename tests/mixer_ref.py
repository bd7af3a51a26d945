"""Plain 64-bit implementations of the token mixers (CPU torch), with bounds on
what the kernels' arithmetic may lose; check() of layer_ref adds half a step of
the output's own type.

A bound follows the computation with absolute values.  32-bit operations cost a
few half units each (U = 2^-24, C of them), a dot product of n terms n more in
the worst order.  With bf16 two factors of each product that makes an output of
that type are rounded to it: the weights of the pairs of a chunk and the state
(or the weights of a softmax, in two parts), by half a step, 2^-8, at most."""
from __future__ import annotations

import torch

from layer_ref import C, F64, U, f64, spans

HALF = {torch.float32: 0.0, torch.bfloat16: 2.0 ** -8}


def _sum_heads(x, H):
    return x.unflatten(-2, (H, x.shape[-2] // H)).sum(-2)


def decay(q, k, v, g, scale=None, h0=None, cu=None, do=None, dht=None):
    """Values and bounds of decay_attn_fwd: o, ht and, with do, dq, dk, dv, dg, dh0."""
    half, H = HALF[q.dtype], q.shape[2]
    q, k, v, h0, do, dht = (f64(t) for t in (q, k, v, h0, do, dht))
    HV, K, V = v.shape[2], q.shape[3], v.shape[3]
    m, per_head = HV // H, g.dim() == 1
    scale = K ** -0.5 if scale is None else scale
    q, k = q.repeat_interleave(m, 2), k.repeat_interleave(m, 2)
    ga = f64(g).expand(v.shape[:3])
    a = torch.exp(ga)[..., None, None]
    # exp(g) over any stretch: the sums of the gates are good to a few units of the gate itself
    ra = torch.where(a > 0, (ga.abs().clamp(max=200.0) + 2 * C)[..., None, None] * U, 0)
    sp = spans(v, cu)
    N = len(sp)
    want = dict(o=torch.zeros_like(v), ht=torch.zeros(N, HV, K, V, dtype=F64))
    err = {n: torch.zeros_like(t) for n, t in want.items()}
    names = dict(dq=q, dk=k, dv=v, dg=ga) if do is not None else {}
    for n, t in names.items():
        want[n], err[n] = torch.zeros(t.shape, dtype=F64), torch.zeros(t.shape, dtype=F64)
    if do is not None:
        want["dh0"], err["dh0"] = torch.zeros_like(want["ht"]), torch.zeros_like(want["ht"])
    outer = lambda x, y: x[..., None] * y[..., None, :]  # noqa: E731
    for n, (b, s, e) in enumerate(sp):
        S = h0[n].clone() if h0 is not None else torch.zeros(HV, K, V, dtype=F64)
        A, E = S.abs(), torch.zeros_like(S)                    # sums of absolute values, and the bound
        before, noise = [], torch.zeros(e - s, HV, dtype=F64)
        for t in range(s, e):
            before.append(S)
            add, mag = outer(k[b, t], v[b, t]), outer(k[b, t].abs(), v[b, t].abs())
            S = a[b, t] * S + add
            E = a[b, t] * (E + ra[b, t] * A) + 2 * C * U * mag
            A = a[b, t] * A + mag
            E = E + C * U * A

            def read(x, X, Xe, n_):                            # x X and its bound
                xa = x.abs()[..., None]
                return (x[..., None] * X).sum(-2), (xa * Xe).sum(-2), (xa * A if X is S else xa * A.mT).sum(-2), n_
            o, oe, om, _ = read(q[b, t], S, E, K)
            want["o"][b, t] = scale * o
            err["o"][b, t] = scale * (oe + (half + (K + 64 + C) * U) * om)
            if do is not None:
                da = do[b, t].abs()
                want["dq"][b, t] = scale * (S * do[b, t][:, None]).sum(-1)
                dm = (A * da[:, None]).sum(-1)
                err["dq"][b, t] = scale * ((E * da[:, None]).sum(-1) + (half + (V + 64 + C) * U) * dm)
                # a token's term of dg's running sum
                qa = q[b, t].abs()
                noise[t - s] += scale * ((qa * (E * da[:, None]).sum(-1)).sum(-1) + (K + V + 64 + 2 * C) * U * (qa * dm).sum(-1))
        want["ht"][n], err["ht"][n] = S, E
        if do is None:
            continue
        D = dht[n].clone() if dht is not None else torch.zeros_like(S)
        B, F = D.abs(), torch.zeros_like(D)
        tail = (E * B + K * V * U * A * B).sum((-1, -2))       # the segment's end: <S, E>
        for t in range(e - 1, s - 1, -1):
            mag = scale * outer(q[b, t].abs(), do[b, t].abs())
            D, B = D + scale * outer(q[b, t], do[b, t]), B + mag
            F = F + 2 * C * U * mag + C * U * B
            ka, va = k[b, t].abs(), v[b, t].abs()
            want["dk"][b, t] = (D * v[b, t][:, None]).sum(-1)
            dm = (B * va[:, None]).sum(-1)
            err["dk"][b, t] = (F * va[:, None]).sum(-1) + (half + (V + 64 + C) * U) * dm
            want["dv"][b, t] = (D * k[b, t][..., None]).sum(-2)
            err["dv"][b, t] = (F * ka[..., None]).sum(-2) + (half + (K + 64 + C) * U) * (B * ka[..., None]).sum(-2)
            want["dg"][b, t] = (a[b, t] * before[t - s] * D).sum((-1, -2))
            noise[t - s] += (ka * (F * va[:, None]).sum(-1)).sum(-1) + (K + V + 64 + 2 * C) * U * (ka * dm).sum(-1)
            D, F, B = a[b, t] * D, a[b, t] * (F + ra[b, t] * B), a[b, t] * B
        want["dh0"][n], err["dh0"][n] = D, F
        # the running sum starts at a segment's end, whose <S, E> is as good as the noise of a token there
        err["dg"][b, s:e] = noise.flip(0).cumsum(0).flip(0) + tail + noise.max(0).values * (K + V) if e > s else 0
    if do is not None:
        for n in ("dq", "dk"):
            big = err[n] + m * U * want[n].abs()
            want[n], err[n] = _sum_heads(want[n], H), _sum_heads(big, H)
        if per_head:
            T = ga.shape[0] * ga.shape[1]
            err["dg"] = (err["dg"] + T * U * want["dg"].abs()).sum((0, 1))
            want["dg"] = want["dg"].sum((0, 1))
    return want, err


def step(q, k, v, g, state, scale=None):
    """decay_attn_step: o and the new state, with bounds."""
    w, e = decay(q[:, None], k[:, None], v[:, None], g if g.dim() == 1 else g[:, None], scale, state)
    # the step kernel rounds nothing but its output
    K, m = q.shape[-1], v.shape[1] // q.shape[1]
    mag = (q.cpu().to(F64).abs().repeat_interleave(m, 1)[..., None] * (w["ht"].abs() + e["ht"])).sum(-2)
    scale = K ** -0.5 if scale is None else scale
    return dict(o=w["o"][:, 0], state=w["ht"]), dict(o=scale * (K + 2 * C) * U * mag * 2 + scale * e["ht"].sum(-2), state=e["ht"])


def rows(cache, table, n, lo, hi):
    """Tokens lo .. hi - 1 of sequence n that are in the cache [pages, P, H, D]: their rows."""
    P, M = cache.shape[1], table.shape[1]
    got = []
    for t in range(max(lo, 0), min(hi, M * P)):
        pg = int(table[n, t // P])
        if 0 <= pg < cache.shape[0]:
            got.append(cache[pg, t % P])
    return f64(torch.stack(got)) if got else None


def attn(q, kc, vc, table, lens, scale=None, window=0):
    """Values and bounds of paged_attn."""
    parts = 2.0 ** -16 if q.dtype == torch.bfloat16 else 0.0
    q, table, kc, vc = f64(q), table.cpu(), kc.cpu(), vc.cpu()
    N, Hq, D = q.shape
    m = Hq // kc.shape[2]
    scale = D ** -0.5 if scale is None else scale
    want, err = torch.zeros_like(q), torch.zeros_like(q)
    for n, L in enumerate(lens.tolist()):
        lo = max(0, min(L, table.shape[1] * kc.shape[1]) - window) if window else 0
        k, v = rows(kc, table, n, lo, L), rows(vc, table, n, lo, L)
        if k is None:
            continue
        k, v = k.repeat_interleave(m, 1), v.repeat_interleave(m, 1)          # [t, Hq, D]
        x = scale * (q[n] * k).sum(-1)
        p = torch.softmax(x, 0)
        # a score's error moves its weight alike; the largest one that of all others
        ex = (D + 2 * C) * U * abs(scale) * (q[n].abs() * k.abs()).sum(-1) + 2 * U * (x - x.max(0).values).abs().clamp(max=200.0)
        mag = (p[..., None] * v.abs()).sum(0)
        want[n] = (p[..., None] * v).sum(0)
        err[n] = (p[..., None] * v.abs() * (ex[..., None] + ex.max(0).values[:, None])).sum(0) * 1.1 \
            + (parts + (k.shape[0] + 4 * C) * U) * (mag + want[n].abs())
    return want, err
