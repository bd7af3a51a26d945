"""Plain 64-bit implementations of the layer operators (CPU torch), with bounds
on what 32-bit arithmetic may lose, for the tests of the HIP kernels.

Every function returns values and, under the same names, error bounds: a
bound follows the computation with absolute values, charging each 32-bit
operation a few half units in the last place (U = 2^-24; C counts them), and
check() adds half a step of the output's own type.  The kernels may order the
sums and products of a recurrence differently; each step of any order costs
the same roundings, so the bounds hold for all of them."""
from __future__ import annotations

import torch

F64 = torch.float64
U = 2.0 ** -24
C = 8.0            # half units charged to each 32-bit step (exp, log1p, division: up to 4)


def f64(t):
    return None if t is None else t.detach().cpu().to(F64)


def spans(x, cu):
    """(batch index, first, last) of every sequence of x [B, T, ...]."""
    if cu is None:
        return [(b, 0, x.shape[1]) for b in range(x.shape[0])]
    cu = cu.tolist()
    return [(0, cu[i], cu[i + 1]) for i in range(len(cu) - 1)]


def check(got, want, err, what):
    """|got - want| within err plus half a step of got's type (and of the smallest normal)."""
    g, half = f64(got), torch.finfo(got.dtype).eps / 2
    assert tuple(g.shape) == tuple(want.shape), (what, g.shape, want.shape)
    lim = err * (1 + half) + half * want.abs() + torch.finfo(torch.float32).tiny
    bad = ~((g - want).abs() <= lim)
    same = (g == want) | (torch.isnan(g) & torch.isnan(want))
    bad &= ~same
    if bad.any():
        i = tuple(bad.nonzero()[0].tolist())
        raise AssertionError("%s%s: got %.9g, want %.9g, bound %.3g; %d of %d off, worst %.3g of the bound"
                             % (what, i, g[i], want[i], lim[i], int(bad.sum()), bad.numel(),
                                ((g - want).abs() / lim)[bad].max()))


def check_all(got, want, err, what=""):
    for name, w in want.items():
        if w is None:
            assert got.get(name) is None, name
        else:
            check(got[name], w, err[name], what + " " + name)


# ---------------------------------------------------------------- linrec
def gates(g, A_log=None, dt_bias=None):
    """log a, its slope in g, and the bound on log a."""
    g = f64(g)
    if A_log is None:
        return g, torch.ones_like(g), torch.zeros_like(g)
    rate, z = -torch.exp(f64(A_log)), g + f64(dt_bias)
    sp = torch.logaddexp(z, torch.zeros_like(z))
    # z is rounded once: softplus moves by at most sigmoid(z) |z| U
    sg = torch.sigmoid(z)
    return rate * sp, rate * sg, -rate * U * (C * sp + 2 * sg * z.abs())


def linrec(x, g, h0=None, cu=None, normalize=False, A_log=None, dt_bias=None, dy=None, dht=None):
    """Values and bounds: y, ht and, with dy, dx, dg, dh0 (dA_log, ddt_bias)."""
    x, h0, dy, dht = f64(x), f64(h0), f64(dy), f64(dht)
    la, slope, ela = gates(g, A_log, dt_bias)
    a = torch.exp(la)
    ra = ela + C * U                                   # relative error of a
    m = torch.sqrt(-torch.expm1(2 * la)) if normalize else torch.ones_like(a)
    # d ln m / d log a = -a^2 / m^2; the 32-bit formula itself is relatively exact to C U
    rm = torch.where(m > 0, ela * a * a / (m * m), torch.zeros_like(m)) + C * U if normalize else 0 * a
    u = m * x
    D, sp = x.shape[-1], spans(x, cu)
    want = dict(y=torch.zeros_like(x), ht=torch.zeros(len(sp), D, dtype=F64))
    err = dict(y=torch.zeros_like(x), ht=torch.zeros(len(sp), D, dtype=F64))
    prev, eprev, aprev = torch.zeros_like(x), torch.zeros_like(x), torch.zeros_like(x)
    for n, (b, s, e) in enumerate(sp):
        h = h0[n].clone() if h0 is not None else torch.zeros(D, dtype=F64)
        habs, eh = h.abs(), torch.zeros(D, dtype=F64)
        for t in range(s, e):
            prev[b, t], aprev[b, t], eprev[b, t] = h, habs, eh
            eh = a[b, t] * (eh + ra[b, t] * habs) + u[b, t].abs() * (rm[b, t] + U)
            habs = a[b, t] * habs + u[b, t].abs()
            eh = eh + C * U * habs
            h = a[b, t] * h + u[b, t]
            want["y"][b, t], err["y"][b, t] = h, eh
        want["ht"][n], err["ht"][n] = h, eh
    if dy is None:
        return want, err
    dx, edx, dla, edla = (torch.zeros_like(x) for _ in range(4))
    tabs = torch.zeros_like(x)
    want["dh0"], err["dh0"] = torch.zeros_like(want["ht"]), torch.zeros_like(want["ht"])
    for n, (b, s, e) in enumerate(sp):
        c = dht[n].clone() if dht is not None else torch.zeros(D, dtype=F64)
        cabs, ec = c.abs(), torch.zeros(D, dtype=F64)
        for t in range(e - 1, s - 1, -1):
            dh, dabs = dy[b, t] + c, dy[b, t].abs() + cabs
            ed = ec + C * U * dabs
            dx[b, t] = m[b, t] * dh
            edx[b, t] = m[b, t] * (ed + (rm[b, t] + U) * dabs)
            c, cabs = a[b, t] * dh, a[b, t] * dabs
            ec = a[b, t] * ed + ra[b, t] * cabs
            dla[b, t] = c * prev[b, t]
            edla[b, t] = ec * aprev[b, t] + cabs * (eprev[b, t] + C * U * aprev[b, t])
            tabs[b, t] = cabs * aprev[b, t]
            if normalize:
                q = torch.where(m[b, t] > 0, a[b, t] / m[b, t], torch.zeros_like(c))
                dla[b, t] -= c * x[b, t] * q
                edla[b, t] += x[b, t].abs() * q * (ec + cabs * (ra[b, t] + rm[b, t] + C * U))
                tabs[b, t] += cabs * x[b, t].abs() * q
        want["dh0"][n], err["dh0"][n] = c, ec
    edla += C * U * tabs
    want["dx"], err["dx"] = dx, edx
    dg = dla * slope
    # the slope moves by its own roundings and by that of z (|sigmoid'| <= sigmoid)
    z = f64(g) + f64(dt_bias) if A_log is not None else torch.zeros_like(x)
    edg = slope.abs() * (edla + tabs * U * (C + 2 * z.abs())) if A_log is not None else edla
    want["dg"], err["dg"] = dg, edg
    if A_log is not None:
        k = x.shape[0] * x.shape[1]
        want["dA_log"], want["ddt_bias"] = (dla * la).sum((0, 1)), dg.sum((0, 1))
        err["dA_log"] = (edla * la.abs() + tabs * (ela + (C + k) * U * la.abs())).sum((0, 1))
        err["ddt_bias"] = (edg + k * U * (tabs * slope.abs())).sum((0, 1))
    return want, err


# ---------------------------------------------------------------- q/k norm
def _pairs(x, R, inter):
    return (x[..., 0:R:2], x[..., 1:R:2]) if inter else (x[..., :R // 2], x[..., R // 2:R])


def _spin(x, c, s, R, inter):
    if R == 0:
        return x.clone()
    a, b = _pairs(x, R, inter)
    u, v = a * c - b * s, b * c + a * s
    head = torch.stack([u, v], -1).flatten(-2) if inter else torch.cat([u, v], -1)
    return torch.cat([head, x[..., R:]], -1)


def qk(t, inv_freq, positions, norm, eps, w, offset, inter, dout=None):
    """One of q, k [B, T, H, D]: dict out (and dx, dw) with bounds."""
    x = f64(t)
    B, T, _, D = x.shape
    R = 0 if inv_freq is None else 2 * inv_freq.numel()
    pos = torch.arange(T).expand(B, T) if positions is None else positions.cpu()
    th = pos.to(F64)[..., None, None] * f64(inv_freq) if R else torch.zeros(B, T, 1, 0, dtype=F64)
    c, s = torch.cos(th), torch.sin(th)
    gain = f64(w) + offset if w is not None else torch.ones(D, dtype=F64)
    n = D if norm == "rms" else 1
    ss = (x * x).sum(-1, keepdim=True) / n + eps
    r = torch.ones_like(ss) if norm == "none" else 1 / torch.sqrt(ss)
    y = x * r * gain
    # sum of squares: D roundings at worst, halved by the root; then norm and gain
    ry = (0 if norm == "none" else D / 2 + C) * U + C * U
    mag = (x * r).abs() * (f64(w).abs() + abs(offset) if w is not None else 1)
    one = torch.ones_like(c)
    # a rotated element is a sum of two products; cos and sin are good to C U, the angle in
    # turns to half a unit of 1/2, that is 2 pi 2^-25 < 4 U
    both = _spin(mag, one, -one, R, inter)          # |a| + |b| at the first of a pair
    if R:
        a, b = _pairs(mag, R, inter)
        tot = torch.stack([a + b, a + b], -1).flatten(-2) if inter else torch.cat([a + b, a + b], -1)
        both = torch.cat([tot, mag[..., R:]], -1)
    want, err = dict(out=_spin(y, c, s, R, inter)), dict(out=both * (ry + (2 * C + 4) * U))
    if dout is None:
        return want, err
    d = f64(dout)
    dn = _spin(d, c, -s, R, inter)
    da = d.abs()
    if R:
        a, b = _pairs(da, R, inter)
        da = torch.cat([torch.stack([a + b, a + b], -1).flatten(-2) if inter else torch.cat([a + b, a + b], -1), da[..., R:]], -1)
    edn = da * (2 * C + 4) * U
    if w is not None:
        want["dw"] = (dn * x * r).sum((0, 1, 2))
        k = x.shape[0] * x.shape[1] * x.shape[2]
        err["dw"] = ((edn + da * (ry + (C + k) * U)) * (x * r).abs()).sum((0, 1, 2))
    dn = dn * gain
    gm = mag / (x * r).abs().clamp(min=1e-300) if w is not None else 1
    gm = (f64(w).abs() + abs(offset)) if w is not None else torch.ones(D, dtype=F64)
    dabs, edn = da * gm, edn * gm + da * gm * C * U
    dx, edx = r * dn, r * (edn + dabs * (ry + C * U))
    if norm != "none":
        dot, dotabs = (x * dn).sum(-1, keepdim=True), (x.abs() * dabs).sum(-1, keepdim=True)
        edot = (x.abs() * edn).sum(-1, keepdim=True) + D * U * dotabs
        k3 = r ** 3 / n
        dx = dx - x * k3 * dot
        edx = edx + x.abs() * k3 * (edot + dotabs * (3 * ry + C * U))
    want["dx"], err["dx"] = dx, edx
    return want, err


# ------------------------------------------------------------- short conv
def conv(x, w, b=None, s0=None, cu=None, silu=True, dy=None, dst=None):
    """Values and bounds: y, st and, with dy, dx, ds0, dweight (dbias)."""
    x, w, b, s0, dy, dst = (f64(t) for t in (x, w, b, s0, dy, dst))
    D, W = w.shape
    sp = spans(x, cu)
    N = len(sp)
    want = dict(y=torch.zeros_like(x), st=torch.zeros(N, W - 1, D, dtype=F64))
    err = dict(y=torch.zeros_like(x), st=torch.zeros(N, W - 1, D, dtype=F64))
    if dy is not None:
        for name, like in (("dx", x), ("ds0", want["st"]), ("dweight", w)) + ((("dbias", w[:, 0]),) if b is not None else ()):
            want[name], err[name] = torch.zeros_like(like), torch.zeros_like(like)
        mags = {k: torch.zeros_like(v) for k, v in want.items() if k in ("dweight", "dbias")}
    for n, (bi, s, e) in enumerate(sp):
        before = s0[n] if s0 is not None else torch.zeros(W - 1, D, dtype=F64)
        win = torch.cat([before, x[bi, s:e]])                 # rows: positions -(W-1) ..
        L = e - s
        z = sum(win[j:j + L] * w[:, j] for j in range(W)) + (b if b is not None else 0)
        za = sum(win[j:j + L].abs() * w[:, j].abs() for j in range(W)) + (b.abs() if b is not None else 0)
        ez = (W + 1) * U * za
        sg = torch.sigmoid(z)
        if silu:                                               # |silu'| < 1.1; sigmoid and product: C U
            want["y"][bi, s:e], err["y"][bi, s:e] = z * sg, 1.1 * ez + C * U * (z * sg).abs()
        else:
            want["y"][bi, s:e], err["y"][bi, s:e] = z, ez
        want["st"][n] = win[L:]
        if dy is None:
            continue
        sl = sg * (1 + z * (1 - sg)) if silu else torch.ones_like(z)
        dz = dy[bi, s:e] * sl
        # |silu''| <= 1/2; the slope's terms are sg and z sg (1 - sg), each to C U
        ed = dy[bi, s:e].abs() * (0.5 * ez + C * U * (sg + z.abs() * sg * (1 - sg)) + U * sl.abs()) if silu else 0 * ez
        dwin, edwin, mwin = (torch.zeros_like(win) for _ in range(3))
        for j in range(W):
            dwin[j:j + L] += dz * w[:, j]
            edwin[j:j + L] += ed * w[:, j].abs()
            mwin[j:j + L] += (dz * w[:, j]).abs()
            want["dweight"][:, j] += (dz * win[j:j + L]).sum(0)
            err["dweight"][:, j] += (ed * win[j:j + L].abs()).sum(0)
            mags["dweight"][:, j] += (dz * win[j:j + L]).abs().sum(0)
        if dst is not None:
            dwin[L:] += dst[n]
            mwin[L:] += dst[n].abs()
        edwin += (W + 2) * U * mwin
        want["dx"][bi, s:e], err["dx"][bi, s:e] = dwin[W - 1:], edwin[W - 1:]
        want["ds0"][n], err["ds0"][n] = dwin[:W - 1], edwin[:W - 1]
        if b is not None:
            want["dbias"] += dz.sum(0)
            err["dbias"] += ed.sum(0)
            mags["dbias"] += dz.abs().sum(0)
    if dy is not None:
        k = x.shape[0] * x.shape[1]
        for name, mg in mags.items():
            err[name] += (k + 2) * U * mg
    return want, err
