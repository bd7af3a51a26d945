"""ctypes binding of the token mixers of include/gdn.h that stand next to the
delta rule: linear attention with a decay for each head, and the append to and
the attention over a paged cache.  As in _binding.py only arguments are
marshalled here; every call needs the library.

q, k and v may be slices of a wider tensor: the last dimension has to be dense,
tokens evenly spaced, and strides multiples of 8 elements."""
from __future__ import annotations

import ctypes
from functools import lru_cache

import torch

from . import _binding as _b
from ._binding import _check, _debug, _on
from ._layer import (_F32, NORMS, QK_INTERLEAVED, QkDesc, _code, _cu, _dense, _device, _heads, _like, _out, _p, _Plan,
                     _run, _words, _workspace)

_i64, _i32, _f32 = ctypes.c_int64, ctypes.c_int32, ctypes.c_float
DECAY_PER_HEAD = 1


class DecayDesc(ctypes.Structure):
    _fields_ = [("batch", _i64), ("seq_len", _i64), ("num_heads", _i64), ("num_v_heads", _i64), ("key_dim", _i64),
                ("value_dim", _i64), ("num_seqs", _i64), ("q_stride", _i64), ("k_stride", _i64), ("v_stride", _i64),
                ("q_head_stride", _i64), ("k_head_stride", _i64), ("v_head_stride", _i64), ("dtype", _i32),
                ("flags", _i32), ("scale", _f32)]


class PagesDesc(ctypes.Structure):
    _fields_ = [("num_seqs", _i64), ("max_pages", _i64), ("pages", _i64), ("page_size", _i64),
                ("k_page_stride", _i64), ("k_token_stride", _i64), ("k_head_stride", _i64),
                ("v_page_stride", _i64), ("v_token_stride", _i64), ("v_head_stride", _i64)]


class PagedAttnDesc(ctypes.Structure):
    _fields_ = [("num_seqs", _i64), ("q_heads", _i64), ("k_heads", _i64), ("head_dim", _i64), ("q_stride", _i64),
                ("q_head_stride", _i64), ("window", _i64), ("dtype", _i32), ("scale", _f32)]


def declare(lib):
    """argtypes of the entry points (called by load())."""
    P, Z, Zp = ctypes.c_void_p, ctypes.c_size_t, ctypes.POINTER(ctypes.c_size_t)
    D, G, A, Q = (ctypes.POINTER(t) for t in (DecayDesc, PagesDesc, PagedAttnDesc, QkDesc))
    for name, args in (
            ("gdn_decay_attn_workspace", [D, _i32, Zp]),
            ("gdn_decay_attn_fwd", [D] + [P] * 9 + [Z, P]),
            ("gdn_decay_attn_bwd", [D] + [P] * 14 + [Z, P]),
            ("gdn_decay_attn_step", [D] + [P] * 7),
            ("gdn_paged_append", [Q, G, P, P, P, _i64, _i64] + [P] * 11),
            ("gdn_paged_attn_workspace", [A, Zp]),
            ("gdn_paged_attn", [A, G] + [P] * 7 + [Z, P])):
        f = getattr(lib, name)
        f.argtypes, f.restype = args, _i32


# ------------------------------------- linear attention with a decay per head
@lru_cache(maxsize=1024)
def _decay_plan(B, T, H, HV, K, V, N, qs, ks, vs, qh, kh, vh, code, flags, scale):
    p = _Plan(DecayDesc(B, T, H, HV, K, V, N, qs, ks, vs, qh, kh, vh, code, flags, scale))
    lib, n = _b.load(), ctypes.c_size_t()
    _check(lib.gdn_decay_attn_workspace(p.at, 0, n))
    p.fwd = n.value
    _check(lib.gdn_decay_attn_workspace(p.at, 1, n))
    p.bwd = n.value
    return p


@lru_cache(maxsize=1024)
def _step_plan(*fields):
    return _Plan(DecayDesc(*fields))


def _decay(q, k, v, g, scale, packed):
    """Checks shared by the entry points (tensors [B, T, heads, width]): the plan and the device."""
    dev, qs, vs = _device(q, "q"), q.shape, v.shape
    if len(qs) != 4 or k.shape != qs or len(vs) != 4 or vs[:2] != qs[:2]:
        raise ValueError("q, k [B, T, H, K] and v [B, T, H_V, V] do not match: %s, %s, %s"
                         % (tuple(qs), tuple(k.shape), tuple(vs)))
    for t, name in ((k, "k"), (v, "v")):
        if t.dtype != q.dtype or t.device != dev:
            raise ValueError("%s must have the type and device of q" % name)
    B, T, H, K = qs
    HV, V = vs[2], vs[3]
    flags = DECAY_PER_HEAD if g.dim() == 1 else 0
    _dense(g, "g", (HV,) if flags else vs[:3], dev)
    (qt, qh), (kt, kh), (vt, vh) = _heads(q, "q"), _heads(k, "k"), _heads(v, "v")
    return _decay_plan(B, T, H, HV, K, V, packed, qt, kt, vt, qh, kh, vh, _code(q, "q"), flags,
                       float(K ** -0.5 if scale is None else scale)), dev


def decay_attn_fwd(q, k, v, g, scale=None, h0=None, cu_seqlens=None, output_final_state=True, workspace=None, o=None,
                   ht=None, stream=None):
    """gdn_decay_attn_fwd: S_t = exp(g_t) S_{t-1} + k_t v_t^T, o_t = scale q_t
    S_t over q, k [B, T, H, K] and v [B, T, H_V, V]; g [B, T, H_V] float32, or
    [H_V] for one gate of each head.  scale defaults to K^-0.5.  Returns (o,
    ht): the outputs in q's type and the final states [N, H_V, K, V] float32
    (None unless output_final_state)."""
    lib = _b.load()
    packed = _cu(cu_seqlens, _device(q, "q"))
    p, dev = _decay(q, k, v, g, scale, packed)
    sh = v.shape
    ends = (packed or sh[0], sh[2], q.shape[3], sh[3])
    if h0 is not None:
        _dense(h0, "h0", ends, dev)
    if ht is not None:
        _dense(ht, "ht", ends, dev)
    if o is not None:
        _dense(o, "o", sh, dev, q.dtype)
    with _on(stream):   # allocated on the kernels' stream (see chunk_fwd)
        if o is None:
            o = _like(v)
        if not output_final_state:
            ht = None
        elif ht is None:
            ht = v.new_empty(ends, dtype=_F32)
        workspace, have = _workspace(workspace, p.fwd, dev, v)
    _run(lib.gdn_decay_attn_fwd, dev, stream, p.at, q.data_ptr(), k.data_ptr(), v.data_ptr(), g.data_ptr(), _p(h0),
         _p(cu_seqlens), o.data_ptr(), _p(ht), _p(workspace), have)
    _words(workspace, dev, stream, packed)
    return o, ht


def decay_attn_bwd(q, k, v, g, do, scale=None, h0=None, dht=None, cu_seqlens=None, want_dh0=True, out=None,
                   workspace=None, stream=None):
    """gdn_decay_attn_bwd: gradients of <do, o> + <dht, ht> of decay_attn_fwd.
    Returns a dict dq, dk, dv (dense, q's type), dg (the shape of g) and dh0
    (None unless want_dh0), float32.  `out` may supply outputs."""
    lib = _b.load()
    packed = _cu(cu_seqlens, _device(q, "q"))
    p, dev = _decay(q, k, v, g, scale, packed)
    qs, vs = q.shape, v.shape
    ends = (packed or vs[0], vs[2], qs[3], vs[3])
    _dense(do, "do", vs, dev, q.dtype)
    if h0 is not None:
        _dense(h0, "h0", ends, dev)
    if dht is not None:
        _dense(dht, "dht", ends, dev)
    out = dict(out or {})
    with _on(stream):   # allocated on the kernels' stream (see chunk_fwd)
        dq, dk = _out(out, "dq", qs, q.dtype, dev, q), _out(out, "dk", qs, q.dtype, dev, k)
        dv, dg = _out(out, "dv", vs, q.dtype, dev, do), _out(out, "dg", g.shape, _F32, dev, g)
        if not want_dh0:
            out["dh0"] = None
        dh0 = _out(out, "dh0", ends, _F32, dev, v if dht is None else dht) if want_dh0 else None
        workspace, have = _workspace(workspace, p.bwd, dev, v)
    _run(lib.gdn_decay_attn_bwd, dev, stream, p.at, q.data_ptr(), k.data_ptr(), v.data_ptr(), g.data_ptr(), _p(h0),
         _p(cu_seqlens), do.data_ptr(), _p(dht), dq, dk, dv, dg, dh0, _p(workspace), have)
    _words(workspace, dev, stream, packed)
    return out


def _rows(t, name):
    """(stride, head stride) of t [N, H, W]; (0, 0) when dense."""
    return (0, 0) if t.is_contiguous() else _heads(t[:, None], name)


def decay_attn_step(q, k, v, g, state, scale=None, o=None, stream=None):
    """gdn_decay_attn_step: one token of N sequences, q, k [N, H, K] and v [N,
    H_V, V]; g [N, H_V] or [H_V]; state [N, H_V, K, V] float32 is updated in
    place.  Returns o [N, H_V, V]."""
    lib = _b.load()
    dev, qs, vs = _device(q, "q"), q.shape, v.shape
    if len(qs) != 3 or k.shape != qs or len(vs) != 3 or vs[0] != qs[0]:
        raise ValueError("q, k [N, H, K] and v [N, H_V, V] do not match: %s, %s, %s" % (tuple(qs), tuple(k.shape), tuple(vs)))
    if k.dtype != q.dtype or v.dtype != q.dtype or k.device != dev or v.device != dev:
        raise ValueError("k and v must have the type and device of q")
    if state is None:
        raise ValueError("state is required")
    N, H, K = qs
    HV, V = vs[1], vs[2]
    _dense(state, "state", (N, HV, K, V), dev)
    flags = DECAY_PER_HEAD if g.dim() == 1 else 0
    _dense(g, "g", (HV,) if flags else (N, HV), dev)
    if o is not None:
        _dense(o, "o", vs, dev, q.dtype)
    else:
        with _on(stream):   # allocated on the kernel's stream (see chunk_fwd)
            o = _like(v)
    (qt, qh), (kt, kh), (vt, vh) = _rows(q, "q"), _rows(k, "k"), _rows(v, "v")
    p = _step_plan(N, 1, H, HV, K, V, 0, qt, kt, vt, qh, kh, vh, _code(q, "q"), flags, K ** -0.5 if scale is None else float(scale))
    _run(lib.gdn_decay_attn_step, dev, stream, p.at, q.data_ptr(), k.data_ptr(), v.data_ptr(), g.data_ptr(),
         state.data_ptr(), o.data_ptr())
    return o


# ------------------------------------------------------------- paged cache
@lru_cache(maxsize=1024)
def _pages_plan(*fields):
    return _Plan(PagesDesc(*fields))


@lru_cache(maxsize=1024)
def _append_plan(*fields):
    return _Plan(QkDesc(*fields))


@lru_cache(maxsize=1024)
def _attn_plan(*fields):
    p = _Plan(PagedAttnDesc(*fields))
    n = ctypes.c_size_t()
    _check(_b.load().gdn_paged_attn_workspace(p.at, n))
    p.fwd = n.value
    return p


def _pages(k_cache, v_cache, page_table, lens, like, heads, D, dev):
    """Checks of a cache [pages, page_size, heads, D] and its table: the plan of gdn_pages."""
    sh, ks, vs, ts, dt = k_cache.shape, k_cache.stride(), v_cache.stride(), page_table.shape, like.dtype
    if len(sh) != 4 or v_cache.shape != sh or sh[2] != heads or sh[3] != D:
        raise ValueError("k_cache and v_cache must be [pages, page_size, %d, %d], got %s, %s"
                         % (heads, D, tuple(sh), tuple(v_cache.shape)))
    if k_cache.dtype is not dt or v_cache.dtype is not dt or k_cache.device != dev or v_cache.device != dev:
        raise ValueError("k_cache and v_cache must have the type and device of the activations")
    if ks[3] != 1 or vs[3] != 1:
        raise ValueError("k_cache and v_cache must be dense in their last dimension")
    if len(ts) != 2:
        raise ValueError("page_table must be [N, max_pages], got %s" % (tuple(ts),))
    N, M = ts
    _dense(page_table, "page_table", ts, dev, torch.int32)
    _dense(lens, "lens", (N,), dev, torch.int64)
    return _pages_plan(N, M, sh[0], sh[1], ks[0], ks[1], ks[2], vs[0], vs[1], vs[2]), N


def _look(k_cache, page_table, lens, stream, dev, T=None, cu_seqlens=None, window=0):
    """With GDN_DEBUG set: raise where a position in use has no page: T tokens (or a packed
    sequence's) from lens on, or without T the last `window` before lens (0: all)."""
    if not _debug():
        return
    (stream or torch.cuda.current_stream(dev)).synchronize()
    table, n, P = page_table.cpu(), lens.cpu(), k_cache.shape[1]
    cap = table.shape[1] * P
    new = 0 if T is None else T if cu_seqlens is None else (cu_seqlens[1:] - cu_seqlens[:-1]).cpu()
    if bool(((n < 0) | (n > cap) | (n + new > cap)).any()):
        raise ValueError("lens must be in 0 .. %d with the new tokens" % cap)
    first, end = (n, n + new) if T is not None else ((n - window).clamp(min=0) if window > 0 else 0 * n, n)
    at = torch.arange(table.shape[1])[None] * P
    used = (at < end[:, None]) & (at + P > first[:, None]) & (first < end)[:, None]
    if bool((used & ((table < 0) | (table >= k_cache.shape[0]))).any()):
        raise ValueError("page_table holds a page outside the cache")


def paged_append(q, k, v, k_cache, v_cache, page_table, lens, inv_freq=None, positions=None, cu_seqlens=None,
                 norm="none", eps=1e-6, q_weight=None, k_weight=None, weight_offset=0.0, interleaved=False,
                 q_out=None, stream=None):
    """gdn_paged_append: k [B, T, Hk, D], normed and rotated as by
    qk_norm_rope, and v [B, T, Hk, D] go to positions lens[n] + t of a cache
    [pages, page_size, Hk, D] (each of k_cache and v_cache, any strides but a
    dense last dimension) through page_table [N, max_pages] int32; lens [N]
    int64 (not changed).  Sequence n is batch row n, or with cu_seqlens [N + 1]
    the n-th packed one.  `positions` [B, T] int64 for the rotation (None:
    lens[n] + t).  q [B, T, Hq, D] is normed and rotated alike; returns it
    (None for q None).  With GDN_DEBUG set, lengths and the pages of the
    positions written are looked at and a ValueError raised for those outside
    the cache, which are otherwise left out."""
    lib = _b.load()
    dev, ks = _device(k, "k"), k.shape
    if len(ks) != 4 or v.shape != ks:
        raise ValueError("k and v must have one shape [B, T, Hk, D], got %s, %s" % (tuple(ks), tuple(v.shape)))
    if v.dtype != k.dtype or v.device != dev:
        raise ValueError("v must have the type and device of k")
    B, T, Hk, D = ks
    Hq, qt, qh = 1, 0, 0
    if q is not None:
        if q.dim() != 4 or q.shape[:2] != ks[:2] or q.shape[3] != D or q.dtype != k.dtype or q.device != dev:
            raise ValueError("q must be [%d, %d, Hq, %d] with the type and device of k, got %s" % (B, T, D, tuple(q.shape)))
        Hq, (qt, qh) = q.shape[2], _heads(q, "q")
    if norm not in NORMS:
        raise ValueError("norm must be one of %s" % sorted(NORMS))
    R = 0
    if inv_freq is not None:
        _dense(inv_freq, "inv_freq", (inv_freq.numel(),), dev, torch.float64)
        R = 2 * inv_freq.numel()
    if positions is not None:
        _dense(positions, "positions", (B, T), dev, torch.int64)
    for w, name in ((q_weight, "q_weight"), (k_weight, "k_weight")):
        if w is not None:
            _dense(w, name, (D,), dev)
    c, N = _pages(k_cache, v_cache, page_table, lens, k, Hk, D, dev)
    packed = _cu(cu_seqlens, dev)
    if (packed or B) != N or (packed and B != 1):
        raise ValueError("page_table has %d rows for %d sequences" % (N, packed or B))
    (kt, kh), (vt, vh) = _heads(k, "k"), _heads(v, "v")
    p = _append_plan(B, T, Hq, Hk, D, R, qt, kt, qh, kh, _code(k, "k"), NORMS[norm],
                     QK_INTERLEAVED if interleaved else 0, float(eps), float(weight_offset))
    if q is None:
        q_out = None
    elif q_out is not None:
        _dense(q_out, "q_out", q.shape, dev, q.dtype)
    else:
        with _on(stream):   # allocated on the kernel's stream (see chunk_fwd)
            q_out = _like(q)
    _look(k_cache, page_table, lens, stream, dev, T=T, cu_seqlens=cu_seqlens)
    _run(lib.gdn_paged_append, dev, stream, p.at, c.at, _p(q), k.data_ptr(), v.data_ptr(), vt, vh, _p(q_weight),
         _p(k_weight), _p(inv_freq), _p(positions), _p(cu_seqlens), page_table.data_ptr(), lens.data_ptr(), _p(q_out),
         k_cache.data_ptr(), v_cache.data_ptr())
    return q_out


def _attn(q, k_cache, v_cache, page_table, lens, scale, window):
    dev = _device(q, "q")
    if q.dim() != 3:
        raise ValueError("q must be [N, Hq, D], got %s" % (tuple(q.shape),))
    n, Hq, D = q.shape
    Hk = k_cache.shape[2] if k_cache.dim() == 4 else 0
    c, N = _pages(k_cache, v_cache, page_table, lens, q, Hk, D, dev)
    if n != N:
        raise ValueError("page_table has %d rows for %d sequences" % (N, n))
    qt, qh = _rows(q, "q") if n else (0, 0)
    return _attn_plan(N, Hq, Hk, D, qt, qh, int(window), _code(q, "q"),
                      float(D ** -0.5 if scale is None else scale)), c, dev


def paged_attn_workspace(q, k_cache, v_cache, page_table, lens, stream=None):
    """A workspace for paged_attn calls of these shapes (one for each that may overlap)."""
    p, _, dev = _attn(q, k_cache, v_cache, page_table, lens, None, 0)
    with _on(stream):
        return _workspace(None, p.fwd, dev, q)[0]


def paged_attn(q, k_cache, v_cache, page_table, lens, scale=None, window=0, o=None, workspace=None, stream=None):
    """gdn_paged_attn: attention of one token of N sequences, q [N, Hq, D],
    over positions max(0, lens[n] - window) .. lens[n] - 1 (window 0: all) of
    their cached tokens (see paged_append), Hq a multiple of Hk.  lens [N]
    int64 counts the new token too where its key is to be seen.  scale
    defaults to D^-0.5.  Returns o [N, Hq, D]; zeros where lens is 0.  With
    GDN_DEBUG set, lengths and pages (of the positions attended to) outside
    the cache raise a ValueError; they are otherwise left out."""
    lib = _b.load()
    p, c, dev = _attn(q, k_cache, v_cache, page_table, lens, scale, window)
    if o is not None:
        _dense(o, "o", q.shape, dev, q.dtype)
    with _on(stream):   # allocated on the kernels' stream (see chunk_fwd)
        if o is None:
            o = _like(q)
        workspace, have = _workspace(workspace, p.fwd, dev, q)
    _look(k_cache, page_table, lens, stream, dev, window=int(window))
    _run(lib.gdn_paged_attn, dev, stream, p.at, c.at, q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(),
         page_table.data_ptr(), lens.data_ptr(), o.data_ptr(), _p(workspace), have)
    return o
