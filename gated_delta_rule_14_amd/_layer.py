"""ctypes binding of the layer operators of include/gdn.h: the gated linear
recurrence, the q/k norm with rotation and the short convolution.  As in
_binding.py only arguments are marshalled here; every call needs the library.

Activations may be slices of a wider tensor: the last dimension (for q and k
the last one) has to be dense, and consecutive tokens evenly spaced."""
from __future__ import annotations

import ctypes

import torch

from . import _binding as _b
from ._binding import ACT_GATE, Activation, GdnError, _check, _debug, _dtype_code, _on

_i64, _i32, _f32 = ctypes.c_int64, ctypes.c_int32, ctypes.c_float
LINREC_NORMALIZE = 1
NORMS = {"none": 0, "l2": 1, "rms": 2}
QK_INTERLEAVED = 1
CONV_SILU = 1


class LinrecDesc(ctypes.Structure):
    _fields_ = [("batch", _i64), ("seq_len", _i64), ("channels", _i64), ("num_seqs", _i64),
                ("x_stride", _i64), ("g_stride", _i64), ("y_stride", _i64),
                ("x_dtype", _i32), ("g_dtype", _i32), ("flags", _i32)]


class QkDesc(ctypes.Structure):
    _fields_ = [("batch", _i64), ("seq_len", _i64), ("q_heads", _i64), ("k_heads", _i64),
                ("head_dim", _i64), ("rot_dim", _i64), ("q_stride", _i64), ("k_stride", _i64),
                ("q_head_stride", _i64), ("k_head_stride", _i64), ("dtype", _i32), ("norm", _i32),
                ("flags", _i32), ("eps", _f32), ("weight_offset", _f32)]


class ConvDesc(ctypes.Structure):
    _fields_ = [("batch", _i64), ("seq_len", _i64), ("channels", _i64), ("num_seqs", _i64),
                ("x_stride", _i64), ("y_stride", _i64), ("dtype", _i32), ("width", _i32), ("flags", _i32)]


def declare(lib):
    """argtypes of the layer entry points (called by load())."""
    P, Z = ctypes.c_void_p, ctypes.c_size_t
    L, Q, C, A = (ctypes.POINTER(t) for t in (LinrecDesc, QkDesc, ConvDesc, Activation))
    for name, args in (
            ("gdn_linrec_workspace", [L, _i32, ctypes.POINTER(Z), ctypes.POINTER(_i64)]),
            ("gdn_linrec_fwd", [L, A] + [P] * 8 + [Z, P]),
            ("gdn_linrec_bwd", [L, A] + [P] * 13 + [Z, P]),
            ("gdn_linrec_step", [L, A] + [P] * 5),
            ("gdn_qk_norm_rope", [Q] + [P] * 9),
            ("gdn_qk_norm_rope_bwd_workspace", [Q, ctypes.POINTER(Z)]),
            ("gdn_qk_norm_rope_bwd", [Q] + [P] * 13 + [Z, P]),
            ("gdn_short_conv_workspace", [C, _i32, ctypes.POINTER(Z)]),
            ("gdn_short_conv_fwd", [C] + [P] * 8 + [Z, P]),
            ("gdn_short_conv_bwd", [C] + [P] * 12 + [Z, P]),
            ("gdn_short_conv_step", [C] + [P] * 6)):
        f = getattr(lib, name)
        f.argtypes, f.restype = args, _i32


# ---------------------------------------------------------------- arguments
def _p(t):
    return None if t is None else t.data_ptr()


def _same(dev, **tensors):
    for name, t in tensors.items():
        if t is not None and t.device != dev:
            raise ValueError("%s must be on %s, got %s" % (name, dev, t.device))


def _f32c(t, name, shape, dev):
    """A dense float32 tensor of `shape` (None: absent)."""
    if t is not None:
        if t.dtype != torch.float32:
            raise TypeError("%s must be torch.float32, got %s" % (name, t.dtype))
        _dense(t, name, shape, dev)


def _dense(t, name, shape, dev, dtype=None):
    if t.device != dev:
        raise ValueError("%s must be on %s, got %s" % (name, dev, t.device))
    if dtype is not None and t.dtype != dtype:
        raise TypeError("%s must be %s, got %s" % (name, dtype, t.dtype))
    if tuple(t.shape) != tuple(shape) or not t.is_contiguous():
        raise ValueError("%s must be contiguous with shape %s, got %s" % (name, tuple(shape), tuple(t.shape)))


def _stride(t, name):
    """Elements between the tokens of t [B, T, ...] ([N, ...]: one token each); 0 for dense rows."""
    if t.is_contiguous() or t.numel() == 0:
        return 0
    B, T, s = t.shape[0], t.shape[1], t.stride()
    inner = t[0, 0]
    if inner.dim() == 1 and inner.numel() > 1 and s[-1] != 1:
        raise ValueError("%s must be dense in its last dimension" % name)
    step = (s[0] if B > 1 else inner.numel()) if T == 1 else s[1]
    if (B > 1 and T > 1 and s[0] != T * step) or (inner.dim() == 1 and step < inner.numel()):
        raise ValueError("%s must hold evenly spaced tokens that do not overlap, got strides %s" % (name, s))
    return step


def _device(t, name):
    if not t.is_cuda:
        raise ValueError("%s must be a device tensor" % name)
    return t.device


def _run(fn, dev, stream, *args):
    """Call fn(*args, stream) with dev current; `stream` None: dev's current stream."""
    raw = torch._C._cuda_getCurrentRawStream(dev.index) if stream is None else stream.cuda_stream
    if torch._C._cuda_getDevice() == dev.index:
        _check(fn(*args, raw))
    else:
        with torch.cuda.device(dev):
            _check(fn(*args, raw))


def _workspace(ws, nbytes, dev):
    if nbytes == 0:
        return None, 0
    if ws is None:
        ws = torch.empty(nbytes, dtype=torch.uint8, device=dev)
    else:
        _same(dev, workspace=ws)
        if not ws.is_contiguous():
            raise ValueError("workspace must be contiguous")
    return ws, ws.numel() * ws.element_size()


def _words(ws, dev, stream, packed, waits=False):
    """With GDN_DEBUG set: raise on the check of the offsets (packed) and on a wait that gave up."""
    if ws is None or not (packed or waits) or not _debug():
        return
    (stream or torch.cuda.current_stream(dev)).synchronize()
    bad, wait = ws.view(torch.uint8)[:8].view(torch.int32).cpu().tolist()
    if packed and bad:
        raise GdnError(8, "cu_seqlens must start at 0, never decrease and end at T")
    if waits and wait:
        raise GdnError(7, "a wait between workgroups gave up: wrong results")


def _cu(cu, dev):
    if cu is None:
        return 0
    if cu.dtype != torch.int64:
        raise TypeError("cu_seqlens must be torch.int64, got %s" % cu.dtype)
    if cu.dim() != 1 or cu.numel() < 2 or not cu.is_contiguous() or cu.device != dev:
        raise ValueError("cu_seqlens must be contiguous [N + 1] on %s" % dev)
    return cu.numel() - 1


# ------------------------------------------------- gated linear recurrence
def _linrec(x, g, cu, normalize, A_log, dt_bias, y=None, lead=2):
    dev = _device(x, "x")
    if x.dim() != lead + 1 or g.shape != x.shape:
        raise ValueError("x and g must have one shape %s, got %s and %s"
                         % ("[N, D]" if lead == 1 else "[B, T, D]", tuple(x.shape), tuple(g.shape)))
    if g.device != dev:
        raise ValueError("g must be on %s" % dev)
    if y is not None and (y.shape != x.shape or y.dtype != x.dtype or y.device != dev):
        raise ValueError("y / dy must have the shape, type and device of x")
    D = x.shape[-1]
    if (A_log is None) != (dt_bias is None):
        raise ValueError("A_log and dt_bias come together")
    _f32c(A_log, "A_log", (D,), dev)
    _f32c(dt_bias, "dt_bias", (D,), dev)
    N = _cu(cu, dev)
    if lead == 1:
        x, g, y = x.unsqueeze(1), g.unsqueeze(1), None if y is None else y.unsqueeze(1)
    d = LinrecDesc(x.shape[0], x.shape[1], D, N, _stride(x, "x"), _stride(g, "g"),
                   0 if y is None else _stride(y, "y / dy"), _dtype_code(x), _dtype_code(g),
                   LINREC_NORMALIZE if normalize else 0)
    act = None if A_log is None else Activation(ACT_GATE, A_log.data_ptr(), dt_bias.data_ptr())
    return d, act, dev, N or x.shape[0]


def _linrec_sizes(d, backward):
    lib = _b.load()
    n, rows = ctypes.c_size_t(), _i64()
    _check(lib.gdn_linrec_workspace(d, backward, n, rows))
    return n.value, rows.value


def linrec_states(x, cu_seqlens=None):
    """A buffer for linrec_fwd's `states` (of x [B, T, D]), to be kept for linrec_bwd."""
    dev = _device(x, "x")
    d = LinrecDesc(x.shape[0], x.shape[1], x.shape[2], _cu(cu_seqlens, dev), 0, 0, 0, 0, 0, 0)
    return torch.empty((_linrec_sizes(d, 0)[1], x.shape[2]), dtype=torch.float32, device=dev)


def linrec_fwd(x, g, h0=None, cu_seqlens=None, normalize=False, A_log=None, dt_bias=None,
               output_final_state=True, states=None, y=None, ht=None, workspace=None, stream=None):
    """gdn_linrec_fwd: h_t = exp(g_t) h_{t-1} + u_t over x [B, T, D], u = x or
    (normalize) sqrt(1 - exp(2 g)) x; with A_log and dt_bias [D] g holds raw
    logits.  x and g may each be bfloat16 or float32.  Returns (y, ht): the
    states in x's type, and the final ones [N, D] in float32 (None unless
    output_final_state).  `states`, from linrec_states(), is filled for
    linrec_bwd."""
    lib = _b.load()
    d, act, dev, N = _linrec(x, g, cu_seqlens, normalize, A_log, dt_bias, y)
    D = x.shape[2]
    _f32c(h0, "h0", (N, D), dev)
    _f32c(ht, "ht", (N, D), dev)
    nbytes, rows = _linrec_sizes(d, 0)
    _f32c(states, "states", (rows, D), dev)
    with _on(stream):   # allocated on the kernels' stream (see chunk_fwd)
        if y is None:
            y = torch.empty(x.shape, dtype=x.dtype, device=dev)
        if output_final_state and ht is None:
            ht = torch.empty((N, D), dtype=torch.float32, device=dev)
        workspace, have = _workspace(workspace, nbytes, dev)
    ht = ht if output_final_state else None
    _run(lib.gdn_linrec_fwd, dev, stream, d, act, _p(x), _p(g), _p(h0), _p(cu_seqlens), _p(y), _p(ht),
         _p(states), _p(workspace), have)
    _words(workspace, dev, stream, cu_seqlens is not None, rows > N)
    return y, ht


def _out(out, name, shape, dtype, dev):
    if out.get(name) is None:
        out[name] = torch.empty(shape, dtype=dtype, device=dev)
    else:
        _dense(out[name], name, shape, dev, dtype)


def linrec_bwd(x, g, dy, h0=None, dht=None, cu_seqlens=None, normalize=False, A_log=None, dt_bias=None,
               states=None, want_dh0=True, out=None, workspace=None, stream=None):
    """gdn_linrec_bwd: gradients of <dy, y> + <dht, ht> of linrec_fwd.  Returns
    a dict dx, dg (types of x and g), dh0 (None unless want_dh0) and, with
    A_log, dA_log and ddt_bias [D], float32.  `states` as linrec_fwd filled
    it for the same inputs (None: recomputed); `out` may supply outputs."""
    lib = _b.load()
    d, act, dev, N = _linrec(x, g, cu_seqlens, normalize, A_log, dt_bias, dy)
    D = x.shape[2]
    _f32c(h0, "h0", (N, D), dev)
    _f32c(dht, "dht", (N, D), dev)
    _f32c(states, "states", (_linrec_sizes(d, 0)[1], D), dev)
    nbytes, rows = _linrec_sizes(d, 1)
    out = dict(out or {})
    with _on(stream):   # allocated on the kernels' stream (see chunk_fwd)
        _out(out, "dx", x.shape, x.dtype, dev)
        _out(out, "dg", g.shape, g.dtype, dev)
        if want_dh0:
            _out(out, "dh0", (N, D), torch.float32, dev)
        else:
            out["dh0"] = None
        if act is not None:
            _out(out, "dA_log", (D,), torch.float32, dev)
            _out(out, "ddt_bias", (D,), torch.float32, dev)
        workspace, have = _workspace(workspace, nbytes, dev)
    _run(lib.gdn_linrec_bwd, dev, stream, d, act, _p(x), _p(g), _p(h0), _p(cu_seqlens), _p(dy), _p(dht),
         _p(states), _p(out["dx"]), _p(out["dg"]), _p(out["dh0"]), _p(out.get("dA_log")) if act else None,
         _p(out.get("ddt_bias")) if act else None, _p(workspace), have)
    _words(workspace, dev, stream, cu_seqlens is not None, rows > N)
    return out


def linrec_step(x, g, state, normalize=False, A_log=None, dt_bias=None, y=None, stream=None):
    """gdn_linrec_step: one token of N sequences, x and g [N, D]; state [N, D]
    float32 is updated in place.  Returns y [N, D], the new state in x's type."""
    lib = _b.load()
    d, act, dev, N = _linrec(x, g, None, normalize, A_log, dt_bias, y, lead=1)
    _f32c(state, "state", (N, x.shape[1]), dev)
    if state is None:
        raise ValueError("state is required")
    if y is None:
        with _on(stream):
            y = torch.empty(x.shape, dtype=x.dtype, device=dev)
    _run(lib.gdn_linrec_step, dev, stream, d, act, _p(x), _p(g), _p(state), _p(y))
    return y


# ------------------------------------------------------ q/k norm + rotation
def _heads(t, name):
    """(token stride, head stride) of t [B, T, H, D]; (0, 0) when dense."""
    if t.is_contiguous() or t.numel() == 0:
        return 0, 0
    H, D, s = t.shape[2], t.shape[3], t.stride()
    if D > 1 and s[3] != 1:
        raise ValueError("%s must be dense in its last dimension" % name)
    hs = s[2] if H > 1 else D
    step = _stride(t, name)
    if t.shape[0] * t.shape[1] == 1:
        step = max(step, (H - 1) * hs + D)
    return step, hs


def _qk(q, k, inv_freq, positions, norm, eps, q_weight, k_weight, weight_offset, interleaved):
    dev = _device(q, "q")
    if q.dim() != 4 or k.dim() != 4 or k.shape[:2] != q.shape[:2] or k.shape[3] != q.shape[3]:
        raise ValueError("q [B, T, Hq, D] and k [B, T, Hk, D] do not match: %s, %s" % (tuple(q.shape), tuple(k.shape)))
    if k.dtype != q.dtype or k.device != dev:
        raise ValueError("k must have the type and device of q")
    if norm not in NORMS:
        raise ValueError("norm must be one of %s" % sorted(NORMS))
    B, T, Hq, D = q.shape
    R = 0
    if inv_freq is not None:
        R = 2 * inv_freq.numel()
        _dense(inv_freq, "inv_freq", (R // 2,), dev, torch.float64)
    if positions is not None:
        _dense(positions, "positions", (B, T), dev, torch.int64)
    _f32c(q_weight, "q_weight", (D,), dev)
    _f32c(k_weight, "k_weight", (D,), dev)
    (qs, qh), (ks, kh) = _heads(q, "q"), _heads(k, "k")
    return QkDesc(B, T, Hq, k.shape[2], D, R, qs, ks, qh, kh, _dtype_code(q), NORMS[norm],
                  QK_INTERLEAVED if interleaved else 0, eps, weight_offset), dev


def qk_norm_rope(q, k, inv_freq=None, positions=None, norm="l2", eps=1e-6, q_weight=None, k_weight=None,
                 weight_offset=0.0, interleaved=False, q_out=None, k_out=None, stream=None):
    """gdn_qk_norm_rope: the norm ("none", "l2", "rms") of every head of q
    [B, T, Hq, D] and k [B, T, Hk, D], times weight + weight_offset where a
    weight [D] is given, then the rotation of the first R = 2 len(inv_freq)
    elements (none without inv_freq, a float64 tensor) at `positions` [B, T]
    int64 (None: t).  q and k may be slices of one projection; returns dense
    (q_out, k_out), which chunk_fwd takes as they are."""
    lib = _b.load()
    d, dev = _qk(q, k, inv_freq, positions, norm, eps, q_weight, k_weight, weight_offset, interleaved)
    with _on(stream):   # allocated on the kernel's stream (see chunk_fwd)
        if q_out is None:
            q_out = torch.empty(q.shape, dtype=q.dtype, device=dev)
        else:
            _dense(q_out, "q_out", q.shape, dev, q.dtype)
        if k_out is None:
            k_out = torch.empty(k.shape, dtype=k.dtype, device=dev)
        else:
            _dense(k_out, "k_out", k.shape, dev, k.dtype)
    _run(lib.gdn_qk_norm_rope, dev, stream, d, _p(q), _p(k), _p(q_weight), _p(k_weight), _p(inv_freq),
         _p(positions), _p(q_out), _p(k_out))
    return q_out, k_out


def qk_norm_rope_bwd(q, k, dq_out, dk_out, inv_freq=None, positions=None, norm="l2", eps=1e-6, q_weight=None,
                     k_weight=None, weight_offset=0.0, interleaved=False, out=None, workspace=None,
                     stream=None):
    """gdn_qk_norm_rope_bwd: gradients of <dq_out, q_out> + <dk_out, k_out>.
    Returns a dict dq, dk (dense, q's type) and, for each weight given,
    dq_weight, dk_weight [D] float32.  `out` may supply outputs."""
    lib = _b.load()
    d, dev = _qk(q, k, inv_freq, positions, norm, eps, q_weight, k_weight, weight_offset, interleaved)
    _dense(dq_out, "dq_out", q.shape, dev, q.dtype)
    _dense(dk_out, "dk_out", k.shape, dev, q.dtype)
    n = ctypes.c_size_t()
    _check(lib.gdn_qk_norm_rope_bwd_workspace(d, n))
    out = dict(out or {})
    with _on(stream):   # allocated on the kernels' stream (see chunk_fwd)
        _out(out, "dq", q.shape, q.dtype, dev)
        _out(out, "dk", k.shape, q.dtype, dev)
        for name, w in (("dq_weight", q_weight), ("dk_weight", k_weight)):
            if w is not None:
                _out(out, name, (q.shape[3],), torch.float32, dev)
        need = n.value if q_weight is not None or k_weight is not None else 0
        workspace, have = _workspace(workspace, need, dev)
    _run(lib.gdn_qk_norm_rope_bwd, dev, stream, d, _p(q), _p(k), _p(q_weight), _p(k_weight), _p(inv_freq),
         _p(positions), _p(dq_out), _p(dk_out), _p(out["dq"]), _p(out["dk"]),
         _p(out["dq_weight"]) if q_weight is not None else None,
         _p(out["dk_weight"]) if k_weight is not None else None, _p(workspace), have)
    return out


# -------------------------------------------------------- short convolution
def _conv(x, weight, bias, cu, silu, y=None, lead=2):
    dev = _device(x, "x")
    if x.dim() != lead + 1:
        raise ValueError("x must be %s, got %s" % ("[N, D]" if lead == 1 else "[B, T, D]", tuple(x.shape)))
    D = x.shape[-1]
    if weight.dim() != 2:
        raise ValueError("weight must be [D, W], got %s" % (tuple(weight.shape),))
    _f32c(weight, "weight", (D, weight.shape[1]), dev)
    _f32c(bias, "bias", (D,), dev)
    if y is not None and (y.shape != x.shape or y.dtype != x.dtype or y.device != dev):
        raise ValueError("y / dy must have the shape, type and device of x")
    N = _cu(cu, dev)
    if lead == 1:
        x, y = x.unsqueeze(1), None if y is None else y.unsqueeze(1)
    return ConvDesc(x.shape[0], x.shape[1], D, N, _stride(x, "x"), 0 if y is None else _stride(y, "y / dy"),
                    _dtype_code(x), weight.shape[1], CONV_SILU if silu else 0), dev, N or x.shape[0]


def _conv_bytes(d, backward):
    lib = _b.load()
    n = ctypes.c_size_t()
    _check(lib.gdn_short_conv_workspace(d, backward, n))
    return n.value


def short_conv_fwd(x, weight, bias=None, s0=None, cu_seqlens=None, silu=True, output_final_state=False,
                   y=None, st=None, workspace=None, stream=None):
    """gdn_short_conv_fwd: y_t = silu(bias + sum_j weight[:, j] x_{t-W+1+j})
    over x [B, T, D], weight [D, W] float32, W in 2..4; s0 [N, W - 1, D] (x's
    type) are the inputs before each sequence.  Returns (y, st), st the last
    W - 1 inputs (None unless output_final_state)."""
    lib = _b.load()
    d, dev, N = _conv(x, weight, bias, cu_seqlens, silu, y)
    win = (N, d.width - 1, d.channels)
    for t, name in ((s0, "s0"), (st, "st")):
        if t is not None:
            _dense(t, name, win, dev, x.dtype)
    nbytes = _conv_bytes(d, 0)
    with _on(stream):   # allocated on the kernels' stream (see chunk_fwd)
        if y is None:
            y = torch.empty(x.shape, dtype=x.dtype, device=dev)
        if output_final_state and st is None:
            st = torch.empty(win, dtype=x.dtype, device=dev)
        workspace, have = _workspace(workspace, nbytes, dev)
    st = st if output_final_state else None
    _run(lib.gdn_short_conv_fwd, dev, stream, d, _p(x), _p(weight), _p(bias), _p(s0), _p(cu_seqlens), _p(y),
         _p(st), _p(workspace), have)
    _words(workspace, dev, stream, cu_seqlens is not None)
    return y, st


def short_conv_bwd(x, weight, dy, bias=None, s0=None, dst=None, cu_seqlens=None, silu=True, want_ds0=True,
                   out=None, workspace=None, stream=None):
    """gdn_short_conv_bwd: gradients of <dy, y> + <dst, st> of short_conv_fwd.
    Returns a dict dx, ds0 (x's type; ds0 None unless want_ds0), dweight and,
    with bias, dbias, float32.  `out` may supply outputs."""
    lib = _b.load()
    d, dev, N = _conv(x, weight, bias, cu_seqlens, silu, dy)
    win = (N, d.width - 1, d.channels)
    for t, name in ((s0, "s0"), (dst, "dst")):
        if t is not None:
            _dense(t, name, win, dev, x.dtype)
    nbytes = _conv_bytes(d, 1)
    out = dict(out or {})
    with _on(stream):   # allocated on the kernels' stream (see chunk_fwd)
        _out(out, "dx", x.shape, x.dtype, dev)
        _out(out, "dweight", weight.shape, torch.float32, dev)
        if bias is not None:
            _out(out, "dbias", bias.shape, torch.float32, dev)
        if want_ds0:
            _out(out, "ds0", win, x.dtype, dev)
        else:
            out["ds0"] = None
        workspace, have = _workspace(workspace, nbytes, dev)
    _run(lib.gdn_short_conv_bwd, dev, stream, d, _p(x), _p(weight), _p(bias), _p(s0), _p(cu_seqlens), _p(dy),
         _p(dst), _p(out["dx"]), _p(out["dweight"]), _p(out["dbias"]) if bias is not None else None,
         _p(out["ds0"]), _p(workspace), have)
    _words(workspace, dev, stream, cu_seqlens is not None)
    return out


def short_conv_step(x, weight, state, bias=None, silu=True, y=None, stream=None):
    """gdn_short_conv_step: one token of N sequences, x [N, D]; the window
    state [N, W - 1, D] (x's type) moves on in place.  Returns y [N, D]."""
    lib = _b.load()
    d, dev, N = _conv(x, weight, bias, None, silu, y, lead=1)
    _dense(state, "state", (N, d.width - 1, d.channels), dev, x.dtype)
    if y is None:
        with _on(stream):
            y = torch.empty(x.shape, dtype=x.dtype, device=dev)
    _run(lib.gdn_short_conv_step, dev, stream, d, _p(x), _p(weight), _p(bias), _p(state), _p(y))
    return y
