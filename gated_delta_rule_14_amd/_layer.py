"""ctypes binding of the layer operators of include/gdn.h: the gated linear
recurrence, the q/k norm with rotation and the short convolution.  As in
_binding.py only arguments are marshalled here; every call needs the library.

Activations may be slices of a wider tensor: the last dimension (for q and k
the last one) has to be dense, and consecutive tokens evenly spaced."""
from __future__ import annotations

import ctypes
from functools import lru_cache

import torch

from . import _binding as _b
from ._binding import ACT_GATE, Activation, GdnError, _check, _debug, _on

_i64, _i32, _f32 = ctypes.c_int64, ctypes.c_int32, ctypes.c_float
LINREC_NORMALIZE = 1
NORMS = {"none": 0, "l2": 1, "rms": 2}
QK_INTERLEAVED = 1
CONV_SILU = 1
_CODES = {torch.float32: _b.DTYPE_F32, torch.bfloat16: _b.DTYPE_BF16}
_F32 = torch.float32


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
    P, Z, Zp = ctypes.c_void_p, ctypes.c_size_t, ctypes.POINTER(ctypes.c_size_t)
    L, Q, C, A = (ctypes.POINTER(t) for t in (LinrecDesc, QkDesc, ConvDesc, Activation))
    for name, args in (
            ("gdn_linrec_workspace", [L, _i32, Zp, ctypes.POINTER(_i64)]),
            ("gdn_linrec_fwd", [L, A] + [P] * 8 + [Z, P]),
            ("gdn_linrec_bwd", [L, A] + [P] * 13 + [Z, P]),
            ("gdn_linrec_step", [L, A] + [P] * 5),
            ("gdn_qk_norm_rope", [Q] + [P] * 9),
            ("gdn_qk_norm_rope_bwd_workspace", [Q, Zp]),
            ("gdn_qk_norm_rope_bwd", [Q] + [P] * 13 + [Z, P]),
            ("gdn_short_conv_workspace", [C, _i32, Zp]),
            ("gdn_short_conv_fwd", [C] + [P] * 8 + [Z, P]),
            ("gdn_short_conv_bwd", [C] + [P] * 12 + [Z, P]),
            ("gdn_short_conv_step", [C] + [P] * 6)):
        f = getattr(lib, name)
        f.argtypes, f.restype = args, _i32


# ---------------------------------------------------------------- arguments
# A plan is what a call needs besides its tensors' addresses: the descriptor
# and the workspace sizes of one set of shapes, strides and options.
class _Plan:
    __slots__ = ("desc", "at", "fwd", "bwd", "rows")

    def __init__(self, desc):
        self.desc, self.at = desc, ctypes.byref(desc)
        self.fwd = self.bwd = self.rows = 0


def _p(t):
    return None if t is None else t.data_ptr()


def _code(t, name):
    c = _CODES.get(t.dtype)
    if c is None:
        raise TypeError("%s must be bfloat16 or float32, got %s" % (name, t.dtype))
    return c


def _dense(t, name, shape, dev, dtype=_F32):
    """t is dense, of `shape` (a tuple) and `dtype`, on dev."""
    if t.shape == shape and t.dtype is dtype and t.is_contiguous() and t.device == dev:
        return
    if t.device != dev:
        raise ValueError("%s must be on %s, got %s" % (name, dev, t.device))
    if t.dtype is not dtype:
        raise TypeError("%s must be %s, got %s" % (name, dtype, t.dtype))
    raise ValueError("%s must be contiguous with shape %s, got %s" % (name, tuple(shape), tuple(t.shape)))


# New outputs, on the device of a tensor at hand and without its values: an
# allocation is a large part of a small call's time, and these forms of it take
# 1.1 and 1.6 us where torch.empty with its arguments takes 2.1.
def _like(t):
    return torch.empty_like(t) if t.is_contiguous() else t.new_empty(t.shape)


def _stride(t, name):
    """Elements between the tokens of t [B, T, D] or [N, D] (one token each); 0 for dense rows."""
    if t.is_contiguous() or t.numel() == 0:
        return 0
    s, D = t.stride(), t.shape[-1]
    if D > 1 and s[-1] != 1:
        raise ValueError("%s must be dense in its last dimension" % name)
    return _spacing(t.shape if t.dim() == 3 else (t.shape[0], 1), s, D, name)


def _spacing(shape, s, width, name):
    """The spacing of tokens [B, T] of `width` elements at strides s."""
    B, T = shape[0], shape[1]
    step = s[1] if T > 1 else s[0] if B > 1 else width
    if (B > 1 and T > 1 and s[0] != T * step) or step < width:
        raise ValueError("%s must hold evenly spaced tokens that do not overlap, got strides %s" % (name, tuple(s)))
    return step


def _device(t, name):
    if not t.is_cuda:
        raise ValueError("%s must be a device tensor" % name)
    return t.device


def _run(fn, dev, stream, *args):
    """Call fn(*args, stream) with dev current; `stream` None: dev's current stream."""
    raw = torch._C._cuda_getCurrentRawStream(dev.index) if stream is None else stream.cuda_stream
    if torch._C._cuda_getDevice() == dev.index:
        status = fn(*args, raw)
    else:
        with torch.cuda.device(dev):
            status = fn(*args, raw)
    if status:
        _check(status)


def _workspace(ws, nbytes, dev, like):
    if nbytes == 0:
        return None, 0
    if ws is None:
        return like.new_empty(nbytes, dtype=torch.uint8), nbytes
    if ws.device != dev or not ws.is_contiguous():
        raise ValueError("workspace must be contiguous on %s" % dev)
    return ws, ws.numel() * ws.element_size()


def _words(ws, dev, stream, packed, waits=False):
    """With GDN_DEBUG set: raise on the check of the offsets (packed) and on a wait that gave up."""
    if ws is None or not (packed or waits) or not _debug():
        return
    (stream or torch.cuda.current_stream(dev)).synchronize()
    bad, wait = ws.view(-1).view(torch.uint8)[:8].view(torch.int32).cpu().tolist()
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
@lru_cache(maxsize=1024)
def _linrec_plan(B, T, D, N, xs, gs, ys, xd, gd, flags):
    p = _Plan(LinrecDesc(B, T, D, N, xs, gs, ys, xd, gd, flags))
    lib, n, rows = _b.load(), ctypes.c_size_t(), _i64()
    _check(lib.gdn_linrec_workspace(p.at, 0, n, rows))
    p.fwd, p.rows = n.value, rows.value
    _check(lib.gdn_linrec_workspace(p.at, 1, n, None))
    p.bwd = n.value
    return p


@lru_cache(maxsize=1024)
def _linrec_step_plan(N, D, xs, gs, ys, xd, gd, flags):
    return _Plan(LinrecDesc(N, 1, D, 0, xs, gs, ys, xd, gd, flags))


def _linrec(x, g, normalize, A_log, dt_bias, y, dims):
    """Checks shared by the entry points: the device, x's shape and what identifies a plan."""
    dev, sh = _device(x, "x"), x.shape
    if len(sh) != dims or g.shape != sh:
        raise ValueError("x and g must have one shape %s, got %s and %s"
                         % ("[N, D]" if dims == 2 else "[B, T, D]", tuple(sh), tuple(g.shape)))
    if g.device != dev:
        raise ValueError("g must be on %s" % dev)
    if y is not None and (y.shape != sh or y.dtype != x.dtype or y.device != dev):
        raise ValueError("y / dy must have the shape, type and device of x")
    act = None
    if A_log is not None and dt_bias is not None:
        D = (sh[-1],)
        _dense(A_log, "A_log", D, dev)
        _dense(dt_bias, "dt_bias", D, dev)
        act = ctypes.byref(Activation(ACT_GATE, A_log.data_ptr(), dt_bias.data_ptr()))
    elif A_log is not None or dt_bias is not None:
        raise ValueError("A_log and dt_bias come together")
    key = (_stride(x, "x"), _stride(g, "g"), 0 if y is None else _stride(y, "y / dy"), _code(x, "x"), _code(g, "g"),
           LINREC_NORMALIZE if normalize else 0)
    return dev, sh, act, key


def linrec_states(x, cu_seqlens=None, stream=None):
    """A buffer for linrec_fwd's `states` (of x [B, T, D]), to be kept for
    linrec_bwd; `stream`: the one these calls are given."""
    dev = _device(x, "x")
    B, T, D = x.shape
    p = _linrec_plan(B, T, D, _cu(cu_seqlens, dev), 0, 0, 0, 0, 0, 0)
    with _on(stream):   # allocated on the kernels' stream (see chunk_fwd)
        return x.new_empty((p.rows, D), dtype=_F32)


def linrec_fwd(x, g, h0=None, cu_seqlens=None, normalize=False, A_log=None, dt_bias=None,
               output_final_state=True, states=None, y=None, ht=None, workspace=None, stream=None):
    """gdn_linrec_fwd: h_t = exp(g_t) h_{t-1} + u_t over x [B, T, D], u = x or
    (normalize) sqrt(1 - exp(2 g)) x; with A_log and dt_bias [D] g holds raw
    logits.  x and g may each be bfloat16 or float32.  Returns (y, ht): the
    states in x's type, and the final ones [N, D] in float32 (None unless
    output_final_state).  `states`, from linrec_states(), is filled for
    linrec_bwd."""
    lib = _b.load()
    dev, sh, act, key = _linrec(x, g, normalize, A_log, dt_bias, y, 3)
    packed = _cu(cu_seqlens, dev)
    p = _linrec_plan(*sh, packed, *key)
    ends = (packed or sh[0], sh[2])
    if h0 is not None:
        _dense(h0, "h0", ends, dev)
    if ht is not None:
        _dense(ht, "ht", ends, dev)
    if states is not None:
        _dense(states, "states", (p.rows, sh[2]), dev)
    with _on(stream):   # allocated on the kernels' stream (see chunk_fwd)
        if y is None:
            y = _like(x)
        if not output_final_state:
            ht = None
        elif ht is None:
            ht = x.new_empty(ends, dtype=_F32)
        workspace, have = _workspace(workspace, p.fwd, dev, x)
    _run(lib.gdn_linrec_fwd, dev, stream, p.at, act, x.data_ptr(), g.data_ptr(), _p(h0),
         _p(cu_seqlens), y.data_ptr(), _p(ht), _p(states), _p(workspace), have)
    _words(workspace, dev, stream, packed, p.fwd > 0)   # (a forward workspace: tiles hand on)
    return y, ht


def _out(out, name, shape, dtype, dev, like):
    """The address of output `name`: the one supplied, or a new one."""
    t = out.get(name)
    if t is None:
        same = like.shape == shape and like.dtype is dtype
        out[name] = t = _like(like) if same else like.new_empty(shape, dtype=dtype)
    else:
        _dense(t, name, shape, dev, dtype)
    return t.data_ptr()


def linrec_bwd(x, g, dy, h0=None, dht=None, cu_seqlens=None, normalize=False, A_log=None, dt_bias=None,
               states=None, want_dh0=True, out=None, workspace=None, stream=None):
    """gdn_linrec_bwd: gradients of <dy, y> + <dht, ht> of linrec_fwd.  Returns
    a dict dx, dg (types of x and g), dh0 (None unless want_dh0) and, with
    A_log, dA_log and ddt_bias [D], float32.  `states` as linrec_fwd filled
    it for the same inputs (None: recomputed); `out` may supply outputs."""
    lib = _b.load()
    dev, sh, act, key = _linrec(x, g, normalize, A_log, dt_bias, dy, 3)
    packed = _cu(cu_seqlens, dev)
    p = _linrec_plan(*sh, packed, *key)
    ends, D = (packed or sh[0], sh[2]), (sh[2],)
    if h0 is not None:
        _dense(h0, "h0", ends, dev)
    if dht is not None:
        _dense(dht, "dht", ends, dev)
    if states is not None:
        _dense(states, "states", (p.rows, sh[2]), dev)
    out = dict(out or {})
    with _on(stream):   # allocated on the kernels' stream (see chunk_fwd)
        dx, dg = _out(out, "dx", sh, x.dtype, dev, x), _out(out, "dg", sh, g.dtype, dev, g)
        if not want_dh0:
            out["dh0"] = None
        dh0 = _out(out, "dh0", ends, _F32, dev, x if dht is None else dht) if want_dh0 else None
        dA = _out(out, "dA_log", D, _F32, dev, A_log) if act else None
        db = _out(out, "ddt_bias", D, _F32, dev, dt_bias) if act else None
        workspace, have = _workspace(workspace, p.bwd, dev, x)
    _run(lib.gdn_linrec_bwd, dev, stream, p.at, act, x.data_ptr(), g.data_ptr(), _p(h0),
         _p(cu_seqlens), dy.data_ptr(), _p(dht), _p(states), dx, dg, dh0, dA, db, _p(workspace), have)
    _words(workspace, dev, stream, packed, p.fwd > 0)   # (a forward workspace: tiles hand on)
    return out


def linrec_step(x, g, state, normalize=False, A_log=None, dt_bias=None, y=None, stream=None):
    """gdn_linrec_step: one token of N sequences, x and g [N, D]; state [N, D]
    float32 is updated in place.  Returns y [N, D], the new state in x's type."""
    lib = _b.load()
    dev, sh, act, key = _linrec(x, g, normalize, A_log, dt_bias, y, 2)
    if state is None:
        raise ValueError("state is required")
    _dense(state, "state", sh, dev)
    p = _linrec_step_plan(*sh, *key)
    if y is None:
        with _on(stream):   # allocated on the kernel's stream (see chunk_fwd)
            y = _like(x)
    _run(lib.gdn_linrec_step, dev, stream, p.at, act, x.data_ptr(), g.data_ptr(),
         state.data_ptr(), y.data_ptr())
    return y


# ------------------------------------------------------ q/k norm + rotation
@lru_cache(maxsize=1024)
def _qk_plan(*fields):
    p = _Plan(QkDesc(*fields))
    n = ctypes.c_size_t()
    _check(_b.load().gdn_qk_norm_rope_bwd_workspace(p.at, n))
    p.bwd = n.value
    return p


def _heads(t, name):
    """(token stride, head stride) of t [B, T, H, D]; (0, 0) when dense."""
    if t.is_contiguous() or t.numel() == 0:
        return 0, 0
    sh, s = t.shape, t.stride()
    H, D = sh[2], sh[3]
    if D > 1 and s[3] != 1:
        raise ValueError("%s must be dense in its last dimension" % name)
    hs = s[2] if H > 1 else D
    if hs < D:
        raise ValueError("%s must hold heads that do not overlap, got strides %s" % (name, tuple(s)))
    return _spacing(sh, s, (H - 1) * hs + D, name), hs


def _qk(q, k, inv_freq, positions, norm, eps, q_weight, k_weight, weight_offset, interleaved):
    dev, qs, ks = _device(q, "q"), q.shape, k.shape
    if len(qs) != 4 or len(ks) != 4 or ks[:2] != qs[:2] or ks[3] != qs[3]:
        raise ValueError("q [B, T, Hq, D] and k [B, T, Hk, D] do not match: %s, %s" % (tuple(qs), tuple(ks)))
    if k.dtype != q.dtype or k.device != dev:
        raise ValueError("k must have the type and device of q")
    if norm not in NORMS:
        raise ValueError("norm must be one of %s" % sorted(NORMS))
    B, T, Hq, D = qs
    R = 0
    if inv_freq is not None:
        n = inv_freq.numel()
        _dense(inv_freq, "inv_freq", (n,), dev, torch.float64)
        R = 2 * n
    if positions is not None:
        _dense(positions, "positions", (B, T), dev, torch.int64)
    if q_weight is not None:
        _dense(q_weight, "q_weight", (D,), dev)
    if k_weight is not None:
        _dense(k_weight, "k_weight", (D,), dev)
    (qt, qh), (kt, kh) = _heads(q, "q"), _heads(k, "k")
    return _qk_plan(B, T, Hq, ks[2], D, R, qt, kt, qh, kh, _code(q, "q"), NORMS[norm],
                    QK_INTERLEAVED if interleaved else 0, float(eps), float(weight_offset)), dev, qs, ks


def qk_norm_rope(q, k, inv_freq=None, positions=None, norm="l2", eps=1e-6, q_weight=None, k_weight=None,
                 weight_offset=0.0, interleaved=False, q_out=None, k_out=None, stream=None):
    """gdn_qk_norm_rope: the norm ("none", "l2", "rms") of every head of q
    [B, T, Hq, D] and k [B, T, Hk, D], times weight + weight_offset where a
    weight [D] is given, then the rotation of the first R = 2 len(inv_freq)
    elements (none without inv_freq, a float64 tensor) at `positions` [B, T]
    int64 (None: t).  q and k may be slices of one projection; returns dense
    (q_out, k_out), which chunk_fwd takes as they are."""
    lib = _b.load()
    p, dev, qs, ks = _qk(q, k, inv_freq, positions, norm, eps, q_weight, k_weight, weight_offset, interleaved)
    with _on(stream):   # allocated on the kernel's stream (see chunk_fwd)
        if q_out is None:
            q_out = _like(q)
        else:
            _dense(q_out, "q_out", qs, dev, q.dtype)
        if k_out is None:
            k_out = _like(k)
        else:
            _dense(k_out, "k_out", ks, dev, k.dtype)
    _run(lib.gdn_qk_norm_rope, dev, stream, p.at, q.data_ptr(), k.data_ptr(), _p(q_weight), _p(k_weight),
         _p(inv_freq), _p(positions), q_out.data_ptr(), k_out.data_ptr())
    return q_out, k_out


def qk_norm_rope_bwd(q, k, dq_out, dk_out, inv_freq=None, positions=None, norm="l2", eps=1e-6, q_weight=None,
                     k_weight=None, weight_offset=0.0, interleaved=False, out=None, workspace=None,
                     stream=None):
    """gdn_qk_norm_rope_bwd: gradients of <dq_out, q_out> + <dk_out, k_out>.
    Returns a dict dq, dk (dense, q's type) and, for each weight given,
    dq_weight, dk_weight [D] float32.  `out` may supply outputs."""
    lib = _b.load()
    p, dev, qs, ks = _qk(q, k, inv_freq, positions, norm, eps, q_weight, k_weight, weight_offset, interleaved)
    _dense(dq_out, "dq_out", qs, dev, q.dtype)
    _dense(dk_out, "dk_out", ks, dev, q.dtype)
    out, D = dict(out or {}), (qs[3],)
    with _on(stream):   # allocated on the kernels' stream (see chunk_fwd)
        dq, dk = _out(out, "dq", qs, q.dtype, dev, dq_out), _out(out, "dk", ks, q.dtype, dev, dk_out)
        dqw = _out(out, "dq_weight", D, _F32, dev, q_weight) if q_weight is not None else None
        dkw = _out(out, "dk_weight", D, _F32, dev, k_weight) if k_weight is not None else None
        workspace, have = _workspace(workspace, p.bwd if dqw or dkw else 0, dev, q)
    _run(lib.gdn_qk_norm_rope_bwd, dev, stream, p.at, q.data_ptr(), k.data_ptr(), _p(q_weight), _p(k_weight),
         _p(inv_freq), _p(positions), dq_out.data_ptr(), dk_out.data_ptr(), dq, dk, dqw, dkw, _p(workspace), have)
    return out


# -------------------------------------------------------- short convolution
@lru_cache(maxsize=1024)
def _conv_plan(B, T, D, N, xs, ys, code, W, flags):
    p = _Plan(ConvDesc(B, T, D, N, xs, ys, code, W, flags))
    lib, n = _b.load(), ctypes.c_size_t()
    _check(lib.gdn_short_conv_workspace(p.at, 0, n))
    p.fwd = n.value
    _check(lib.gdn_short_conv_workspace(p.at, 1, n))
    p.bwd = n.value
    return p


@lru_cache(maxsize=1024)
def _conv_step_plan(N, D, xs, ys, code, W, flags):
    return _Plan(ConvDesc(N, 1, D, 0, xs, ys, code, W, flags))


def _conv(x, weight, bias, silu, y, dims):
    """Checks shared by the entry points: the device, x's shape and what identifies a plan."""
    dev, sh, ws = _device(x, "x"), x.shape, weight.shape
    if len(sh) != dims:
        raise ValueError("x must be %s, got %s" % ("[N, D]" if dims == 2 else "[B, T, D]", tuple(sh)))
    if len(ws) != 2:
        raise ValueError("weight must be [D, W], got %s" % (tuple(ws),))
    _dense(weight, "weight", (sh[-1], ws[1]), dev)
    if bias is not None:
        _dense(bias, "bias", (sh[-1],), dev)
    if y is not None and (y.shape != sh or y.dtype != x.dtype or y.device != dev):
        raise ValueError("y / dy must have the shape, type and device of x")
    return dev, sh, (_stride(x, "x"), 0 if y is None else _stride(y, "y / dy"), _code(x, "x"), ws[1],
                     CONV_SILU if silu else 0)


def short_conv_fwd(x, weight, bias=None, s0=None, cu_seqlens=None, silu=True, output_final_state=False,
                   y=None, st=None, workspace=None, stream=None):
    """gdn_short_conv_fwd: y_t = silu(bias + sum_j weight[:, j] x_{t-W+1+j})
    over x [B, T, D], weight [D, W] float32, W in 2..4; s0 [N, W - 1, D] (x's
    type) are the inputs before each sequence.  Returns (y, st), st the last
    W - 1 inputs (None unless output_final_state)."""
    lib = _b.load()
    dev, sh, key = _conv(x, weight, bias, silu, y, 3)
    packed = _cu(cu_seqlens, dev)
    p = _conv_plan(*sh, packed, *key)
    win = (packed or sh[0], key[3] - 1, sh[2])
    if s0 is not None:
        _dense(s0, "s0", win, dev, x.dtype)
    if st is not None:
        _dense(st, "st", win, dev, x.dtype)
    with _on(stream):   # allocated on the kernels' stream (see chunk_fwd)
        if y is None:
            y = _like(x)
        if not output_final_state:
            st = None
        elif st is None:
            st = x.new_empty(win)
        workspace, have = _workspace(workspace, p.fwd, dev, x)
    _run(lib.gdn_short_conv_fwd, dev, stream, p.at, x.data_ptr(), weight.data_ptr(), _p(bias), _p(s0),
         _p(cu_seqlens), y.data_ptr(), _p(st), _p(workspace), have)
    _words(workspace, dev, stream, packed)
    return y, st


def short_conv_bwd(x, weight, dy, bias=None, s0=None, dst=None, cu_seqlens=None, silu=True, want_ds0=True,
                   out=None, workspace=None, stream=None):
    """gdn_short_conv_bwd: gradients of <dy, y> + <dst, st> of short_conv_fwd.
    Returns a dict dx, ds0 (x's type; ds0 None unless want_ds0), dweight and,
    with bias, dbias, float32.  `out` may supply outputs."""
    lib = _b.load()
    dev, sh, key = _conv(x, weight, bias, silu, dy, 3)
    packed = _cu(cu_seqlens, dev)
    p = _conv_plan(*sh, packed, *key)
    win = (packed or sh[0], key[3] - 1, sh[2])
    if s0 is not None:
        _dense(s0, "s0", win, dev, x.dtype)
    if dst is not None:
        _dense(dst, "dst", win, dev, x.dtype)
    out = dict(out or {})
    with _on(stream):   # allocated on the kernels' stream (see chunk_fwd)
        dx = _out(out, "dx", sh, x.dtype, dev, x)
        dw = _out(out, "dweight", weight.shape, _F32, dev, weight)
        db = _out(out, "dbias", bias.shape, _F32, dev, bias) if bias is not None else None
        if not want_ds0:
            out["ds0"] = None
        ds0 = _out(out, "ds0", win, x.dtype, dev, x if dst is None else dst) if want_ds0 else None
        workspace, have = _workspace(workspace, p.bwd, dev, x)
    _run(lib.gdn_short_conv_bwd, dev, stream, p.at, x.data_ptr(), weight.data_ptr(), _p(bias), _p(s0),
         _p(cu_seqlens), dy.data_ptr(), _p(dst), dx, dw, db, ds0, _p(workspace), have)
    _words(workspace, dev, stream, packed)
    return out


def short_conv_step(x, weight, state, bias=None, silu=True, y=None, stream=None):
    """gdn_short_conv_step: one token of N sequences, x [N, D]; the window
    state [N, W - 1, D] (x's type) moves on in place.  Returns y [N, D]."""
    lib = _b.load()
    dev, sh, key = _conv(x, weight, bias, silu, y, 2)
    p = _conv_step_plan(*sh, *key)
    _dense(state, "state", (sh[0], key[3] - 1, sh[1]), dev, x.dtype)
    if y is None:
        with _on(stream):   # allocated on the kernel's stream (see chunk_fwd)
            y = _like(x)
    _run(lib.gdn_short_conv_step, dev, stream, p.at, x.data_ptr(), weight.data_ptr(), _p(bias), state.data_ptr(),
         y.data_ptr())
    return y
