"""ctypes binding of libgdn.so (include/gdn.h): argument marshalling only.

Tensors are PyTorch device tensors (PyTorch provides memory and streams);
every step of the computation runs in the HIP kernels behind the C ABI.
There is no fallback: without the built library every call raises.
"""
from __future__ import annotations

import ctypes
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libgdn.so")
ABI_VERSION = 11

DTYPE_F32, DTYPE_BF16 = 0, 1
GATE_SCALAR, GATE_PER_KEY = 0, 1
STATUS = {0: "GDN_OK", 1: "GDN_ERR_NULL_ARG", 2: "GDN_ERR_BAD_SHAPE", 3: "GDN_ERR_BAD_DTYPE",
          4: "GDN_ERR_UNSUPPORTED", 5: "GDN_ERR_WORKSPACE_TOO_SMALL", 6: "GDN_ERR_MISALIGNED",
          7: "GDN_ERR_HIP", 8: "GDN_ERR_BAD_SEQLENS"}
EXPORTS = sorted(["gdn_abi_version", "gdn_status_str", "gdn_last_error",
                  "gdn_chunk_fwd_workspace", "gdn_chunk_fwd_workspace_act", "gdn_chunk_fwd",
                  "gdn_workspace_layout_of",
                  "gdn_chunk_intra", "gdn_chunk_scan", "gdn_recurrent_step",
                  "gdn_chunk_fwd_act", "gdn_recurrent_step_act",
                  "gdn_chunk_bwd_workspace", "gdn_chunk_bwd", "gdn_chunk_bwd_act",
                  "gdn_seqlens_status_offset", "gdn_sync_status_offset",
                  "gdn_chunk_fwd_noalloc",
                  "gdn_linrec_workspace", "gdn_linrec_fwd", "gdn_linrec_bwd", "gdn_linrec_step",
                  "gdn_qk_norm_rope", "gdn_qk_norm_rope_bwd_workspace", "gdn_qk_norm_rope_bwd",
                  "gdn_short_conv_workspace", "gdn_short_conv_fwd", "gdn_short_conv_bwd",
                  "gdn_short_conv_step",
                  "gdn_decay_attn_workspace", "gdn_decay_attn_fwd", "gdn_decay_attn_bwd",
                  "gdn_decay_attn_step",
                  "gdn_paged_append", "gdn_paged_attn_workspace", "gdn_paged_attn"])
INTRA_STORE_AINV = 1
ACT_GATE, ACT_BETA_SIGMOID, ACT_BETA_NEG_EIG, ACT_QK_L2NORM = 1, 2, 4, 8


class FwdDesc(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int64), ("seq_len", ctypes.c_int64),
                ("num_heads", ctypes.c_int64), ("key_dim", ctypes.c_int64),
                ("value_dim", ctypes.c_int64), ("num_seqs", ctypes.c_int64),
                ("chunk", ctypes.c_int32), ("qkv_dtype", ctypes.c_int32),
                ("gate", ctypes.c_int32), ("scale", ctypes.c_float),
                ("num_v_heads", ctypes.c_int64)]


class StepDesc(ctypes.Structure):
    _fields_ = [("num_seqs", ctypes.c_int64), ("num_heads", ctypes.c_int64),
                ("key_dim", ctypes.c_int64), ("value_dim", ctypes.c_int64),
                ("qkv_dtype", ctypes.c_int32), ("gate", ctypes.c_int32),
                ("scale", ctypes.c_float), ("num_v_heads", ctypes.c_int64)]


class Activation(ctypes.Structure):
    _fields_ = [("flags", ctypes.c_int32), ("A_log", ctypes.c_void_p), ("dt_bias", ctypes.c_void_p)]


class WorkspaceLayout(ctypes.Structure):
    _fields_ = [(n, ctypes.c_size_t) for n in
                ("gcum", "w", "u", "qs", "ks", "aqk", "ainv", "chunks", "seqs", "total")] + \
               [("max_chunks", ctypes.c_int64)]


class GdnError(RuntimeError):
    def __init__(self, status: int, detail: str):
        super().__init__("%s: %s" % (STATUS.get(status, str(status)), detail))
        self.status = status


_lib = None


def load(path: str = LIB_PATH):
    """Load libgdn.so once; raise if it is missing or of another ABI."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise RuntimeError("libgdn.so not built (%s): run `python -m gated_delta_rule_14_amd.build`"
                           % path)
    lib = ctypes.CDLL(path)
    P, S = ctypes.c_void_p, ctypes.c_int32
    lib.gdn_abi_version.restype = ctypes.c_int
    lib.gdn_status_str.restype = ctypes.c_char_p
    lib.gdn_status_str.argtypes = [S]
    lib.gdn_last_error.restype = ctypes.c_char_p
    lib.gdn_chunk_fwd_workspace.argtypes = [ctypes.POINTER(FwdDesc), ctypes.POINTER(ctypes.c_size_t)]
    lib.gdn_chunk_fwd_workspace.restype = S
    lib.gdn_chunk_fwd_workspace_act.argtypes = [ctypes.POINTER(FwdDesc), ctypes.POINTER(Activation),
                                                ctypes.POINTER(ctypes.c_size_t)]
    lib.gdn_chunk_fwd_workspace_act.restype = S
    lib.gdn_workspace_layout_of.argtypes = [ctypes.POINTER(FwdDesc), ctypes.POINTER(WorkspaceLayout)]
    lib.gdn_workspace_layout_of.restype = S
    lib.gdn_chunk_fwd.argtypes = [ctypes.POINTER(FwdDesc), P, P, P, P, P, P, P, P, P, P,
                                  ctypes.c_size_t, P]
    lib.gdn_chunk_fwd.restype = S
    lib.gdn_chunk_intra.argtypes = [ctypes.POINTER(FwdDesc), P, P, P, P, P, P, P,
                                    ctypes.c_size_t, ctypes.c_int32, P]
    lib.gdn_chunk_intra.restype = S
    lib.gdn_chunk_scan.argtypes = [ctypes.POINTER(FwdDesc), P, P, P, P, P, ctypes.c_size_t, P]
    lib.gdn_chunk_scan.restype = S
    lib.gdn_recurrent_step.argtypes = [ctypes.POINTER(StepDesc), P, P, P, P, P, P, P, P]
    lib.gdn_recurrent_step.restype = S
    lib.gdn_chunk_fwd_act.argtypes = [ctypes.POINTER(FwdDesc), ctypes.POINTER(Activation), P, P, P,
                                      P, P, P, P, P, P, P, ctypes.c_size_t, P]
    lib.gdn_chunk_fwd_act.restype = S
    lib.gdn_recurrent_step_act.argtypes = [ctypes.POINTER(StepDesc), ctypes.POINTER(Activation),
                                           P, P, P, P, P, P, P, P]
    lib.gdn_recurrent_step_act.restype = S
    lib.gdn_chunk_bwd_workspace.argtypes = [ctypes.POINTER(FwdDesc), ctypes.POINTER(ctypes.c_size_t)]
    lib.gdn_chunk_bwd_workspace.restype = S
    lib.gdn_chunk_bwd.argtypes = [ctypes.POINTER(FwdDesc)] + [P] * 16 + [ctypes.c_size_t, P]
    lib.gdn_chunk_bwd.restype = S
    lib.gdn_chunk_bwd_act.argtypes = [ctypes.POINTER(FwdDesc), ctypes.POINTER(Activation)] + \
        [P] * 18 + [ctypes.c_size_t, P]
    lib.gdn_chunk_bwd_act.restype = S
    lib.gdn_seqlens_status_offset.argtypes = [ctypes.POINTER(FwdDesc), ctypes.POINTER(Activation),
                                              ctypes.c_int32, ctypes.POINTER(ctypes.c_size_t)]
    lib.gdn_seqlens_status_offset.restype = S
    lib.gdn_sync_status_offset.argtypes = [ctypes.POINTER(FwdDesc), ctypes.POINTER(Activation),
                                           ctypes.POINTER(ctypes.c_size_t)]
    lib.gdn_sync_status_offset.restype = S
    lib.gdn_chunk_fwd_noalloc.argtypes = [ctypes.POINTER(FwdDesc), ctypes.POINTER(Activation),
                                          P, P, P, P, P, P, P, P, P, P]
    lib.gdn_chunk_fwd_noalloc.restype = S
    v = lib.gdn_abi_version()
    if v != ABI_VERSION:
        raise RuntimeError("libgdn.so ABI %d, binding expects %d" % (v, ABI_VERSION))
    from . import _layer, _mixer
    _layer.declare(lib)
    _mixer.declare(lib)
    _lib = lib
    return lib


def _check(status: int):
    if status != 0:
        raise GdnError(status, _lib.gdn_last_error().decode())


def _debug():
    return os.environ.get("GDN_DEBUG", "") not in ("", "0")


def _word(workspace, off, stream):
    """The int32 at byte offset `off` of the workspace, once `stream` (None:
    the current stream) has reached everything enqueued so far."""
    (stream or torch.cuda.current_stream()).synchronize()
    return int(workspace[off:off + 4].view(torch.int32).cpu().item())


def seqlens_status(desc, workspace, act=None, backward=False, stream=None):
    """The check of cu_seqlens that a packed call left in its workspace
    (gdn_seqlens_status_offset): raises GdnError(GDN_ERR_BAD_SEQLENS) if the
    offsets did not start at 0, decreased or did not end at T.  Waits for
    `stream` (None: the current stream).  chunk_fwd and chunk_bwd call it
    when GDN_DEBUG is set."""
    lib = load()
    off = ctypes.c_size_t()
    _check(lib.gdn_seqlens_status_offset(ctypes.byref(desc),
                                         ctypes.byref(act) if act is not None else None,
                                         1 if backward else 0, ctypes.byref(off)))
    if _word(workspace, off.value, stream) != 0:
        raise GdnError(8, "cu_seqlens must start at 0, never decrease and end at T")


def sync_status_offset(desc, act=None):
    """gdn_sync_status_offset: byte offset of the single-pass kernel's
    synchronisation status word in the workspace, or None for shapes that run
    the two-stage route (which has no waits between waves)."""
    lib = load()
    off = ctypes.c_size_t()
    st = lib.gdn_sync_status_offset(ctypes.byref(desc), ctypes.byref(act) if act is not None else None,
                                    ctypes.byref(off))
    if st == 4:
        return None
    _check(st)
    return off.value


def sync_status(desc, workspace, act=None, stream=None):
    """The single-pass kernel's synchronisation status word (0: every wait
    between its waves was met; 1: a wait gave up and the results are wrong).
    The library never clears the word: the binding allocates its workspaces
    zeroed.  Waits for `stream`.  0 for shapes without the single-pass
    kernel.  chunk_fwd raises on a nonzero word when GDN_DEBUG is set."""
    off = sync_status_offset(desc, act)
    return 0 if off is None else _word(workspace, off, stream)


class _on:
    """Context: allocations go to `stream` (None: the current stream)."""

    def __init__(self, stream):
        self.ctx = torch.cuda.stream(stream) if stream is not None else None

    def __enter__(self):
        if self.ctx is not None:
            self.ctx.__enter__()

    def __exit__(self, *exc):
        if self.ctx is not None:
            return self.ctx.__exit__(*exc)
        return False


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _dtype_code(t):
    if t.dtype == torch.bfloat16:
        return DTYPE_BF16
    if t.dtype == torch.float32:
        return DTYPE_F32
    raise TypeError("q/k/v must be bfloat16 or float32, got %s" % t.dtype)


def _need(t, name, dtype=None):
    if not t.is_cuda:
        raise ValueError("%s must be a device tensor" % name)
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)
    if dtype is not None and t.dtype != dtype:
        raise TypeError("%s must be %s, got %s" % (name, dtype, t.dtype))


def fwd_desc(q, v, gate="scalar", chunk=64, scale=None, num_seqs=0):
    """Descriptor of q [B, T, H, K] and v [B, T, H_V, V] (H_V a multiple of H:
    grouped value heads when H_V > H)."""
    B, T, H, K = q.shape
    HV = v.shape[2]
    return FwdDesc(B, T, H, K, v.shape[-1], num_seqs, chunk, _dtype_code(q),
                   GATE_PER_KEY if gate == "per_key" else GATE_SCALAR,
                   float(K ** -0.5 if scale is None else scale), HV if HV != H else 0)


def workspace_layout(desc: FwdDesc) -> WorkspaceLayout:
    lib = load()
    out = WorkspaceLayout()
    _check(lib.gdn_workspace_layout_of(ctypes.byref(desc), ctypes.byref(out)))
    return out


def workspace_bytes(desc: FwdDesc, act=None) -> int:
    lib = load()
    n = ctypes.c_size_t()
    if act is None:
        _check(lib.gdn_chunk_fwd_workspace(ctypes.byref(desc), ctypes.byref(n)))
    else:
        _check(lib.gdn_chunk_fwd_workspace_act(ctypes.byref(desc), ctypes.byref(act), ctypes.byref(n)))
    return n.value


def activation(gate_logits=False, beta_sigmoid=False, neg_eig=False, A_log=None, dt_bias=None,
               qk_l2norm=False):
    """The optional in-kernel input activation (gdn_activation): with
    gate_logits, g holds raw logits a and log alpha = -exp(A_log) softplus(a +
    dt_bias) (A_log [H], dt_bias [H] or [H, K] float32 device tensors); with
    beta_sigmoid, beta holds raw logits b and beta = sigmoid(b), times 2 with
    neg_eig (beta in (0, 2)); with qk_l2norm, q and k are L2-normalised per
    token and head inside the kernels."""
    flags = (ACT_GATE if gate_logits else 0) | (ACT_BETA_SIGMOID if beta_sigmoid else 0) | \
        (ACT_BETA_NEG_EIG if neg_eig else 0) | (ACT_QK_L2NORM if qk_l2norm else 0)
    if gate_logits:
        _need(A_log, "A_log", torch.float32)
        _need(dt_bias, "dt_bias", torch.float32)
    act = Activation(flags, _ptr(A_log) if gate_logits else None,
                     _ptr(dt_bias) if gate_logits else None)
    act._keep = (A_log, dt_bias)   # the tensors outlive the struct's use
    return act


def _act_shapes(act, H, K, gate):
    if act is None or not (act.flags & ACT_GATE):
        return
    A_log, dt_bias = act._keep
    want_dt = (H, K) if gate == "per_key" else (H,)
    if tuple(A_log.shape) != (H,) or tuple(dt_bias.shape) != want_dt:
        raise ValueError("A_log must have shape %s and dt_bias %s" % ((H,), want_dt))


def _inputs(q, k, v, beta, g, cu_seqlens, gate):
    for t, name in ((q, "q"), (k, "k"), (v, "v")):
        _need(t, name, q.dtype)
    _need(beta, "beta", torch.float32)
    _need(g, "g", torch.float32)
    if cu_seqlens is not None:
        _need(cu_seqlens, "cu_seqlens", torch.int64)
    HV = v.shape[2]
    if k.shape != q.shape or v.shape[:2] != q.shape[:2] or HV % q.shape[2] != 0 or \
            tuple(beta.shape) != tuple(v.shape[:3]):
        raise ValueError("shape mismatch among q, k, v, beta (v may have a multiple of q's heads)")
    want_g = tuple(v.shape[:3]) + ((q.shape[3],) if gate == "per_key" else ())
    if tuple(g.shape) != tuple(want_g):
        raise ValueError("g must have shape %s for gate=%s" % (tuple(want_g), gate))


def chunk_fwd(q, k, v, beta, g, scale=None, h0=None, cu_seqlens=None, chunk=64,
              gate="scalar", output_final_state=True, workspace=None, o=None, ht=None,
              stream=None, act=None):
    """gdn_chunk_fwd (gdn_chunk_fwd_act when act, from activation(), is given):
    returns (o, ht) (ht is None unless output_final_state)."""
    lib = load()
    _inputs(q, k, v, beta, g, cu_seqlens, gate)
    N = q.shape[0] if cu_seqlens is None else cu_seqlens.numel() - 1
    desc = fwd_desc(q, v, gate, chunk, scale, 0 if cu_seqlens is None else N)
    H, K, V = v.shape[2], q.shape[3], v.shape[3]   # state heads: the value heads
    if h0 is not None:
        _need(h0, "h0", torch.float32)
        if tuple(h0.shape) != (N, H, K, V):
            raise ValueError("h0 must have shape %s" % ((N, H, K, V),))
    nbytes = workspace_bytes(desc, act)
    # what is allocated here is allocated on the stream the kernels run on,
    # so the caching allocator never hands it out while they still use it
    with _on(stream):
        if o is None:
            o = torch.empty(v.shape, dtype=q.dtype, device=q.device)
        if output_final_state and ht is None:
            ht = torch.empty((N, H, K, V), dtype=torch.float32, device=q.device)
        if workspace is None or workspace.numel() * workspace.element_size() < nbytes:
            # zeroed: the single-pass kernel's synchronisation word starts clear
            workspace = torch.zeros(nbytes, dtype=torch.uint8, device=q.device)
    args = (_ptr(q), _ptr(k), _ptr(v), _ptr(beta), _ptr(g), _ptr(h0), _ptr(cu_seqlens), _ptr(o),
            _ptr(ht) if output_final_state else None, _ptr(workspace),
            workspace.numel() * workspace.element_size(), _stream(stream))
    if act is None:
        _check(lib.gdn_chunk_fwd(ctypes.byref(desc), *args))
    else:
        _act_shapes(act, H, K, gate)
        _check(lib.gdn_chunk_fwd_act(ctypes.byref(desc), ctypes.byref(act), *args))
    if _debug():
        if cu_seqlens is not None:
            seqlens_status(desc, workspace, act, stream=stream)
        if sync_status(desc, workspace, act, stream=stream) != 0:
            raise GdnError(7, "a wait between the single-pass kernel's waves gave up: wrong results")
    return o, (ht if output_final_state else None)


def bwd_workspace_bytes(desc: FwdDesc) -> int:
    lib = load()
    n = ctypes.c_size_t()
    _check(lib.gdn_chunk_bwd_workspace(ctypes.byref(desc), ctypes.byref(n)))
    return n.value


def chunk_bwd(q, k, v, beta, g, do, scale=None, h0=None, dht=None, cu_seqlens=None, chunk=64,
              want_dh0=True, workspace=None, out=None, stream=None, act=None, gate="scalar"):
    """gdn_chunk_bwd (gdn_chunk_bwd_act when act, from activation(), is
    given): gradients of <do, o> + <dht, ht> of the chunked forward with
    respect to q, k, v, beta, g (scalar or, bf16 only, per-key gate) and h0.
    Returns a dict dq, dk, dv (dtype of q), dbeta, dg (the shape of g), dh0
    (float32; dh0 None unless want_dh0).  With act, beta and g are the raw
    logits, dbeta and dg their gradients, and with the gate activation the
    dict also holds dA_log ([H]) and ddt_bias (the shape of dt_bias), float32.
    `out` may supply any of these tensors."""
    lib = load()
    _inputs(q, k, v, beta, g, cu_seqlens, gate)
    _need(do, "do", q.dtype)
    if do.shape != v.shape:
        raise ValueError("do must have the shape of v")
    N = q.shape[0] if cu_seqlens is None else cu_seqlens.numel() - 1
    desc = fwd_desc(q, v, gate, chunk, scale, 0 if cu_seqlens is None else N)
    H, K, V = v.shape[2], q.shape[3], v.shape[3]
    for t, name in ((h0, "h0"), (dht, "dht")):
        if t is not None:
            _need(t, name, torch.float32)
            if tuple(t.shape) != (N, H, K, V):
                raise ValueError("%s must have shape %s" % (name, (N, H, K, V)))
    out = dict(out or {})
    dev = q.device
    act_gate = act is not None and bool(act.flags & ACT_GATE)
    nbytes = bwd_workspace_bytes(desc)
    with _on(stream):   # allocated on the kernels' stream (see chunk_fwd)
        for name, shape, dt in (("dq", q.shape, q.dtype), ("dk", k.shape, q.dtype),
                                ("dv", v.shape, q.dtype), ("dbeta", beta.shape, torch.float32),
                                ("dg", g.shape, torch.float32)):
            if out.get(name) is None:
                out[name] = torch.empty(shape, dtype=dt, device=dev)
            _need(out[name], name, dt)
        if want_dh0 and out.get("dh0") is None:
            out["dh0"] = torch.empty((N, H, K, V), dtype=torch.float32, device=dev)
        if not want_dh0:
            out["dh0"] = None
        if act_gate:
            _act_shapes(act, H, K, gate)
            for name, shape in (("dA_log", (H,)), ("ddt_bias", (H, K) if gate == "per_key" else (H,))):
                if out.get(name) is None:
                    out[name] = torch.empty(shape, dtype=torch.float32, device=dev)
                _need(out[name], name, torch.float32)
        if workspace is None or workspace.numel() * workspace.element_size() < nbytes:
            workspace = torch.empty(nbytes, dtype=torch.uint8, device=dev)
    args = [_ptr(q), _ptr(k), _ptr(v), _ptr(beta), _ptr(g), _ptr(h0), _ptr(cu_seqlens), _ptr(do),
            _ptr(dht), _ptr(out["dq"]), _ptr(out["dk"]), _ptr(out["dv"]), _ptr(out["dbeta"]),
            _ptr(out["dg"]), _ptr(out["dh0"])]
    tail = [_ptr(workspace), workspace.numel() * workspace.element_size(), _stream(stream)]
    if act is None:
        _check(lib.gdn_chunk_bwd(ctypes.byref(desc), *args, *tail))
    else:
        _check(lib.gdn_chunk_bwd_act(ctypes.byref(desc), ctypes.byref(act), *args,
                                     _ptr(out.get("dA_log")) if act_gate else None,
                                     _ptr(out.get("ddt_bias")) if act_gate else None, *tail))
    if cu_seqlens is not None and _debug():
        seqlens_status(desc, workspace, act, backward=True, stream=stream)
    return out


def chunk_intra(q, k, v, beta, g, scale=None, cu_seqlens=None, chunk=64, gate="scalar",
                store_ainv=True, workspace=None, stream=None, views=True):
    """gdn_chunk_intra: the intra-chunk stage alone.  Returns a dict: gcum and
    ainv (views into the workspace), w, u, qs, ks, aqk (row-major copies of
    the workspace arrays, which the library keeps in MFMA fragment /
    accumulator order), max_chunks, workspace and desc.  With the per-key
    gate only gcum[:, :, C - 1] is written.  views=False skips the arrays
    (no work beyond the library call)."""
    lib = load()
    _inputs(q, k, v, beta, g, cu_seqlens, gate)
    N = q.shape[0] if cu_seqlens is None else cu_seqlens.numel() - 1
    desc = fwd_desc(q, v, gate, chunk, scale, 0 if cu_seqlens is None else N)
    L = workspace_layout(desc)
    if workspace is None or workspace.numel() * workspace.element_size() < L.total:
        with _on(stream):   # allocated on the kernels' stream (see chunk_fwd)
            workspace = torch.zeros(L.total, dtype=torch.uint8, device=q.device)
    ws = workspace
    _check(lib.gdn_chunk_intra(ctypes.byref(desc), _ptr(q), _ptr(k), _ptr(v), _ptr(beta),
                               _ptr(g), _ptr(cu_seqlens), _ptr(ws),
                               ws.numel() * ws.element_size(),
                               INTRA_STORE_AINV if store_ainv else 0, _stream(stream)))
    H, K, V, C, mc = v.shape[2], q.shape[3], v.shape[3], chunk, L.max_chunks
    if not views:
        return dict(max_chunks=mc, workspace=ws, desc=desc)

    def view(off, dtype, shape):
        n = 1
        for s_ in shape:
            n *= s_
        es = torch.empty(0, dtype=dtype).element_size()
        return ws[off:off + n * es].view(dtype).view(*shape)
    gshape = (H, mc, C, K) if gate == "per_key" else (H, mc, C)
    lead = (H, mc)
    return dict(gcum=view(L.gcum, torch.float32, gshape),
                w=from_frag_order(view(L.w, q.dtype, lead + (C * K,)), C, K),
                u=from_acc_order(view(L.u, q.dtype, lead + (C * V,)), C, V),
                qs=from_frag_order(view(L.qs, q.dtype, lead + (C * K,)), C, K),
                ks=from_frag_order(view(L.ks, q.dtype, lead + (K * C,)), K, C).transpose(-1, -2),
                aqk=from_frag_order(view(L.aqk, q.dtype, lead + (C * C,)), C, C),
                ainv=view(L.ainv, torch.float32, (H, mc, C, C)), max_chunks=mc,
                workspace=ws, desc=desc)


def from_frag_order(x, R, D):
    """An R x D matrix stored in MFMA fragment order (last dim of x, R*D
    elements) as an [..., R, D] tensor (a reordered copy).  Group (rt, sg),
    lane l = 16 g + r, element e holds X[16 rt + r][KG sg + col], col = 8 g + e
    for bf16 (KG 32) and 4 e + g for fp32 (KG 16)."""
    lead = tuple(x.shape[:-1])
    n = len(lead)
    if x.dtype == torch.bfloat16:
        y = x.reshape(*lead, R // 16, D // 32, 4, 16, 8)           # rt sg g r e
        order = (0, 3, 1, 2, 4)                                      # rt r sg g e
    else:
        y = x.reshape(*lead, R // 16, D // 16, 4, 16, 4)           # rt sg g r e
        order = (0, 3, 1, 4, 2)                                      # rt r sg e g
    y = y.permute(*range(n), *(n + o for o in order))
    return y.reshape(*lead, R, D)


def from_acc_order(x, R, D):
    """An R x D matrix stored in accumulator order (tile (rt, ct), lane
    l = 16 g + c, element e holds X[16 rt + 4 g + e][16 ct + c]) as [..., R, D]."""
    lead = tuple(x.shape[:-1])
    n = len(lead)
    y = x.reshape(*lead, R // 16, D // 16, 4, 16, 4)                # rt ct g c e
    y = y.permute(*range(n), *(n + o for o in (0, 2, 4, 1, 3)))     # rt g e ct c
    return y.reshape(*lead, R, D)


def chunk_scan(desc, workspace, o, h0=None, ht=None, cu_seqlens=None, stream=None):
    """gdn_chunk_scan: the state pass on a workspace prepared by chunk_intra
    for the same descriptor and inputs.  Writes o (and ht if given)."""
    lib = load()
    _need(o, "o")
    _check(lib.gdn_chunk_scan(ctypes.byref(desc), _ptr(h0), _ptr(cu_seqlens), _ptr(o), _ptr(ht),
                              _ptr(workspace), workspace.numel() * workspace.element_size(),
                              _stream(stream)))
    return o, ht


def recurrent_step(q, k, v, beta, g, state, scale=None, gate="scalar", o=None, stream=None,
                   act=None):
    """gdn_recurrent_step (gdn_recurrent_step_act with act): one token for N
    sequences; state updated in place.  q, k [N, H, K]; v [N, H, V];
    beta [N, H]; g [N, H] or [N, H, K]."""
    lib = load()
    for t, name in ((q, "q"), (k, "k"), (v, "v")):
        _need(t, name, q.dtype)
    _need(beta, "beta", torch.float32)
    _need(g, "g", torch.float32)
    _need(state, "state", torch.float32)
    N, Hq, K = q.shape
    H, V = v.shape[1], v.shape[-1]    # value heads (a multiple of q's: grouped value heads)
    if tuple(state.shape) != (N, H, K, V):
        raise ValueError("state must have shape %s" % ((N, H, K, V),))
    want_g = (N, H, K) if gate == "per_key" else (N, H)
    if tuple(g.shape) != want_g or tuple(beta.shape) != (N, H) or H % Hq != 0:
        raise ValueError("beta/g shape mismatch")
    if o is None:
        with _on(stream):   # allocated on the kernel's stream (see chunk_fwd)
            o = torch.empty((N, H, V), dtype=q.dtype, device=q.device)
    desc = StepDesc(N, Hq, K, V, _dtype_code(q),
                    GATE_PER_KEY if gate == "per_key" else GATE_SCALAR,
                    float(K ** -0.5 if scale is None else scale), H if H != Hq else 0)
    args = (_ptr(q), _ptr(k), _ptr(v), _ptr(beta), _ptr(g), _ptr(state), _ptr(o), _stream(stream))
    if act is None:
        _check(lib.gdn_recurrent_step(ctypes.byref(desc), *args))
    else:
        _act_shapes(act, H, K, gate)
        _check(lib.gdn_recurrent_step_act(ctypes.byref(desc), ctypes.byref(act), *args))
    return o
