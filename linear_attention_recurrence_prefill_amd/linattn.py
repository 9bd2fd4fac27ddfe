"""Linear attention with a decay for each head (``include/gdn_linattn.h``): the chunked forward and
backward over packed sequences and the step of one token,

    S_t = exp(g_t) S_{t-1} + k_t v_t^T,    o_t = scale * S_t^T q_t

per head.  Argument checks and marshalling only, as in :mod:`.gdn`: the computation runs in the HIP
library on torch's current stream of the tensors' device.
"""
from __future__ import annotations

import ctypes

import torch

from .gdn import (GDN_DTYPE_BF16, GDN_DTYPE_F32, _check, _check_out, _nbytes, _workspace,
                  load_library)


class LinattnProblem(ctypes.Structure):
    _fields_ = [("total_tokens", ctypes.c_int64), ("num_seqs", ctypes.c_int32),
                ("num_heads", ctypes.c_int32), ("num_k_heads", ctypes.c_int32),
                ("head_dim", ctypes.c_int32), ("dtype", ctypes.c_int32),
                ("head_decay", ctypes.c_int32), ("seg_chunks", ctypes.c_int32),
                ("num_slots", ctypes.c_int32), ("scale", ctypes.c_float),
                ("reserved", ctypes.c_int32), ("h0_seq_stride", ctypes.c_int64)]


class _Here:
    """The context of a call whose tensors are on the current device."""

    def __enter__(self):
        return self

    def __exit__(self, *exc):
        return False


_HERE = _Here()


def _on(device):
    """A context in which ``device`` is the current device (the library launches there)."""
    return _HERE if torch.cuda.current_device() == device.index else torch.cuda.device(device)


_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream_of(device):
    if _raw_stream is not None:  # the same handle without a stream object
        return _raw_stream(device.index)
    return torch.cuda.current_stream(device).cuda_stream


def _at(t):
    """A tensor's address as the C calls take it (None: NULL)."""
    return None if t is None else t.data_ptr()


def _same_device(device, **tensors):
    index = device.index
    for name, t in tensors.items():
        if t is not None and (t.get_device() != index or not t.is_contiguous()):
            raise ValueError(f"{name} must be a contiguous device tensor on {device}")


def _device_of(t):
    if not t.is_cuda:
        raise ValueError("inputs must be contiguous device tensors")
    return t.device


def _no_overlap(name, out, *inputs):
    lo, hi = out.data_ptr(), out.data_ptr() + _nbytes(out)
    for t in inputs:
        if t is not None and t.data_ptr() < hi and lo < t.data_ptr() + _nbytes(t):
            raise ValueError(f"{name} must not overlap an input")


def _dtype_of(q):
    if q.dtype == torch.bfloat16:
        return GDN_DTYPE_BF16
    if q.dtype == torch.float32:
        return GDN_DTYPE_F32
    raise ValueError("q must be bfloat16 or float32")


def _heads(q, k, v, g, rows):
    """Sizes of q, k [n, Hk, D], v [n, H, D], g [n, H] or [H]: (n, H, Hk, D, head_decay)."""
    if q.dim() != 3 or v.dim() != 3:
        raise ValueError(f"q, k and v must be [{rows}, heads, D]")
    n, Hk, D = q.shape
    H = v.shape[1]
    if k.shape != (n, Hk, D) or v.shape != (n, H, D) or Hk < 1 or H % Hk != 0:
        raise ValueError(f"q and k must be [{rows}, Hk, D] and v [{rows}, H, D] with Hk dividing H")
    if g.shape != (n, H) and g.shape != (H,):
        raise ValueError(f"g must be [{rows}, H], or [H] for a constant decay per head")
    if k.dtype != q.dtype or v.dtype != q.dtype:
        raise ValueError("k and v must have q's dtype")
    if g.dtype != torch.float32:
        raise ValueError("g must be float32")
    return n, H, Hk, D, 1 if g.dim() == 1 else 0


def _problem(q, k, v, g, cu_seqlens, h0, scale, seg_chunks, num_slots):
    T, H, Hk, D, head = _heads(q, k, v, g, "T")
    if cu_seqlens.dtype != torch.int32 or cu_seqlens.dim() != 1 or cu_seqlens.numel() < 2:
        raise ValueError("cu_seqlens must be a 1-D int32 tensor of at least two offsets")
    dtype, device = _dtype_of(q), _device_of(q)
    _same_device(device, q=q, k=k, v=v, g=g, cu_seqlens=cu_seqlens, h0=h0)
    N = cu_seqlens.numel() - 1
    stride = H * D * D
    if h0 is not None:
        if h0.dtype != torch.float32:
            raise ValueError("h0 must be float32")
        if tuple(h0.shape) == (H, D, D):
            stride = 0
        elif tuple(h0.shape) != (N, H, D, D):
            raise ValueError("h0 must be [N, H, D, D] or [H, D, D] (shared by all sequences)")
    p = LinattnProblem(T, N, H, Hk, D, dtype, head, int(seg_chunks), int(num_slots), float(scale), 0,
                       stride)
    return p, device, N, H, D


def _workspace_bytes(fn, p):
    n = ctypes.c_size_t(0)
    _check(fn(ctypes.byref(p), ctypes.byref(n)))
    return n.value


def linattn_fwd(q, k, v, g, cu_seqlens, h0=None, *, scale=1.0, seg_chunks=0, num_slots=0,
                output_final_state=True, out=None, final_state=None, workspace=None):
    """Forward: q, k [T, Hk, D], v [T, H, D] (bf16 or fp32; value head h reads key head
    h // (H // Hk)), g fp32 log decays [T, H] or [H], cu_seqlens int32 [N + 1], h0 fp32
    [N, H, D, D] or [H, D, D] (shared by all sequences).  Returns (o, final states or None).
    seg_chunks: 64-token chunks per unit that sequences are split into (0: from the mean length; set
    it, to 8 or so, for one long sequence among many short ones)."""
    p, device, N, H, D = _problem(q, k, v, g, cu_seqlens, h0, scale, seg_chunks, num_slots)
    ins = (q, k, v, g, cu_seqlens, h0)
    if out is not None:
        _check_out("out", out, tuple(v.shape), v.dtype, device)
        _no_overlap("out", out, *ins)
    if final_state is not None:
        _check_out("final_state", final_state, (N, H, D, D), torch.float32, device)
        _no_overlap("final_state", final_state, out, *ins)
    lib = load_library()
    with _on(device):
        nbytes = _workspace_bytes(lib.gdn_linattn_fwd_workspace_size, p)
        ws = _workspace(workspace, nbytes, device) if nbytes or workspace is not None else None
        o = out if out is not None else torch.empty_like(v)
        ht = None
        if output_final_state:
            ht = final_state if final_state is not None else torch.empty(
                (N, H, D, D), dtype=torch.float32, device=device)
        _check(lib.gdn_linattn_fwd(ctypes.byref(p), _at(q), _at(k), _at(v), _at(g),
                                   _at(cu_seqlens), _at(h0), _at(o), _at(ht), _at(ws),
                                   0 if ws is None else _nbytes(ws), _stream_of(device)))
    return o, ht


def linattn_bwd(q, k, v, g, cu_seqlens, dout, h0=None, dht=None, *, scale=1.0, need_dh0=True,
                seg_chunks=0, num_slots=0, workspace=None):
    """Backward of :func:`linattn_fwd` for dout [T, H, D] (q's dtype) and optionally the final
    states' gradient dht fp32 [N, H, D, D].  Returns dict(dq, dk, dv, dg, dh0): dq, dk summed over
    the value heads that share a key head, dg fp32 in g's shape, dh0 fp32 [N, H, D, D], or [H, D, D]
    summed over the sequences when h0 is shared (None without need_dh0)."""
    p, device, N, H, D = _problem(q, k, v, g, cu_seqlens, h0, scale, seg_chunks, num_slots)
    if tuple(dout.shape) != tuple(v.shape) or dout.dtype != q.dtype:
        raise ValueError("dout must have v's shape and q's dtype")
    if dht is not None and (tuple(dht.shape) != (N, H, D, D) or dht.dtype != torch.float32):
        raise ValueError("dht must be float32 [N, H, D, D]")
    _same_device(device, dout=dout, dht=dht)
    lib = load_library()
    with _on(device):
        ws = _workspace(workspace, _workspace_bytes(lib.gdn_linattn_bwd_workspace_size, p), device)
        res = dict(dq=torch.empty_like(q), dk=torch.empty_like(k), dv=torch.empty_like(v),
                   dg=torch.empty_like(g), dh0=None)
        if need_dh0:
            res["dh0"] = torch.empty((H, D, D) if p.h0_seq_stride == 0 else (N, H, D, D),
                                     dtype=torch.float32, device=device)
        _check(lib.gdn_linattn_bwd(ctypes.byref(p), _at(q), _at(k), _at(v), _at(g), _at(cu_seqlens),
                                   _at(h0), _at(dout), _at(dht), _at(res["dq"]), _at(res["dk"]),
                                   _at(res["dv"]), _at(res["dg"]), _at(res["dh0"]), _at(ws),
                                   _nbytes(ws), _stream_of(device)))
    return res


def linattn_step(q, k, v, g, state, pages=None, *, scale=1.0, out=None):
    """One token per row, the states advanced in place: q, k [B, Hk, D], v [B, H, D], g [B, H] or
    [H].  Without ``pages`` state is [B, H, D, D]; with pages (int32 [B]) state is a pool
    [P, H, D, D] and row b's state is state[pages[b]], -1 marking a row without a sequence (its
    output is zero).  Returns o [B, H, D]."""
    B, H, Hk, D, head = _heads(q, k, v, g, "B")
    dtype = _dtype_of(q)
    if state.dtype != torch.float32 or state.dim() != 4 or state.shape[1:] != (H, D, D) or \
            (pages is None and state.shape[0] != B):
        raise ValueError("state must be float32 [B, H, D, D], or a pool [P, H, D, D] with pages")
    if pages is not None and (pages.dtype != torch.int32 or pages.shape != (B,)):
        raise ValueError("pages must be int32 [B]")
    device = _device_of(q)
    _same_device(device, q=q, k=k, v=v, g=g, state=state, pages=pages)
    if out is not None:
        _check_out("out", out, tuple(v.shape), v.dtype, device)
        _no_overlap("out", out, q, k, v, g, state, pages)
    lib = load_library()
    with _on(device):
        o = out if out is not None else torch.empty_like(v)
        _check(lib.gdn_linattn_step(B, H, Hk, D, dtype, head, scale, _at(q), _at(k), _at(v), _at(g),
                                    _at(pages), state.shape[0], _at(state), _at(o),
                                    _stream_of(device)))
    return o


def linattn_fwd_workspace_bytes(q, k, v, g, cu_seqlens, h0=None, *, seg_chunks=0, num_slots=0):
    """Workspace bytes of :func:`linattn_fwd` for these tensors (gdn_linattn_fwd_workspace_size)."""
    p = _problem(q, k, v, g, cu_seqlens, h0, 1.0, seg_chunks, num_slots)[0]
    with _on(q.device):
        return _workspace_bytes(load_library().gdn_linattn_fwd_workspace_size, p)


def linattn_bwd_workspace_bytes(q, k, v, g, cu_seqlens, h0=None, *, seg_chunks=0, num_slots=0):
    """Workspace bytes of :func:`linattn_bwd` for these tensors (gdn_linattn_bwd_workspace_size)."""
    p = _problem(q, k, v, g, cu_seqlens, h0, 1.0, seg_chunks, num_slots)[0]
    with _on(q.device):
        return _workspace_bytes(load_library().gdn_linattn_bwd_workspace_size, p)


def _declare(lib):
    vp, sz, i32, f32 = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int32, ctypes.c_float
    P, st = ctypes.POINTER(LinattnProblem), ctypes.c_int
    for fn in (lib.gdn_linattn_fwd_workspace_size, lib.gdn_linattn_bwd_workspace_size):
        fn.argtypes, fn.restype = [P, ctypes.POINTER(sz)], st
    lib.gdn_linattn_fwd.argtypes = [P] + [vp] * 9 + [sz, vp]
    lib.gdn_linattn_fwd.restype = st
    lib.gdn_linattn_bwd.argtypes = [P] + [vp] * 14 + [sz, vp]
    lib.gdn_linattn_bwd.restype = st
    lib.gdn_linattn_step.argtypes = [i32] * 6 + [f32] + [vp] * 5 + [i32] + [vp] * 3
    lib.gdn_linattn_step.restype = st


# The C entry points' names (include/gdn_linattn.h).
gdn_linattn_fwd = linattn_fwd
gdn_linattn_bwd = linattn_bwd
gdn_linattn_step = linattn_step
gdn_linattn_fwd_workspace_size = linattn_fwd_workspace_bytes
gdn_linattn_bwd_workspace_size = linattn_bwd_workspace_bytes
