"""Operators on the pages of a pool (``include/gdn_pages.h``): copy, fork, free and compact.

A pool is any contiguous device tensor whose first axis counts pages, for instance recurrent states
[P, H, D, D]; its ``live`` flags are int32 [P], 0 for a free page.  Page numbers are int32 device
tensors, read on the device: no call waits for the host.  A page number that a call cannot take
sets a fault flag (``device_faults()``: ``FAULT_PAGE_*``) and its entry is left out.
"""
from __future__ import annotations

import ctypes
import functools

import torch

from .gdn import _check, _nbytes, _workspace, load_library
from .linattn import _at, _on, _same_device, _stream_of

# Bits of device_faults() that page numbers can set.
FAULT_PAGE_RANGE, FAULT_PAGE_TWICE, FAULT_NO_PAGE = 2, 4, 8


def _pool(name, pool):
    if pool.dim() < 2 or not pool.is_cuda or not pool.is_contiguous() or pool.shape[0] < 1:
        raise ValueError(f"{name} must be a contiguous device tensor [pages, ...]")
    nbytes = _nbytes(pool) // pool.shape[0]
    if nbytes < 16 or nbytes % 16 != 0:
        raise ValueError(f"a page of {name} must be a positive multiple of 16 bytes")
    return pool.shape[0], nbytes


def _index(name, x, shape=None):
    if x.dtype != torch.int32 or x.dim() != 1 or (shape is not None and tuple(x.shape) != shape):
        raise ValueError(f"{name} must be a 1-D int32 tensor" +
                         (f" of {shape[0]} entries" if shape is not None else ""))


@functools.lru_cache(maxsize=256)
def pages_workspace_bytes(num_pages, count):
    """Workspace bytes of the calls below (gdn_pages_workspace_size)."""
    n = ctypes.c_size_t(0)
    _check(load_library().gdn_pages_workspace_size(int(num_pages), int(count), ctypes.byref(n)))
    return n.value


def pages_copy(dst, src, dst_pages, src_pages, *, workspace=None):
    """dst[dst_pages[i]] = src[src_pages[i]]; a source of -1 writes zeros, a destination of -1 skips
    the pair.  dst and src are one pool (or the pool and its first pages) or do not overlap.  Of pairs
    with one destination the first is done; in one pool a pair whose source is another pair's
    destination is left out.  Returns dst."""
    P, nbytes = _pool("dst", dst)
    Ps, nb_src = _pool("src", src)
    if nb_src != nbytes or src.dtype != dst.dtype:
        raise ValueError("dst and src must have pages of the same type and size")
    _index("dst_pages", dst_pages)
    _index("src_pages", src_pages, tuple(dst_pages.shape))
    _same_device(dst.device, src=src, dst_pages=dst_pages, src_pages=src_pages)
    lib = load_library()
    n = dst_pages.numel()
    with _on(dst.device):
        ws = _workspace(workspace, pages_workspace_bytes(P, n), dst.device)
        _check(lib.gdn_pages_copy(_at(dst), P, _at(src), Ps, nbytes, _at(dst_pages),
                                  _at(src_pages), n, _at(ws), _nbytes(ws),
                                  _stream_of(dst.device)))
    return dst


def pages_fork(pool, live, parents, *, children=None, workspace=None):
    """Takes the lowest free page for each parent in order, copies the parent's page to it (zeros for
    a parent of -1) and marks it live.  Returns children, int32 like parents: the pages taken, -1
    where no page was free or the parent is not a live page."""
    P, nbytes = _pool("pool", pool)
    _index("live", live, (P,))
    _index("parents", parents)
    if children is not None:
        _index("children", children, tuple(parents.shape))
    _same_device(pool.device, live=live, parents=parents, children=children)
    lib = load_library()
    with _on(pool.device):
        res = children if children is not None else torch.empty_like(parents)
        ws = _workspace(workspace, pages_workspace_bytes(P, 0), pool.device)
        _check(lib.gdn_pages_fork(_at(pool), _at(live), P, nbytes, _at(parents), parents.numel(),
                                  _at(res), _at(ws), _nbytes(ws), _stream_of(pool.device)))
    return res


def pages_free(live, pages):
    """Marks pages free in ``live`` (entries of -1 are skipped)."""
    if not live.is_cuda:
        raise ValueError("live must be a contiguous device tensor")
    _index("live", live)
    _index("pages", pages)
    _same_device(live.device, live=live, pages=pages)
    lib = load_library()
    with _on(live.device):
        _check(lib.gdn_pages_free(_at(live), live.numel(), _at(pages), pages.numel(),
                                  _stream_of(live.device)))


def pages_compact(pool, live, *, workspace=None):
    """Moves the live pages to the front of the pool with the fewest copies.  Returns remap, int32
    [P]: where each page went, -1 for a free one."""
    P, nbytes = _pool("pool", pool)
    _index("live", live, (P,))
    _same_device(pool.device, live=live)
    lib = load_library()
    with _on(pool.device):
        remap = torch.empty_like(live)
        ws = _workspace(workspace, pages_workspace_bytes(P, 0), pool.device)
        _check(lib.gdn_pages_compact(_at(pool), _at(live), P, nbytes, _at(remap), _at(ws),
                                     _nbytes(ws), _stream_of(pool.device)))
    return remap


def _declare(lib):
    vp, sz, i32, i64, st = (ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int32, ctypes.c_int64,
                            ctypes.c_int)
    lib.gdn_pages_workspace_size.argtypes = [i32, i32, ctypes.POINTER(sz)]
    lib.gdn_pages_copy.argtypes = [vp, i32, vp, i32, i64, vp, vp, i32, vp, sz, vp]
    lib.gdn_pages_fork.argtypes = [vp, vp, i32, i64, vp, i32, vp, vp, sz, vp]
    lib.gdn_pages_free.argtypes = [vp, i32, vp, i32, vp]
    lib.gdn_pages_compact.argtypes = [vp, vp, i32, i64, vp, vp, sz, vp]
    for name in ("workspace_size", "copy", "fork", "free", "compact"):
        getattr(lib, "gdn_pages_" + name).restype = st


# The C entry points' names (include/gdn_pages.h).
gdn_pages_workspace_size = pages_workspace_bytes
gdn_pages_copy = pages_copy
gdn_pages_fork = pages_fork
gdn_pages_free = pages_free
gdn_pages_compact = pages_compact
