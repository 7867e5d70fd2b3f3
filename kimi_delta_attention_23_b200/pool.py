"""Slots of a state pool copied, forked, freed and packed.

A pool is a float32 tensor [slots, ...] (KDA's [slots, Hv, dk, dv] or the recurrence's [slots, H, d]),
or with ``stacked`` the pools of several layers that share their slot numbers, [layers, slots, ...].
``live`` [slots] i32 marks the slots in use (nonzero).  Which slots are free is decided on the device:
no call waits for it, and all of them can be captured in a CUDA graph.  Entries of -1 in the lists
are padding.
"""
from __future__ import annotations

import ctypes

import torch

from . import KdaError, _dev, _on_device, _Owned, _ptr, _shape, _stream, load_library

__all__ = ["kda_pool_copy", "kda_pool_fork", "kda_pool_free", "kda_pool_compact", "kda_pool_workspace_size",
           "MAX_POOL_COPIES"]

MAX_POOL_COPIES = 8192  # pairs of one kda_pool_copy

_vp, _i32, _i64, _sz, _int = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t, ctypes.c_int
SIGNATURES = {
    "kda_pool_workspace_size": (_sz, [_i32, _i32]),
    "kda_pool_copy": (_int, [_vp, _i32, _i32, _i64, _vp, _vp, _i32, _vp, _sz, _vp, _vp]),
    "kda_pool_fork": (_int, [_vp, _i32, _i32, _i64, _vp, _vp, _vp, _i32, _vp, _sz, _vp, _vp]),
    "kda_pool_free": (_int, [_vp, _i32, _i32, _i64, _vp, _vp, _i32, _vp, _sz, _vp, _vp]),
    "kda_pool_compact": (_int, [_vp, _i32, _i32, _i64, _vp, _vp, _i32, _vp, _vp, _sz, _vp, _vp]),
}


def kda_pool_workspace_size(n, max_slots) -> int:
    """Workspace bytes of a call with lists of n entries."""
    return int(load_library().kda_pool_workspace_size(n, max_slots))


def _layout(pool, stacked):
    _dev(pool, "state_pool", torch.float32)
    lead = 2 if stacked else 1
    if pool.dim() < lead + 1 or pool.numel() == 0:
        raise ValueError(f"state_pool has shape {tuple(pool.shape)}, expected "
                         f"{'[layers, slots, ...]' if stacked else '[slots, ...]'} with at least one element")
    layers, slots = (pool.shape[0], pool.shape[1]) if stacked else (1, pool.shape[0])
    return pool.device, layers, slots, pool.numel() // (layers * slots)


def _list(t, name, dev, n=None):
    _dev(t, name, torch.int32, dev)
    if t.dim() != 1:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected one dimension")
    if n is not None:
        _shape(t, name, (n,))
    return t.numel()


def _call(what, pool, layers, slots, elems, lists, n, results, workspace, device_status, stream, own, dev):
    lib = load_library()
    if device_status is not None:
        _shape(_dev(device_status, "device_status", torch.int32, dev), "device_status", (1,))
    with _on_device(dev):
        if workspace is None:
            workspace = own.empty(lib.kda_pool_workspace_size(n, slots), dtype=torch.uint8, device=dev)
        _dev(workspace, "workspace", torch.uint8, dev)
        rc = getattr(lib, what)(_ptr(pool), layers, slots, elems, *[_ptr(t) for t in lists], n,
                                *[_ptr(t) for t in results], _ptr(workspace), workspace.numel(), _ptr(device_status),
                                _stream(stream, dev))
    own.launched()
    if rc != 0:
        raise KdaError(rc, what)


def kda_pool_copy(state_pool, src, dst, *, stacked=False, workspace=None, device_status=None, stream=None):
    """Slot dst[i] = slot src[i] for all i, as one simultaneous assignment (swaps and chains included).

    ``src``, ``dst`` [n] i32, n <= 8192.  Slots out of range, and a destination that is named again
    (its first pair counts), are reported in ``device_status`` and skipped.
    """
    dev, layers, slots, elems = _layout(state_pool, stacked)
    n = _list(src, "src", dev)
    _list(dst, "dst", dev, n)
    if n > MAX_POOL_COPIES:
        raise ValueError(f"at most {MAX_POOL_COPIES} pairs per call, got {n}")
    _call("kda_pool_copy", state_pool, layers, slots, elems, (src, dst), n, (), workspace, device_status, stream,
          _Owned(stream, dev), dev)


def kda_pool_fork(state_pool, live, src, dst=None, *, stacked=False, workspace=None, device_status=None, stream=None):
    """Every slot src[i] copied to a free slot of its own, which becomes live; returns dst [n] i32.

    The lowest free slots are taken in the order of the list.  A source that is not live, or one for
    which no slot is left, is reported in ``device_status`` and gets -1.
    """
    dev, layers, slots, elems = _layout(state_pool, stacked)
    own = _Owned(stream, dev)
    _list(live, "live", dev, slots)
    n = _list(src, "src", dev)
    if dst is None:
        dst = own.empty(n, dtype=torch.int32, device=dev)
    _list(dst, "dst", dev, n)
    _call("kda_pool_fork", state_pool, layers, slots, elems, (live, src, dst), n, (), workspace, device_status, stream,
          own, dev)
    return dst


def kda_pool_free(state_pool, live, slots, *, stacked=False, workspace=None, device_status=None, stream=None):
    """The listed slots marked free and cleared to zero, the state a new sequence starts from.

    A slot that is not live, or is listed again, is reported in ``device_status`` and left alone.
    """
    dev, layers, max_slots, elems = _layout(state_pool, stacked)
    _list(live, "live", dev, max_slots)
    n = _list(slots, "slots", dev)
    _call("kda_pool_free", state_pool, layers, max_slots, elems, (live, slots), n, (), workspace, device_status, stream,
          _Owned(stream, dev), dev)


def kda_pool_compact(state_pool, live, state_indices, num_live=None, *, stacked=False, workspace=None,
                     device_status=None, stream=None):
    """Live slots moved down so that they fill the pool from slot 0; returns num_live [1] i32.

    The j-th empty slot below the number of live ones receives the j-th live slot above it.
    ``state_indices`` [n] i32 (any list of slots in use) and ``live`` are rewritten in place to the
    new places; an index that names no live slot is reported in ``device_status`` and kept.  What is
    left in the slots above is unspecified.
    """
    dev, layers, slots, elems = _layout(state_pool, stacked)
    own = _Owned(stream, dev)
    _list(live, "live", dev, slots)
    n = _list(state_indices, "state_indices", dev)
    if num_live is None:
        num_live = own.empty(1, dtype=torch.int32, device=dev)
    _list(num_live, "num_live", dev, 1)
    _call("kda_pool_compact", state_pool, layers, slots, elems, (live, state_indices), n, (num_live,), workspace,
          device_status, stream, own, dev)
    return num_live
