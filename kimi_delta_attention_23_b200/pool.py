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

from . import KdaError, _MOST, _dev, _extents, _hand_over, _launch, _make, _need, _need_rank, _on_stream, load_library

__all__ = ["kda_pool_copy", "kda_pool_fork", "kda_pool_free", "kda_pool_compact", "kda_pool_workspace_size",
           "MAX_POOL_COPIES"]

MAX_POOL_COPIES = 8192  # pairs of one kda_pool_copy
FEW_COPIES = 256  # up to so many it takes one launch and no workspace

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
    """The pool itself, its device's number, and its layers, slots and elements per slot."""
    shape, lead = getattr(pool, "shape", ()), 2 if stacked else 1
    if len(shape) <= lead or pool.dtype is not torch.float32 or not pool.is_cuda or not pool.is_contiguous() or not pool.numel():
        _dev(pool, "state_pool", torch.float32)
        raise ValueError(f"state_pool has shape {tuple(shape)}, expected "
                         f"{'[layers, slots, ...]' if stacked else '[slots, ...]'} with at least one element")
    layers, slots = (shape[0], shape[1]) if stacked else (1, shape[0])
    if slots > _MOST or layers > _MOST:
        _extents((layers, slots), "state_pool")
    return pool, pool.get_device(), layers, slots, pool.numel() // (layers * slots)


def _list(t, name, pool, index, n=None):
    """The length and address of a list of slots."""
    if n is not None:
        return n, _need(t, name, torch.int32, (n,), pool, index)
    (n,), at = _need_rank(t, name, torch.int32, 1, pool, index)
    return n, at


def _call(what, pool, layout, lists, n, results, workspace, device_status, stream, made=()):
    _, index, layers, slots, elems = layout
    lib = load_library()
    status = None if device_status is None else _need(device_status, "device_status", torch.int32, (1,), pool, index)
    if workspace is not None:
        _dev(workspace, "workspace", torch.uint8, pool.device)
    elif what != "kda_pool_copy" or n > FEW_COPIES:
        need = lib.kda_pool_workspace_size(n, slots)
        workspace = _make(stream, index, torch.empty, need, dtype=torch.uint8, device=pool.device)
    at, size = (None, 0) if workspace is None else (workspace.data_ptr(), workspace.numel())
    rc = _launch(index, getattr(lib, what), pool.data_ptr(), layers, slots, elems, *lists, n, *results, at, size, status,
                 _on_stream(stream, index))
    _hand_over(stream, index, *made)
    if rc != 0:
        raise KdaError(rc, what)


def kda_pool_copy(state_pool, src, dst, *, stacked=False, workspace=None, device_status=None, stream=None):
    """Slot dst[i] = slot src[i] for all i, as one simultaneous assignment (swaps and chains included).

    ``src``, ``dst`` [n] i32, n <= 8192.  Slots out of range, and a destination that is named again
    (its first pair counts), are reported in ``device_status`` and skipped.
    """
    layout = _, index, _, _, _ = _layout(state_pool, stacked)
    n, srcs = _list(src, "src", state_pool, index)
    _, dsts = _list(dst, "dst", state_pool, index, n)
    if n > MAX_POOL_COPIES:
        raise ValueError(f"at most {MAX_POOL_COPIES} pairs per call, got {n}")
    _call("kda_pool_copy", state_pool, layout, (srcs, dsts), n, (), workspace, device_status, stream)


def kda_pool_fork(state_pool, live, src, dst=None, *, stacked=False, workspace=None, device_status=None, stream=None):
    """Every slot src[i] copied to a free slot of its own, which becomes live; returns dst [n] i32.

    The lowest free slots are taken in the order of the list.  A source that is not live, or one for
    which no slot is left, is reported in ``device_status`` and gets -1.
    """
    layout = _, index, _, slots, _ = _layout(state_pool, stacked)
    _, lives = _list(live, "live", state_pool, index, slots)
    n, srcs = _list(src, "src", state_pool, index)
    made = ()
    if dst is None:
        dst = _make(stream, index, torch.empty_like, src)
        made = (dst,)
    _, dsts = _list(dst, "dst", state_pool, index, n)
    _call("kda_pool_fork", state_pool, layout, (lives, srcs, dsts), n, (), workspace, device_status, stream, made)
    return dst


def kda_pool_free(state_pool, live, slots, *, stacked=False, workspace=None, device_status=None, stream=None):
    """The listed slots marked free and cleared to zero, the state a new sequence starts from.

    A slot that is not live, or is listed again, is reported in ``device_status`` and left alone.
    """
    layout = _, index, _, max_slots, _ = _layout(state_pool, stacked)
    _, lives = _list(live, "live", state_pool, index, max_slots)
    n, listed = _list(slots, "slots", state_pool, index)
    _call("kda_pool_free", state_pool, layout, (lives, listed), n, (), workspace, device_status, stream)


def kda_pool_compact(state_pool, live, state_indices, num_live=None, *, stacked=False, workspace=None,
                     device_status=None, stream=None):
    """Live slots moved down so that they fill the pool from slot 0; returns num_live [1] i32.

    The j-th empty slot below the number of live ones receives the j-th live slot above it.
    ``state_indices`` [n] i32 (any list of slots in use) and ``live`` are rewritten in place to the
    new places; an index that names no live slot is reported in ``device_status`` and kept.  What is
    left in the slots above is unspecified.
    """
    layout = _, index, _, slots, _ = _layout(state_pool, stacked)
    _, lives = _list(live, "live", state_pool, index, slots)
    n, indices = _list(state_indices, "state_indices", state_pool, index)
    made = ()
    if num_live is None:
        num_live = _make(stream, index, torch.empty, 1, dtype=torch.int32, device=state_pool.device)
        made = (num_live,)
    _, counts = _list(num_live, "num_live", state_pool, index, 1)
    _call("kda_pool_compact", state_pool, layout, (lives, indices), n, (counts,), workspace, device_status, stream, made)
    return num_live
