"""KDA over trees of drafted tokens, and the accepted path written into the state.

A step of speculative decoding checks, for every sequence, a tree of drafted tokens against the
sequence's state: ``kda_tree_decode`` reads each state once and returns every node's output, leaving
the pool as it was; when the accepted node is known, ``kda_tree_commit`` advances each state along
the path to it.  With kda_pool_fork and kda_pool_free next to them, samples can part ways.
"""
from __future__ import annotations

import ctypes

import torch

from . import (_DTYPES, KdaError, _dev, _flags, _on_device, _Owned, _ptr, _shape, _stream, load_library)

__all__ = ["kda_tree_decode", "kda_tree_commit", "MAX_TREE_NODES"]

MAX_TREE_NODES = 64  # drafted tokens of one sequence

_vp, _i32, _i64, _u32, _f32, _int = (ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_uint32, ctypes.c_float,
                                     ctypes.c_int)
SIGNATURES = {
    "kda_tree_decode": (_int, [_vp, _vp, _vp, _int, _vp, _vp, _vp, _vp, _vp, _vp, _i32, _i64, _i32, _i32, _i32, _i32, _i32,
                               _vp, _i32, _vp, _vp, _int, _vp, _u32, _f32, _vp, _vp]),
    "kda_tree_commit": (_int, [_vp, _int, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i32, _i64, _i32, _i32, _i32, _i32, _i32, _vp,
                               _i32, _vp, _u32, _f32, _vp, _vp]),
}


def _tree(cu_nodes, parents, max_nodes, M, dev):
    _dev(cu_nodes, "cu_nodes", torch.int32, dev)
    if cu_nodes.dim() != 1 or cu_nodes.numel() < 1:
        raise ValueError("cu_nodes must hold B + 1 offsets")
    _shape(_dev(parents, "parents", torch.int32, dev), "parents", (M,))
    if max_nodes is None:
        max_nodes = max(1, min(M, MAX_TREE_NODES))
    if not 1 <= max_nodes <= MAX_TREE_NODES:
        raise ValueError(f"max_nodes must be 1 .. {MAX_TREE_NODES}, got {max_nodes}")
    return cu_nodes.numel() - 1, int(max_nodes)


def _pool(state_pool, state_indices, state_layout, dev, B, Hv, dk, dv):
    blk = (Hv, dk, dv) if state_layout == "K_FIRST" else (Hv, dv, dk)
    _dev(state_pool, "state_pool", torch.float32, dev)
    if state_pool.dim() != 4 or tuple(state_pool.shape[1:]) != blk:
        raise ValueError(f"state_pool has shape {tuple(state_pool.shape)}, expected [slots, {blk}]")
    _shape(_dev(state_indices, "state_indices", torch.int32, dev), "state_indices", (B,))


def kda_tree_decode(q, k, v, raw_gate, beta_logits, a_log, dt_bias, cu_nodes, parents, state_pool, state_indices,
                    out=None, deltas=None, *, max_nodes=None, output_dtype=None, gate_mode="original",
                    beta_mode="logits", state_layout="K_FIRST", gate_lower_bound=-5.0, device_status=None, stream=None):
    """Outputs of all drafted tokens; the states are only read.

    Sequence b drafts the nodes cu_nodes[b] .. cu_nodes[b+1] - 1; ``parents`` [M] i32 numbers each
    node's parent within its sequence (smaller than the node's own number; -1: the node follows the
    state).  Shapes: q, k [M,Hk,dk]; v [M,Hv,dv]; raw_gate [M,Hv,dk] f32; beta_logits [M,Hv] f32;
    a_log, dt_bias, state_pool and state_indices [B] as kda_decode.  ``max_nodes`` (1 .. 64): no
    sequence drafts more (a longer one is reported in ``device_status`` and skipped; the default is
    M, at most 64); naming it close to the real size takes a smaller kernel.  Returns (out [M,Hv,dv],
    deltas [M,Hv,dv] f32), the second for kda_tree_commit.
    """
    lib = load_library()
    dev = _dev(q, "q").device
    own = _Owned(stream, dev)
    if q.dtype not in _DTYPES:
        raise ValueError("q/k/v must be float32 or bfloat16")
    if q.dim() != 3:
        raise ValueError(f"q has shape {tuple(q.shape)}, expected [M, Hk, dk]")
    M, Hk, dk = q.shape
    _shape(_dev(k, "k", q.dtype, dev), "k", (M, Hk, dk))
    _dev(v, "v", q.dtype, dev)
    if v.dim() != 3 or v.shape[0] != M:
        raise ValueError(f"v has shape {tuple(v.shape)}, expected [{M}, Hv, dv]")
    Hv, dv = v.shape[1], v.shape[2]
    _shape(_dev(raw_gate, "raw_gate", torch.float32, dev), "raw_gate", (M, Hv, dk))
    _shape(_dev(beta_logits, "beta_logits", torch.float32, dev), "beta_logits", (M, Hv))
    _shape(_dev(a_log, "a_log", torch.float32, dev), "a_log", (Hv,))
    _shape(_dev(dt_bias, "dt_bias", torch.float32, dev), "dt_bias", (Hv, dk))
    B, max_nodes = _tree(cu_nodes, parents, max_nodes, M, dev)
    flags = _flags(gate_mode, beta_mode, state_layout)
    _pool(state_pool, state_indices, state_layout, dev, B, Hv, dk, dv)
    if output_dtype is None:
        output_dtype = v.dtype if out is None else out.dtype
    if output_dtype not in _DTYPES:
        raise ValueError("output_dtype must be float32 or bfloat16")
    if out is None:
        out = own.empty((M, Hv, dv), dtype=output_dtype, device=dev)
    _shape(_dev(out, "out", output_dtype, dev), "out", (M, Hv, dv))
    if deltas is None:
        deltas = own.empty((M, Hv, dv), dtype=torch.float32, device=dev)
    _shape(_dev(deltas, "deltas", torch.float32, dev), "deltas", (M, Hv, dv))
    if device_status is not None:
        _shape(_dev(device_status, "device_status", torch.int32, dev), "device_status", (1,))
    with _on_device(dev):
        rc = lib.kda_tree_decode(_ptr(q), _ptr(k), _ptr(v), _DTYPES[q.dtype], _ptr(raw_gate), _ptr(beta_logits),
                                 _ptr(a_log), _ptr(dt_bias), _ptr(cu_nodes), _ptr(parents), B, M, max_nodes, Hk, Hv,
                                 dk, dv, _ptr(state_pool), state_pool.shape[0], _ptr(state_indices), _ptr(out),
                                 _DTYPES[output_dtype], _ptr(deltas), flags, float(gate_lower_bound),
                                 _ptr(device_status), _stream(stream, dev))
    own.launched()
    if rc != 0:
        raise KdaError(rc, "kda_tree_decode")
    return out, deltas


def kda_tree_commit(k, raw_gate, a_log, dt_bias, deltas, cu_nodes, parents, accepted, state_pool, state_indices, *,
                    max_nodes=None, gate_mode="original", state_layout="K_FIRST", gate_lower_bound=-5.0,
                    device_status=None, stream=None):
    """Every state advanced along its tree's accepted path, in place.

    ``accepted`` [B] i32: the last accepted node of each sequence, numbered within it (-1: none, the
    state stays).  The other tensors as in the kda_tree_decode call that returned ``deltas``.
    """
    lib = load_library()
    dev = _dev(k, "k").device
    if k.dtype not in _DTYPES:
        raise ValueError("k must be float32 or bfloat16")
    if k.dim() != 3:
        raise ValueError(f"k has shape {tuple(k.shape)}, expected [M, Hk, dk]")
    M, Hk, dk = k.shape
    _dev(deltas, "deltas", torch.float32, dev)
    if deltas.dim() != 3 or deltas.shape[0] != M:
        raise ValueError(f"deltas has shape {tuple(deltas.shape)}, expected [{M}, Hv, dv]")
    Hv, dv = deltas.shape[1], deltas.shape[2]
    _shape(_dev(raw_gate, "raw_gate", torch.float32, dev), "raw_gate", (M, Hv, dk))
    _shape(_dev(a_log, "a_log", torch.float32, dev), "a_log", (Hv,))
    _shape(_dev(dt_bias, "dt_bias", torch.float32, dev), "dt_bias", (Hv, dk))
    B, max_nodes = _tree(cu_nodes, parents, max_nodes, M, dev)
    _shape(_dev(accepted, "accepted", torch.int32, dev), "accepted", (B,))
    flags = _flags(gate_mode, "logits", state_layout)
    _pool(state_pool, state_indices, state_layout, dev, B, Hv, dk, dv)
    if device_status is not None:
        _shape(_dev(device_status, "device_status", torch.int32, dev), "device_status", (1,))
    with _on_device(dev):
        rc = lib.kda_tree_commit(_ptr(k), _DTYPES[k.dtype], _ptr(raw_gate), _ptr(a_log), _ptr(dt_bias), _ptr(deltas),
                                 _ptr(cu_nodes), _ptr(parents), _ptr(accepted), B, M, max_nodes, Hk, Hv, dk, dv,
                                 _ptr(state_pool), state_pool.shape[0], _ptr(state_indices), flags,
                                 float(gate_lower_bound), _ptr(device_status), _stream(stream, dev))
    if rc != 0:
        raise KdaError(rc, "kda_tree_commit")
