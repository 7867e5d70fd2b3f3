"""KDA over trees of drafted tokens, and the accepted path written into the state.

A step of speculative decoding checks, for every sequence, a tree of drafted tokens against the
sequence's state: ``kda_tree_decode`` reads each state once and returns every node's output, leaving
the pool as it was; when the accepted node is known, ``kda_tree_commit`` advances each state along
the path to it.  With kda_pool_fork and kda_pool_free next to them, samples can part ways.
"""
from __future__ import annotations

import ctypes

import torch

from . import (_checker, _DTYPES, KdaError, _flags, _hand_over, _launch, _make, _need, _need_rank, _on_stream, _where,
               load_library)

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


_BLOCKS = {"K_FIRST": "S,Hv,dk,dv", "V_FIRST": "S,Hv,dv,dk"}
_TREE = {layout: _checker("q v M,Hk,dk; k s M,Hk,dk; v s M,Hv,dv; raw f M,Hv,dk; beta f M,Hv; a_log f Hv; dt_bias f Hv,dk; "
                          f"cu i B+1; parents i M; pool f {block}; idx i B") for layout, block in _BLOCKS.items()}
_COMMIT = {layout: _checker("k v M,Hk,dk; deltas f M,Hv,dv; raw f M,Hv,dk; a_log f Hv; dt_bias f Hv,dk; cu i B+1; parents i M; "
                            f"accepted i B; pool f {block}; idx i B") for layout, block in _BLOCKS.items()}
_FLAGS = {}


def _tree_flags(gate_mode, beta_mode, state_layout):
    key = (gate_mode, beta_mode, state_layout)
    if key not in _FLAGS:
        _FLAGS[key] = _flags(*key)
    return _FLAGS[key]


def _tree(cu_nodes, parents, M, like, index):
    (count,), cu = _need_rank(cu_nodes, "cu_nodes", torch.int32, 1, like, index)
    if count < 1:
        raise ValueError("cu_nodes must hold B + 1 offsets")
    return count - 1, cu, _need(parents, "parents", torch.int32, (M,), like, index)


def _most(max_nodes, M):
    if max_nodes is None:
        return max(1, min(M, MAX_TREE_NODES))
    if not 1 <= max_nodes <= MAX_TREE_NODES:
        raise ValueError(f"max_nodes must be 1 .. {MAX_TREE_NODES}, got {max_nodes}")
    return int(max_nodes)


def _pool(state_pool, state_indices, state_layout, like, index, B, Hv, dk, dv):
    shape, at = _need_rank(state_pool, "state_pool", torch.float32, 4, like, index)
    if shape[1:] != ((Hv, dk, dv) if state_layout == "K_FIRST" else (Hv, dv, dk)):
        raise ValueError(f"state_pool has shape {tuple(shape)}, expected [slots, {Hv}] and blocks of {dk} keys by {dv} "
                         f"values stored {state_layout}")
    return at, shape[0], _need(state_indices, "state_indices", torch.int32, (B,), like, index)


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
    lib, flags = load_library(), _tree_flags(gate_mode, beta_mode, state_layout)
    found = _TREE[state_layout](q, k, v, raw_gate, beta_logits, a_log, dt_bias, cu_nodes, parents, state_pool, state_indices)
    if found is None:
        index, (M, Hk, dk), qs = _where(q, "q", 3)
        dtype = q.dtype
        if dtype not in _DTYPES:
            raise ValueError("q/k/v must be float32 or bfloat16")
        ks = _need(k, "k", dtype, (M, Hk, dk), q, index)
        (rows, Hv, dv), vs = _need_rank(v, "v", dtype, 3, q, index)
        if rows != M:
            raise ValueError(f"v has shape {tuple(v.shape)}, expected [{M}, Hv, dv]")
        raws = _need(raw_gate, "raw_gate", torch.float32, (M, Hv, dk), q, index)
        betas = _need(beta_logits, "beta_logits", torch.float32, (M, Hv), q, index)
        alogs = _need(a_log, "a_log", torch.float32, (Hv,), q, index)
        biases = _need(dt_bias, "dt_bias", torch.float32, (Hv, dk), q, index)
        B, cu, pars = _tree(cu_nodes, parents, M, q, index)
        pool, slots, indices = _pool(state_pool, state_indices, state_layout, q, index, B, Hv, dk, dv)
        in_type = _DTYPES[dtype]
    else:
        index, M, Hk, dk, Hv, dv, B, slots, qs, ks, vs, raws, betas, alogs, biases, cu, pars, pool, indices, in_type = found
    max_nodes = _most(max_nodes, M)
    if output_dtype is None:
        output_dtype = v.dtype if out is None else out.dtype
    if output_dtype not in _DTYPES:
        raise ValueError("output_dtype must be float32 or bfloat16")
    status = None if device_status is None else _need(device_status, "device_status", torch.int32, (1,), q, index)
    new_out, new_deltas = out is None, deltas is None
    if new_out:
        out = _make(stream, index, torch.empty_like, v, dtype=output_dtype)
    if new_deltas:
        deltas = _make(stream, index, torch.empty_like, v, dtype=torch.float32)
    rc = _launch(index, lib.kda_tree_decode, qs, ks, vs, in_type, raws, betas, alogs, biases, cu, pars, B, M, max_nodes, Hk,
                 Hv, dk, dv, pool, slots, indices,
                 out.data_ptr() if new_out else _need(out, "out", output_dtype, (M, Hv, dv), q, index), _DTYPES[output_dtype],
                 deltas.data_ptr() if new_deltas else _need(deltas, "deltas", torch.float32, (M, Hv, dv), q, index), flags,
                 gate_lower_bound, status, _on_stream(stream, index))
    _hand_over(stream, index, out if new_out else None, deltas if new_deltas else None)
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
    lib, flags = load_library(), _tree_flags(gate_mode, "logits", state_layout)
    found = _COMMIT[state_layout](k, deltas, raw_gate, a_log, dt_bias, cu_nodes, parents, accepted, state_pool, state_indices)
    if found is None:
        index, (M, Hk, dk), ks = _where(k, "k", 3)
        if k.dtype not in _DTYPES:
            raise ValueError("k must be float32 or bfloat16")
        (rows, Hv, dv), dls = _need_rank(deltas, "deltas", torch.float32, 3, k, index)
        if rows != M:
            raise ValueError(f"deltas has shape {tuple(deltas.shape)}, expected [{M}, Hv, dv]")
        raws = _need(raw_gate, "raw_gate", torch.float32, (M, Hv, dk), k, index)
        alogs = _need(a_log, "a_log", torch.float32, (Hv,), k, index)
        biases = _need(dt_bias, "dt_bias", torch.float32, (Hv, dk), k, index)
        B, cu, pars = _tree(cu_nodes, parents, M, k, index)
        took = _need(accepted, "accepted", torch.int32, (B,), k, index)
        pool, slots, indices = _pool(state_pool, state_indices, state_layout, k, index, B, Hv, dk, dv)
        k_type = _DTYPES[k.dtype]
    else:
        index, M, Hk, dk, Hv, dv, B, slots, ks, dls, raws, alogs, biases, cu, pars, took, pool, indices, k_type = found
    max_nodes = _most(max_nodes, M)
    status = None if device_status is None else _need(device_status, "device_status", torch.int32, (1,), k, index)
    rc = _launch(index, lib.kda_tree_commit, ks, k_type, raws, alogs, biases, dls, cu, pars, took, B, M, max_nodes, Hk, Hv,
                 dk, dv, pool, slots, indices, flags, gate_lower_bound, status, _on_stream(stream, index))
    if rc != 0:
        raise KdaError(rc, "kda_tree_commit")
