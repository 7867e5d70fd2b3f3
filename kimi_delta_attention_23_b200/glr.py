"""The gated linear recurrence: prefill, gradients and the single-token step.

The diagonal-state relative of KDA (one number of state per channel instead of a dk x dv block), with
the same forget gate, the same per-head beta and the same varlen and pool conventions.  For every
sequence, head, channel and token

    g = -exp(a_log) * softplus(raw_gate + dt_bias)        (gate_mode "safe": max(g, gate_lower_bound))
    a = exp(g)
    state = a * state + beta * s * x                      s = 1, or sqrt(1 - a^2) with input_mode "norm"
    out = state

with beta = sigmoid(beta_logits), or beta_logits itself with beta_mode "probability".  Types: x float32
with raw_gate and out float32; or x bfloat16 with raw_gate and out each bfloat16 or float32.  States,
parameters, beta and the sums over tokens are float32.

Autograd does not see these calls: what kda_glr_fwd returns has no history, also where its inputs require
gradients.  Those come from kda_glr_bwd, called with the gradient of the outputs (a torch.autograd.Function
of the two makes them one operation of a model).
"""
from __future__ import annotations

import ctypes

import torch

from . import (_checker, _DTYPES, KdaError, _dev, _flags, _hand_over, _launch, _make, _need, _need_rank, _on_stream,
               _where, load_library)

__all__ = ["kda_glr_fwd", "kda_glr_bwd", "kda_glr_decode", "kda_glr_checkpoint_shape", "kda_glr_bwd_workspace_size"]

INPUT_NORM = 1 << 9  # flag bit of include/kda.h

_vp, _i32, _i64, _u32, _f32, _sz, _int = (ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_uint32,
                                          ctypes.c_float, ctypes.c_size_t, ctypes.c_int)
SIGNATURES = {
    "kda_glr_fwd": (_int, [_vp, _int, _vp, _int, _vp, _vp, _vp, _vp, _i32, _i64, _i32, _i32, _vp, _i32, _vp, _vp, _int,
                           _vp, _u32, _f32, _vp, _vp]),
    "kda_glr_decode": (_int, [_vp, _int, _vp, _int, _vp, _vp, _vp, _i32, _i32, _i32, _vp, _i32, _vp, _vp, _int, _u32,
                              _f32, _vp, _vp]),
    "kda_glr_bwd": (_int, [_vp, _int, _vp, _int, _vp, _int, _vp, _vp, _vp, _vp, _i32, _i64, _i32, _i32, _vp, _vp, _vp,
                           _vp, _vp, _vp, _vp, _vp, _u32, _f32, _vp, _sz, _vp, _vp]),
    "kda_glr_bwd_workspace_size": (_sz, [_i64, _i32, _i32, _i32]),
    "kda_glr_checkpoints": (_i64, [_i64, _i32]),
}


def kda_glr_checkpoint_shape(total_tokens, batch, num_heads, d):
    """Shape of the float32 ``checkpoints`` tensor that kda_glr_fwd fills and kda_glr_bwd reads."""
    return (int(load_library().kda_glr_checkpoints(total_tokens, batch)), num_heads, d)


def kda_glr_bwd_workspace_size(total_tokens, batch, num_heads, d) -> int:
    """Workspace bytes of kda_glr_bwd on the current device."""
    return int(load_library().kda_glr_bwd_workspace_size(total_tokens, batch, num_heads, d))


_CELLS = "x v T,H,d; raw g T,H,d; beta f T,H; a_log f H; dt_bias f H,d"
_FWD = _checker(_CELLS + "; cu i B+1; pool f S,H,d; idx i B")
_DECODE = _checker(_CELLS + "; pool f S,H,d; idx i T")
_FLAGS = {}


def _glr_flags(gate_mode, beta_mode, input_mode):
    key = (gate_mode, beta_mode, input_mode)
    if key not in _FLAGS:
        if input_mode not in ("unit", "norm"):
            raise ValueError(f"input_mode must be 'unit' or 'norm', got {input_mode!r}")
        _FLAGS[key] = _flags(gate_mode, beta_mode, "K_FIRST") | (INPUT_NORM if input_mode == "norm" else 0)
    return _FLAGS[key]


def _inputs(x, raw_gate, beta_logits, a_log, dt_bias):
    """Checks what all three calls read; returns the device's number, x's shape and the addresses."""
    index, (T, H, d), xs = _where(x, "x", 3)
    dtype, gate_dtype = x.dtype, getattr(raw_gate, "dtype", None)
    if dtype not in _DTYPES:
        raise ValueError("x must be float32 or bfloat16")
    if gate_dtype not in _DTYPES or (dtype is torch.float32 and gate_dtype is not torch.float32):
        _dev(raw_gate, "raw_gate", None, x.device)
        raise ValueError("raw_gate must be float32, or bfloat16 beside a bfloat16 x")
    return index, T, H, d, (xs, _DTYPES[dtype], _need(raw_gate, "raw_gate", gate_dtype, (T, H, d), x, index),
                            _DTYPES[gate_dtype], _need(beta_logits, "beta_logits", torch.float32, (T, H), x, index),
                            _need(a_log, "a_log", torch.float32, (H,), x, index),
                            _need(dt_bias, "dt_bias", torch.float32, (H, d), x, index))


def _offsets(cu_seqlens, like, index):
    (count,), at = _need_rank(cu_seqlens, "cu_seqlens", torch.int32, 1, like, index)
    if count < 1:
        raise ValueError("cu_seqlens must hold B + 1 offsets")
    return count - 1, at


def _pool(state_pool, state_indices, like, index, B, H, d):
    shape, at = _need_rank(state_pool, "state_pool", torch.float32, 3, like, index)
    if shape[1] != H or shape[2] != d:
        raise ValueError(f"state_pool has shape {tuple(shape)}, expected [slots, {H}, {d}]")
    return at, shape[0], _need(state_indices, "state_indices", torch.int32, (B,), like, index)


def _output(out, output_dtype, x, index, stream):
    """The output (made here if ``out`` is None), its address and type."""
    if output_dtype is None:
        output_dtype = x.dtype if out is None else out.dtype
    if output_dtype not in _DTYPES or (x.dtype is torch.float32 and output_dtype is not torch.float32):
        raise ValueError("output_dtype must be float32, or bfloat16 beside a bfloat16 x")
    if out is None:
        out = _make(stream, index, torch.empty_like, x, dtype=output_dtype)
        return out, out.data_ptr(), _DTYPES[output_dtype]
    return out, _need(out, "out", output_dtype, x.shape, x, index), _DTYPES[output_dtype]


def _status(device_status, like, index):
    return None if device_status is None else _need(device_status, "device_status", torch.int32, (1,), like, index)


def kda_glr_fwd(x, raw_gate, beta_logits, a_log, dt_bias, cu_seqlens, state_pool, state_indices, out=None, *,
                output_dtype=None, checkpoints=None, gate_mode="original", beta_mode="logits", input_mode="unit",
                gate_lower_bound=-5.0, device_status=None, stream=None):
    """The recurrence over a varlen batch, states read from and written to their pool slots.

    Shapes: x, raw_gate [T,H,d]; beta_logits [T,H] f32; a_log [H] f32; dt_bias [H,d] f32; cu_seqlens
    [B+1] i32; state_pool [slots,H,d] f32, mutated in place; state_indices [B] i32.  Returns out
    [T,H,d] in ``output_dtype`` (default: the dtype of x); rows outside every sequence are not written.
    ``checkpoints`` (f32, kda_glr_checkpoint_shape(T, B, H, d)) keeps what kda_glr_bwd needs.
    """
    lib, flags = load_library(), _glr_flags(gate_mode, beta_mode, input_mode)
    found = _FWD(x, raw_gate, beta_logits, a_log, dt_bias, cu_seqlens, state_pool, state_indices)
    if found is None:
        index, T, H, d, (xs, x_type, raws, gate_type, betas, a_logs, biases) = _inputs(x, raw_gate, beta_logits, a_log, dt_bias)
        B, cu = _offsets(cu_seqlens, x, index)
        pool, slots, indices = _pool(state_pool, state_indices, x, index, B, H, d)
    else:
        index, T, H, d, B, slots, xs, raws, betas, a_logs, biases, cu, pool, indices, x_type, gate_type = found
    kept = None
    if checkpoints is not None:
        kept = _need(checkpoints, "checkpoints", torch.float32, (lib.kda_glr_checkpoints(T, B), H, d), x, index)
    status, given = _status(device_status, x, index), out
    out, to, out_type = _output(out, output_dtype, x, index, stream)
    rc = _launch(index, lib.kda_glr_fwd, xs, x_type, raws, gate_type, betas, a_logs, biases, cu, B, T, H, d, pool, slots,
                 indices, to, out_type, kept, flags, gate_lower_bound, status, _on_stream(stream, index))
    if given is None:
        _hand_over(stream, index, out)
    if rc != 0:
        raise KdaError(rc, "kda_glr_fwd")
    return out


def kda_glr_decode(x, raw_gate, beta_logits, a_log, dt_bias, state_pool, state_indices, out=None, *, output_dtype=None,
                   gate_mode="original", beta_mode="logits", input_mode="unit", gate_lower_bound=-5.0,
                   device_status=None, stream=None):
    """One token of each sequence: x, raw_gate [B,H,d]; beta_logits [B,H]; the rest as kda_glr_fwd."""
    lib, flags = load_library(), _glr_flags(gate_mode, beta_mode, input_mode)
    found = _DECODE(x, raw_gate, beta_logits, a_log, dt_bias, state_pool, state_indices)
    if found is None:
        index, B, H, d, (xs, x_type, raws, gate_type, betas, a_logs, biases) = _inputs(x, raw_gate, beta_logits, a_log, dt_bias)
        pool, slots, indices = _pool(state_pool, state_indices, x, index, B, H, d)
    else:
        index, B, H, d, slots, xs, raws, betas, a_logs, biases, pool, indices, x_type, gate_type = found
    status, given = _status(device_status, x, index), out
    out, to, out_type = _output(out, output_dtype, x, index, stream)
    rc = _launch(index, lib.kda_glr_decode, xs, x_type, raws, gate_type, betas, a_logs, biases, B, H, d, pool, slots, indices,
                 to, out_type, flags, gate_lower_bound, status, _on_stream(stream, index))
    if given is None:
        _hand_over(stream, index, out)
    if rc != 0:
        raise KdaError(rc, "kda_glr_decode")
    return out


def kda_glr_bwd(dout, x, raw_gate, beta_logits, a_log, dt_bias, cu_seqlens, checkpoints, d_final=None, *, dx=None,
                draw_gate=None, dbeta=None, da_log=None, ddt_bias=None, d_initial=None, gate_mode="original",
                beta_mode="logits", input_mode="unit", gate_lower_bound=-5.0, workspace=None, device_status=None,
                stream=None):
    """Gradients of kda_glr_fwd for the same inputs, modes and bound.

    ``dout`` [T,H,d] in the forward pass's output dtype; ``checkpoints`` as kda_glr_fwd filled them;
    ``d_final`` [B,H,d] f32 (None: zero) the gradient of each sequence's final state.  Returns
    dict(dx, draw_gate, dbeta, da_log, ddt_bias, d_initial): in the shapes and dtypes of x, raw_gate,
    beta_logits, a_log and dt_bias, and [B,H,d] f32 for the states the sequences started from.
    Tensors to fill can be given; rows outside every sequence are left as they are in those, and
    unwritten in new ones.  ``workspace``: uint8 CUDA tensor of kda_glr_bwd_workspace_size bytes,
    allocated when not given.
    """
    lib = load_library()
    index, T, H, d, inputs = _inputs(x, raw_gate, beta_logits, a_log, dt_bias)
    dtype = getattr(dout, "dtype", None)
    if dtype not in _DTYPES or (x.dtype == torch.float32 and dtype != torch.float32):
        _dev(dout, "dout", None, x.device)
        raise ValueError("dout must be float32, or bfloat16 beside a bfloat16 x")
    douts = _need(dout, "dout", dtype, (T, H, d), x, index)
    B, cu = _offsets(cu_seqlens, x, index)
    kept = _need(checkpoints, "checkpoints", torch.float32, (lib.kda_glr_checkpoints(T, B), H, d), x, index)
    final = None if d_final is None else _need(d_final, "d_final", torch.float32, (B, H, d), x, index)
    flags, status = _glr_flags(gate_mode, beta_mode, input_mode), _status(device_status, x, index)
    made = []

    def grad(t, name, shape, dtype=torch.float32):
        if t is None:
            t = _make(stream, index, torch.empty, shape, dtype=dtype, device=x.device)
            made.append(t)
            return t, t.data_ptr()
        return t, _need(t, name, dtype, shape, x, index)

    dx, dxs = grad(dx, "dx", (T, H, d), x.dtype)
    draw_gate, draws = grad(draw_gate, "draw_gate", (T, H, d), raw_gate.dtype)
    dbeta, dbetas = grad(dbeta, "dbeta", (T, H))
    da_log, das = grad(da_log, "da_log", (H,))
    ddt_bias, dbs = grad(ddt_bias, "ddt_bias", (H, d))
    d_initial, dis = grad(d_initial, "d_initial", (B, H, d))
    if workspace is None:
        need = _launch(index, lib.kda_glr_bwd_workspace_size, T, B, H, d)
        workspace = _make(stream, index, torch.empty, need, dtype=torch.uint8, device=x.device)
    _dev(workspace, "workspace", torch.uint8, x.device)
    rc = _launch(index, lib.kda_glr_bwd, douts, _DTYPES[dtype], *inputs, cu, B, T, H, d, kept, final, dxs, draws, dbetas, das,
                 dbs, dis, flags, gate_lower_bound, workspace.data_ptr(), workspace.numel(), status,
                 _on_stream(stream, index))
    _hand_over(stream, index, *made)
    if rc != 0:
        raise KdaError(rc, "kda_glr_bwd")
    return {"dx": dx, "draw_gate": draw_gate, "dbeta": dbeta, "da_log": da_log, "ddt_bias": ddt_bias,
            "d_initial": d_initial}
