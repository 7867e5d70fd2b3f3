"""Gradients of the recurrence at head sizes whose inputs come by tensor copies while the gradients leave by plain
stores (a warp's rows do not start on 128 bytes of shared memory), and at their neighbours; also mixed with gradients
given at odd addresses."""
import pytest
import torch

import kimi_delta_attention_23_b200 as kda
import state_ops_reference as R
import test_glr_gpu as G

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16


def odd_place(shape, dtype):
    n = 1
    for s in shape:
        n *= s
    return torch.empty(n + 1, dtype=dtype, device="cuda")[1:].view(shape)


@pytest.mark.parametrize("types", [(F32, F32, F32), (BF16, BF16, BF16), (BF16, F32, BF16), (BF16, BF16, F32)])
@pytest.mark.parametrize("d", [4, 8, 12, 16, 24, 40, 72, 96, 120])
@pytest.mark.parametrize("lengths", [[3, 0, 70], [400, 61]])
@pytest.mark.parametrize("modes", [dict(input_mode="norm"), dict(gate_mode="safe", gate_lower_bound=-0.4)])
@pytest.mark.parametrize("odd", [False, True])
def test_gradients_by_plain_stores(types, d, lengths, modes, odd):
    x, raw, out_dtype = types
    H = 3
    c = G.make(lengths, H, d, x=x, raw=raw, seed=sum(lengths) + d)
    g = torch.Generator().manual_seed(7)
    dout = torch.randn(c["x"].shape, generator=g).to(out_dtype)
    dfinal = torch.randn(len(lengths), H, d, generator=g)
    _, _, kept = G.forward(c, out_dtype, checkpoints=True, **modes)
    given = dict(dx=odd_place(c["x"].shape, x), draw_gate=odd_place(c["x"].shape, raw)) if odd else {}
    got = kda.kda_glr_bwd(dout.cuda(), c["x"].cuda(), *G.params(c), c["cu"].cuda(), kept, dfinal.cuda(), **given, **modes)
    leaves = {k: c[k].double().requires_grad_() for k in ("x", "raw", "beta", "a_log", "dt_bias")}
    leaves["initial"] = c["pool"].double()[c["idx"].long()].requires_grad_()
    out, final = G.reference(c, leaves, **G.ref_modes(modes))
    loss = (out * dout.double()).sum() + (final * dfinal.double()).sum()
    ref = dict(zip(leaves, torch.autograd.grad(loss, list(leaves.values()))))
    for name, key in zip(("dx", "draw_gate", "dbeta", "d_initial"), ("x", "raw", "beta", "initial")):
        dtype = {"dx": x, "draw_gate": raw}.get(name, F32)
        assert got[name].dtype == dtype and R.rel(got[name], ref[key]) < G.tol(dtype, G.TOL_GRAD), name
    scale = float(ref["raw"].norm())  # sums over tokens that may cancel: against the size of what is summed
    for name, key in (("da_log", "a_log"), ("ddt_bias", "dt_bias")):
        err = float((got[name].double().cpu() - ref[key]).norm())
        assert err < G.TOL_GRAD * max(scale, float(ref[key].norm())), name
