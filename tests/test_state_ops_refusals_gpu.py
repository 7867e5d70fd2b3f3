"""What the binding refuses on a GPU: wrong types, shapes and strides of every tensor, one at a time.
Nothing is launched; a call with all of them right runs."""
import pytest
import torch

import kimi_delta_attention_23_b200 as kda

pytestmark = pytest.mark.gpu

F32, BF16, I32 = torch.float32, torch.bfloat16, torch.int32


def f(*shape, dtype=F32):
    return torch.zeros(*shape, dtype=dtype, device="cuda")


def glr(B=2, T=5, H=2, d=8):
    return dict(x=f(T, H, d, dtype=BF16), raw_gate=f(T, H, d), beta_logits=f(T, H), a_log=f(H), dt_bias=f(H, d),
                cu_seqlens=torch.tensor([0, 2, 5], dtype=I32, device="cuda"), state_pool=f(3, H, d),
                state_indices=torch.tensor([0, 2], dtype=I32, device="cuda"))


def tree(M=5, Hk=1, Hv=2, dk=8, dv=4):
    return dict(q=f(M, Hk, dk), k=f(M, Hk, dk), v=f(M, Hv, dv), raw_gate=f(M, Hv, dk), beta_logits=f(M, Hv), a_log=f(Hv),
                dt_bias=f(Hv, dk), cu_nodes=torch.tensor([0, 2, 5], dtype=I32, device="cuda"),
                parents=torch.tensor([-1, 0, -1, 0, 0], dtype=I32, device="cuda"), state_pool=f(3, Hv, dk, dv),
                state_indices=torch.tensor([0, 2], dtype=I32, device="cuda"))


def calls():
    g = glr()
    yield kda.kda_glr_fwd, g
    one = {k: v for k, v in glr(T=2).items() if k != "cu_seqlens"}
    yield kda.kda_glr_decode, one
    kept = f(*kda.kda_glr_checkpoint_shape(5, 2, 2, 8))
    back = {k: v for k, v in g.items() if not k.startswith("state")}
    yield kda.kda_glr_bwd, dict(dout=f(5, 2, 8, dtype=BF16), **back, checkpoints=kept, d_final=f(2, 2, 8))
    t = tree()
    yield kda.kda_tree_decode, t
    yield kda.kda_tree_commit, dict(k=t["k"], raw_gate=t["raw_gate"], a_log=t["a_log"], dt_bias=t["dt_bias"], deltas=f(5, 2, 4),
                                    cu_nodes=t["cu_nodes"], parents=t["parents"],
                                    accepted=torch.tensor([-1, 2], dtype=I32, device="cuda"), state_pool=t["state_pool"],
                                    state_indices=t["state_indices"])
    ints = lambda *v: torch.tensor(v, dtype=I32, device="cuda")  # noqa: E731
    yield kda.kda_pool_copy, dict(state_pool=f(4, 3), src=ints(0, 1), dst=ints(2, 3))
    yield kda.kda_pool_fork, dict(state_pool=f(4, 3), live=ints(1, 1, 0, 0), src=ints(0, 1))
    yield kda.kda_pool_free, dict(state_pool=f(4, 3), live=ints(1, 1, 0, 0), slots=ints(0, 1))
    yield kda.kda_pool_compact, dict(state_pool=f(4, 3), live=ints(1, 0, 1, 0), state_indices=ints(0, 2))


def test_every_tensor_is_checked():
    for call, args in calls():
        call(**args)
        for name, t in args.items():
            wrong = {
                "type": t.to(torch.float64 if t.is_floating_point() else torch.int64),
                "rank": t[None],
                "device": t.cpu(),
            }
            if t.numel() > 1 and t.shape[-1] > 1:
                wrong["strides"] = torch.zeros(*t.shape[:-1], 2 * t.shape[-1], dtype=t.dtype, device="cuda")[..., ::2]
            for what, bad in wrong.items():
                if what == "rank" and name == "state_pool" and call.__name__.startswith("kda_pool"):
                    continue  # a pool may have any number of dimensions
                with pytest.raises((ValueError, TypeError)):
                    call(**{**args, name: bad})
            with pytest.raises((TypeError, ValueError)):
                call(**{**args, name: 3})
        torch.cuda.synchronize()


@pytest.mark.parametrize("name,bad", [
    ("raw_gate", (5, 2, 7)), ("beta_logits", (5, 3)), ("a_log", (3,)), ("dt_bias", (2, 9)), ("state_pool", (3, 2, 9)),
    ("state_pool", (3, 3, 8)), ("raw_gate", (6, 2, 8)),
])
def test_extents_have_to_agree_glr(name, bad):
    with pytest.raises(ValueError):
        kda.kda_glr_fwd(**{**glr(), name: f(*bad)})


@pytest.mark.parametrize("name,bad", [
    ("k", (5, 2, 8)), ("v", (4, 2, 4)), ("raw_gate", (5, 2, 4)), ("beta_logits", (5, 1)), ("a_log", (1,)), ("dt_bias", (2, 4)),
    ("state_pool", (3, 2, 4, 8)), ("state_pool", (3, 1, 8, 4)),
])
def test_extents_have_to_agree_tree(name, bad):
    with pytest.raises(ValueError):
        kda.kda_tree_decode(**{**tree(), name: f(*bad)})


def test_options():
    g, t = glr(), tree()
    for kw in (dict(input_mode="x"), dict(gate_mode="x"), dict(beta_mode="x")):
        with pytest.raises(ValueError):
            kda.kda_glr_fwd(**g, **kw)
    with pytest.raises(ValueError):
        kda.kda_glr_fwd(**g, output_dtype=torch.float16)
    with pytest.raises(ValueError):
        kda.kda_glr_fwd(**{**g, "x": g["x"].float(), "raw_gate": g["raw_gate"].to(BF16)})
    for kw in (dict(max_nodes=0), dict(max_nodes=65), dict(state_layout="x"), dict(gate_mode="x"), dict(output_dtype=torch.float16)):
        with pytest.raises(ValueError):
            kda.kda_tree_decode(**t, **kw)
    with pytest.raises(kda.KdaError):  # fp32 inputs need an fp32 output
        kda.kda_tree_decode(**t, output_dtype=BF16)
    with pytest.raises(ValueError):
        n = kda.MAX_POOL_COPIES + 1
        kda.kda_pool_copy(f(4, 3), torch.zeros(n, dtype=I32, device="cuda"), torch.zeros(n, dtype=I32, device="cuda"))
    # Hv not a multiple of Hk
    bad = {**t, "q": f(5, 3, 8), "k": f(5, 3, 8)}
    with pytest.raises(kda.KdaError):
        kda.kda_tree_decode(**bad)
