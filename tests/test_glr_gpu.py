"""The gated linear recurrence on the GPU against its 64-bit definition, gradients included.

Tolerances (relative L2).  A step's decay is off by at most 2^-21 of itself (2^-22 of the hardware
exponential, as much again from its argument), and the state remembers about 1 / |g| tokens.  The
tests' gates are drawn so that nearly all |g| > 0.02: errors that all fell on one side would come to
50 * 2^-21 = 2.4e-5, so fp32 results are held to 5e-5 (gradients pass two such scans: 1e-4).  A bf16
result may be half a step further off: 2^-8.
"""
import pytest
import torch

import kimi_delta_attention_23_b200 as kda
import state_ops_reference as R

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
TOL, TOL_GRAD, HALF_STEP = 5e-5, 1e-4, 2.0 ** -8


def tol(dtype, base):
    return base + (HALF_STEP if dtype == BF16 else 0.0)


def make(lengths, H, d, *, x=F32, raw=F32, seed=0, slots=None, shift=-1.5):
    g = torch.Generator().manual_seed(seed)
    T, B = sum(lengths), len(lengths)
    n = lambda *s, m=0.0: torch.randn(*s, generator=g) + m  # noqa: E731
    slots = slots or B + 2
    c = dict(x=n(T, H, d).to(x), raw=n(T, H, d).to(raw), beta=n(T, H), a_log=torch.rand(H, generator=g) * 2.0,
             dt_bias=n(H, d) * 0.5 + shift, pool=n(slots, H, d))
    c["cu"] = torch.tensor([0] + lengths, dtype=torch.int32).cumsum(0).to(torch.int32)
    c["idx"] = torch.randperm(slots, generator=g)[:B].to(torch.int32)
    c["lengths"] = lengths
    return c


def params(c):
    return [c[k].cuda() for k in ("raw", "beta", "a_log", "dt_bias")]


def reference(c, leaves=None, **modes):
    l64 = leaves or {k: c[k].double() for k in ("x", "raw", "beta", "a_log", "dt_bias")}
    init = leaves["initial"] if leaves else c["pool"].double()[c["idx"].long()]
    return R.glr(l64["x"], l64["raw"], l64["beta"], l64["a_log"], l64["dt_bias"], c["lengths"], init, **modes)


def forward(c, out_dtype, checkpoints=False, **modes):
    T, H, d = c["x"].shape
    pool, status = c["pool"].cuda(), torch.zeros(1, dtype=torch.int32, device="cuda")
    kept = torch.full(kda.kda_glr_checkpoint_shape(T, len(c["lengths"]), H, d), float("nan"), device="cuda") if checkpoints else None
    out = kda.kda_glr_fwd(c["x"].cuda(), *params(c), c["cu"].cuda(), pool, c["idx"].cuda(), output_dtype=out_dtype,
                          checkpoints=kept, device_status=status, **modes)
    assert int(status) == 0
    return out, pool, kept


MODES = [dict(), dict(input_mode="norm"), dict(gate_mode="safe", gate_lower_bound=-0.4, beta_mode="probability"),
         dict(gate_mode="safe", gate_lower_bound=-0.4, input_mode="norm")]


def ref_modes(m):
    return {("lower" if k == "gate_lower_bound" else k): v for k, v in m.items()}


@pytest.mark.parametrize("types", [(F32, F32, F32), (BF16, BF16, BF16), (BF16, F32, BF16), (BF16, BF16, F32)])
@pytest.mark.parametrize("lengths,H,d", [
    ([1], 1, 1), ([3, 0, 5], 2, 7), ([64], 1, 128), ([65, 63, 64, 1], 3, 128), ([200, 0, 0, 333], 2, 37),
    ([130], 2, 64), ([129, 70], 1, 34), ([1500], 1, 128), ([700], 4, 127),
])
@pytest.mark.parametrize("modes", MODES)
def test_forward(types, lengths, H, d, modes):
    x, raw, out_dtype = types
    c = make(lengths, H, d, x=x, raw=raw, seed=sum(lengths) + d)
    out, pool, _ = forward(c, out_dtype, **modes)
    ref, final = reference(c, **ref_modes(modes))
    assert out.dtype == out_dtype and R.rel(out, ref) < tol(out_dtype, TOL)
    expect = c["pool"].double()
    expect[c["idx"].long()] = final
    assert R.rel(pool, expect) < TOL
    untouched = [s for s in range(pool.shape[0]) if s not in c["idx"].tolist()]
    assert torch.equal(pool.cpu()[untouched], c["pool"][untouched])
    empty = [int(s) for s, n in zip(c["idx"], lengths) if n == 0]
    assert torch.equal(pool.cpu()[empty], c["pool"][empty])


@pytest.mark.parametrize("types", [(F32, F32, F32), (BF16, BF16, BF16), (BF16, F32, BF16), (BF16, F32, F32),
                                   (BF16, BF16, F32)])
@pytest.mark.parametrize("lengths,H,d", [
    ([1], 1, 1), ([3, 0, 5], 2, 7), ([64], 1, 128), ([65, 63, 1], 2, 128), ([200, 0, 133], 2, 37), ([130], 2, 64),
    ([1100], 1, 128),
])
@pytest.mark.parametrize("modes", MODES)
@pytest.mark.parametrize("with_final", [True, False])
def test_gradients(types, lengths, H, d, modes, with_final):
    x, raw, out_dtype = types
    c = make(lengths, H, d, x=x, raw=raw, seed=sum(lengths) + d + 1)
    g = torch.Generator().manual_seed(5)
    dout = torch.randn(c["x"].shape, generator=g).to(out_dtype)
    dfinal = torch.randn(len(lengths), H, d, generator=g) if with_final else None
    _, _, kept = forward(c, out_dtype, checkpoints=True, **modes)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = kda.kda_glr_bwd(dout.cuda(), c["x"].cuda(), *params(c), c["cu"].cuda(), kept,
                          None if dfinal is None else dfinal.cuda(), device_status=status, **modes)
    assert int(status) == 0
    leaves = {k: c[k].double().requires_grad_() for k in ("x", "raw", "beta", "a_log", "dt_bias")}
    leaves["initial"] = c["pool"].double()[c["idx"].long()].requires_grad_()
    out, final = reference(c, leaves, **ref_modes(modes))
    loss = (out * dout.double()).sum() + (0 if dfinal is None else (final * dfinal.double()).sum())
    ref = torch.autograd.grad(loss, list(leaves.values()), allow_unused=True)
    for name, key, want in zip(("dx", "draw_gate", "dbeta", "da_log", "ddt_bias", "d_initial"), leaves, ref):
        want = torch.zeros_like(leaves[key]) if want is None else want
        dtype = {"dx": x, "draw_gate": raw}.get(name, F32)
        assert got[name].dtype == dtype
        if name in ("da_log", "ddt_bias"):
            # sums over tokens that may cancel: measured against the size of what is summed
            scale = float(ref[1].norm()) + 1e-30
            err = float((got[name].double().cpu() - want).norm()) / max(scale, float(want.norm()))
        else:
            err = R.rel(got[name], want)
        assert err < tol(dtype, TOL_GRAD), name


def test_gradients_against_differences():
    lengths, H, d = [90, 41], 2, 24
    modes = dict(input_mode="norm")
    c = make(lengths, H, d, seed=9)
    g = torch.Generator().manual_seed(6)
    dout, dfinal = torch.randn(c["x"].shape, generator=g), torch.randn(2, H, d, generator=g)
    _, _, kept = forward(c, F32, checkpoints=True, **modes)
    got = kda.kda_glr_bwd(dout.cuda(), c["x"].cuda(), *params(c), c["cu"].cuda(), kept, dfinal.cuda(), **modes)
    leaves = {k: c[k].double() for k in ("x", "raw", "beta", "a_log", "dt_bias")}
    leaves["initial"] = c["pool"].double()[c["idx"].long()]

    def loss(at):
        out, final = reference(c, at, **modes)
        return float((out * dout.double()).sum() + (final * dfinal.double()).sum())

    for key, name in zip(leaves, ("dx", "draw_gate", "dbeta", "da_log", "ddt_bias", "d_initial")):
        way = torch.randn(leaves[key].shape, generator=g, dtype=torch.float64)
        step = 1e-5
        up, down = ({**leaves, key: leaves[key] + s * way} for s in (step, -step))
        slope = (loss(up) - loss(down)) / (2 * step)
        grad = got[name].double().cpu()
        # the difference is off by step^2 terms and rounding (about 1e-8 of the loss's terms); the
        # gradient by TOL_GRAD of its norm, along the way's
        assert abs(float((grad * way).sum()) - slope) < 1e-6 * abs(slope) + TOL_GRAD * float(grad.norm() * way.norm()), name


@pytest.mark.parametrize("types", [(F32, F32, F32), (BF16, BF16, BF16), (BF16, F32, F32)])
@pytest.mark.parametrize("B,H,d", [(1, 1, 1), (5, 3, 37), (9, 2, 128)])
@pytest.mark.parametrize("modes", MODES)
def test_decode_equals_one_token_prefill(types, B, H, d, modes):
    x, raw, out_dtype = types
    c = make([1] * B, H, d, x=x, raw=raw, seed=B)
    out, pool, _ = forward(c, out_dtype, **modes)
    pool2 = c["pool"].cuda()
    out2 = kda.kda_glr_decode(c["x"].cuda(), *params(c), pool2, c["idx"].cuda(), output_dtype=out_dtype, **modes)
    ref, _ = reference(c, **ref_modes(modes))
    assert R.rel(out2, ref) < tol(out_dtype, TOL)
    assert R.rel(pool2, pool) < 2 * TOL and R.rel(out2, out) < 2 * tol(out_dtype, TOL)


def test_prefill_then_decode_continues_the_sequence():
    c = make([75, 20], 2, 128, seed=3)
    out, pool, _ = forward(c, F32)
    split = {**c, "lengths": [74, 19]}
    rows = [t for t in range(95) if t not in (74, 94)]
    for k in ("x", "raw", "beta"):
        split[k] = c[k][rows]
    split["cu"] = torch.tensor([0, 74, 93], dtype=torch.int32)
    _, pool2, _ = forward(split, F32)
    last = kda.kda_glr_decode(c["x"][[74, 94]].cuda(), c["raw"][[74, 94]].cuda(), c["beta"][[74, 94]].cuda(),
                              c["a_log"].cuda(), c["dt_bias"].cuda(), pool2, c["idx"].cuda())
    assert R.rel(last, out[[74, 94]]) < 2 * TOL and R.rel(pool2, pool) < 2 * TOL


def test_extreme_gates_stay_finite():
    # shut, wide open and saturated gates; with +-inf the state is dropped or kept whole
    c = make([70], 1, 8, seed=4)
    c["raw"][:, 0, 0] = float("inf")    # a = 0: only the token's own input
    c["raw"][:, 0, 1] = float("-inf")   # a = 1
    c["raw"][:, 0, 2] = 200.0
    c["raw"][:, 0, 3] = -200.0
    for modes in (dict(), dict(input_mode="norm")):
        out, pool, kept = forward(c, F32, checkpoints=True, **modes)
        ref, _ = reference(c, **modes)
        assert R.rel(out, ref) < TOL
        grads = kda.kda_glr_bwd(torch.ones_like(out), c["x"].cuda(), *params(c), c["cu"].cuda(), kept, **modes)
        assert all(bool(torch.isfinite(t).all()) for t in grads.values())
        assert float(grads["draw_gate"][:, 0, :2].abs().max()) == 0.0


def test_results_do_not_depend_on_timing():
    c = make([3000, 500], 2, 128, x=BF16, raw=BF16, seed=8)
    first = forward(c, BF16, checkpoints=True)
    dout = torch.randn(c["x"].shape, generator=torch.Generator().manual_seed(1)).to(BF16).cuda()
    bwd = lambda kept: kda.kda_glr_bwd(dout, c["x"].cuda(), *params(c), c["cu"].cuda(), kept)  # noqa: E731
    grads = bwd(first[2])
    for _ in range(3):
        again = forward(c, BF16, checkpoints=True)
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])
        more = bwd(again[2])
        assert all(torch.equal(grads[k], more[k]) for k in grads)


def test_rows_behind_the_last_sequence_stay():
    c = make([40, 30], 2, 16, seed=11)
    extra = 9
    for k in ("x", "raw", "beta"):
        c[k] = torch.cat([c[k], torch.full((extra, *c[k].shape[1:]), float("nan"), dtype=c[k].dtype)])
    out = torch.full(c["x"].shape, 7.0, device="cuda")
    pool = c["pool"].cuda()
    kept = torch.zeros(kda.kda_glr_checkpoint_shape(79, 2, 2, 16), device="cuda")
    kda.kda_glr_fwd(c["x"].cuda(), *params(c), c["cu"].cuda(), pool, c["idx"].cuda(), out=out, checkpoints=kept)
    assert bool((out[70:] == 7.0).all()) and bool(torch.isfinite(out).all())
    given = {k: torch.full(s, 3.0, device="cuda") for k, s in
             (("dx", (79, 2, 16)), ("draw_gate", (79, 2, 16)), ("dbeta", (79, 2)))}
    dout = torch.full((79, 2, 16), float("nan"), device="cuda")
    dout[:70] = 1.0
    res = kda.kda_glr_bwd(dout, c["x"].cuda(), *params(c), c["cu"].cuda(), kept, **given)
    assert all(bool((t[70:] == 3.0).all()) for t in given.values())
    assert all(bool(torch.isfinite(t).all()) for t in res.values())


def test_unaligned_views():
    # contiguous slices that start in the middle of a wide access
    for dtype in (F32, BF16):
        c = make([50, 33], 1, 12, x=dtype, raw=dtype, seed=12)
        shifted = {}
        for k in ("x", "raw"):
            flat = torch.empty(c[k].numel() + 1, dtype=dtype, device="cuda")
            flat[1:] = c[k].cuda().flatten()
            shifted[k] = flat[1:].view(c[k].shape)
        out, pool, _ = forward(c, F32)
        pool2 = c["pool"].cuda()
        flat = torch.empty(out.numel() + 1, device="cuda")
        out2 = kda.kda_glr_fwd(shifted["x"], shifted["raw"], *params(c)[1:], c["cu"].cuda(), pool2, c["idx"].cuda(),
                               out=flat[1:].view(out.shape))
        assert torch.equal(out, out2) and torch.equal(pool, pool2)


@pytest.mark.parametrize("what", ["slot", "decreasing", "past the end"])
def test_bad_sequences_are_reported_and_skipped(what):
    c = make([20, 30, 10], 2, 16, seed=13)
    if what == "slot":
        c["idx"][1] = c["pool"].shape[0]
    elif what == "decreasing":
        c["cu"] = torch.tensor([0, 20, 10, 60], dtype=torch.int32)
    else:
        c["cu"] = torch.tensor([0, 20, 50, 61], dtype=torch.int32)
    bad = 2 if what == "past the end" else 1
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    pool, out = c["pool"].cuda(), torch.full(c["x"].shape, 9.0, device="cuda")
    kda.kda_glr_fwd(c["x"].cuda(), *params(c), c["cu"].cuda(), pool, c["idx"].cuda(), out=out, device_status=status)
    assert int(status) == kda.ERR_DEVICE_CHECK
    if what != "slot":
        slot = int(c["idx"][bad])
        assert torch.equal(pool[slot].cpu(), c["pool"][slot])
    ref, final = R.glr(*(c[k][:20].double() for k in ("x", "raw", "beta")), c["a_log"].double(), c["dt_bias"].double(),
                       [20], c["pool"].double()[c["idx"][:1].long()])
    own = 10 if what == "decreasing" else 20  # the third sequence then starts at token 10, over the first one's rows
    assert R.rel(out[:own], ref[:own]) < TOL and R.rel(pool[int(c["idx"][0])], final[0]) < TOL


def test_other_stream_and_graph():
    c = make([100, 77], 2, 128, x=BF16, raw=BF16, seed=14)
    out, pool, kept = forward(c, BF16, checkpoints=True)
    dout = torch.ones_like(out)
    grads = kda.kda_glr_bwd(dout, c["x"].cuda(), *params(c), c["cu"].cuda(), kept)
    x, ps, cu, idx = c["x"].cuda(), params(c), c["cu"].cuda(), c["idx"].cuda()
    side = torch.cuda.Stream()
    pool2, kept2 = c["pool"].cuda(), torch.zeros_like(kept)
    torch.cuda.synchronize()
    out2 = kda.kda_glr_fwd(x, *ps, cu, pool2, idx, checkpoints=kept2, stream=side)
    grads2 = kda.kda_glr_bwd(dout, x, *ps, cu, kept2, stream=side)
    side.synchronize()
    assert torch.equal(out, out2) and torch.equal(pool, pool2) and all(torch.equal(grads[k], grads2[k]) for k in grads)
    # captured, and replayed on other values in the same places
    pool3 = c["pool"].cuda()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out3 = kda.kda_glr_fwd(x, *ps, cu, pool3, idx, checkpoints=kept2)
        grads3 = kda.kda_glr_bwd(dout, x, *ps, cu, kept2)
        step3 = kda.kda_glr_decode(x[:2], ps[0][:2], ps[1][:2], ps[2], ps[3], pool3, idx)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, out3) and all(torch.equal(grads[k], grads3[k]) for k in grads)
    x.copy_(-x)
    pool3.copy_(c["pool"].cuda())
    pool4 = c["pool"].cuda()
    want = kda.kda_glr_fwd(x, *ps, cu, pool4, idx)
    want_step = kda.kda_glr_decode(x[:2], ps[0][:2], ps[1][:2], ps[2], ps[3], pool4, idx)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(want, out3) and torch.equal(want_step, step3) and torch.equal(pool3, pool4)
