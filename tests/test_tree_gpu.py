"""Drafted trees on the GPU against the 64-bit token-by-token definition, and the commit against it.

Tolerances (relative L2).  The products with the state drop 2^-18 of each split factor and the
fourth partial product (2^-18 too): at most 3 * 2^-18 = 1.2e-5 of the terms' sizes, and the solve
carries them down the tree with weights |A_ij| <= 1; the terms cancel to no less than about a third
of their size in these draws.  So fp32 results are held to 4e-5, a bf16 output to half a step (2^-8)
more.  The commit is plain fp32: 64 products along a path, 64 * 2^-23 = 8e-6 of the terms' sizes.
"""
import pytest
import torch

import kimi_delta_attention_23_b200 as kda
import state_ops_reference as R

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
TOL, TOL_COMMIT, HALF_STEP = 4e-5, 8e-6, 2.0 ** -8


def make(counts, Hk, Hv, dk, dv, *, dtype=F32, shape="tree", layout="K_FIRST", seed=0, shift=0.0):
    g = torch.Generator().manual_seed(seed)
    M, B = sum(counts), len(counts)
    n = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    unit = lambda t: t / t.norm(dim=-1, keepdim=True).clamp_min(1e-6)  # noqa: E731
    c = dict(q=unit(n(M, Hk, dk)).to(dtype), k=unit(n(M, Hk, dk)).to(dtype), v=n(M, Hv, dv).to(dtype), raw=n(M, Hv, dk),
             beta=n(M, Hv), a_log=torch.rand(Hv, generator=g) * 2.0, dt_bias=n(Hv, dk) * 0.3 + shift)
    at = [i for k in counts for i in range(k)]
    if shape == "chain":
        par = [i - 1 for i in at]
    elif shape == "star":
        par = [-1 for _ in at]
    else:
        par = [int(torch.randint(-1, i, (1,), generator=g)) if i else -1 for i in at]
    c["parents"] = torch.tensor(par, dtype=torch.int32)
    c["cu"] = torch.tensor([0] + list(counts), dtype=torch.int32).cumsum(0).to(torch.int32)
    slots = B + 2
    c["idx"] = torch.randperm(slots, generator=g)[:B].to(torch.int32)
    S = n(slots, Hv, dk, dv) * 0.3
    c["pool"] = S if layout == "K_FIRST" else S.transpose(2, 3).contiguous()
    c["states"] = S[c["idx"].long()].double()
    c["counts"], c["layout"] = counts, layout
    return c


def gpu(c, *names):
    return [c[k].cuda() for k in names]


def decode(c, out_dtype=F32, max_nodes=None, status=None, pool=None, **modes):
    st = torch.zeros(1, dtype=torch.int32, device="cuda") if status is None else status
    pool = c["pool"].cuda() if pool is None else pool
    before = pool.clone()
    out, deltas = kda.kda_tree_decode(*gpu(c, "q", "k", "v", "raw", "beta", "a_log", "dt_bias", "cu", "parents"), pool,
                                      c["idx"].cuda(), max_nodes=max_nodes or max(1, max(c["counts"])),
                                      output_dtype=out_dtype, state_layout=c["layout"], device_status=st, **modes)
    assert torch.equal(pool, before)
    if status is None:
        assert int(st) == 0
    return out, deltas


def commit(c, deltas, accepted, pool=None, status=None, max_nodes=None, **modes):
    st = torch.zeros(1, dtype=torch.int32, device="cuda") if status is None else status
    pool = c["pool"].cuda() if pool is None else pool
    kda.kda_tree_commit(*gpu(c, "k", "raw", "a_log", "dt_bias"), deltas, *gpu(c, "cu", "parents"),
                        torch.tensor(accepted, dtype=torch.int32, device="cuda"), pool, c["idx"].cuda(),
                        max_nodes=max_nodes or max(1, max(c["counts"])), state_layout=c["layout"], device_status=st, **modes)
    if status is None:
        assert int(st) == 0
    return pool


def reference(c, **modes):
    m = {("lower" if k == "gate_lower_bound" else k): v for k, v in modes.items()}
    args = [c[k].double() for k in ("q", "k", "v", "raw", "beta", "a_log", "dt_bias")]
    return R.tree(*args, c["counts"], c["parents"], c["states"], **m)


MODES = [dict(), dict(gate_mode="safe", gate_lower_bound=-0.5, beta_mode="probability")]


@pytest.mark.parametrize("layout", ["K_FIRST", "V_FIRST"])
@pytest.mark.parametrize("counts,Hk,Hv,dk,dv,dtype,shape", [
    ([1], 1, 1, 128, 128, F32, "tree"), ([8], 2, 2, 128, 128, BF16, "tree"), ([9, 0, 3], 1, 2, 128, 128, BF16, "tree"),
    ([16, 5], 1, 1, 128, 128, F32, "chain"), ([17], 2, 4, 128, 128, BF16, "tree"), ([64], 1, 1, 128, 128, F32, "chain"),
    ([64, 1, 33], 1, 2, 128, 128, BF16, "tree"), ([40], 1, 1, 128, 128, F32, "star"), ([5, 7], 1, 1, 1, 1, F32, "tree"),
    ([12], 2, 2, 37, 91, F32, "tree"), ([30, 2], 1, 3, 64, 16, BF16, "tree"), ([64], 1, 1, 33, 128, F32, "chain"),
    ([10], 1, 1, 128, 5, BF16, "tree"), ([0, 0, 2], 1, 1, 128, 128, F32, "tree"),
])
@pytest.mark.parametrize("modes", MODES)
def test_tree_decode_and_commit(layout, counts, Hk, Hv, dk, dv, dtype, shape, modes):
    c = make(counts, Hk, Hv, dk, dv, dtype=dtype, shape=shape, layout=layout, seed=sum(counts) + dk)
    ref, ref_deltas, nodes = reference(c, **modes)
    for out_dtype in ([F32] if dtype == F32 else [BF16, F32]):
        out, deltas = decode(c, out_dtype, **modes)
        assert out.dtype == out_dtype and R.rel(out, ref) < TOL + (HALF_STEP if out_dtype == BF16 else 0)
        assert R.rel(deltas, ref_deltas) < TOL
    g = torch.Generator().manual_seed(1)
    accepted = [int(torch.randint(-1, n, (1,), generator=g)) if n else -1 for n in counts]
    gates = {k: v for k, v in modes.items() if k != "beta_mode"}
    for take in (accepted, [n - 1 for n in counts]):
        pool = commit(c, ref_deltas.float().cuda(), take, **gates)
        expect = c["pool"].double()
        for b, a in enumerate(take):
            if a >= 0:
                S = nodes[b][a]
                expect[int(c["idx"][b])] = S if layout == "K_FIRST" else S.transpose(1, 2)
        assert R.rel(pool, expect) < TOL_COMMIT
        kept = [s for s in range(pool.shape[0]) if s not in [int(c["idx"][b]) for b, a in enumerate(take) if a >= 0]]
        assert torch.equal(pool.cpu()[kept], c["pool"][kept])


@pytest.mark.parametrize("max_nodes", [5, 8, 9, 16, 32, 33, 64])
def test_every_kernel_size_gives_the_same(max_nodes):
    c = make([5, 0, 4], 1, 2, 128, 128, dtype=BF16, seed=2)
    out, deltas = decode(c, F32, max_nodes=max_nodes)
    ref, ref_deltas, _ = reference(c)
    assert R.rel(out, ref) < TOL and R.rel(deltas, ref_deltas) < TOL
    pool = commit(c, deltas, [4, -1, 2], max_nodes=max_nodes)
    assert R.rel(pool, commit(c, deltas, [4, -1, 2])) < 2 * TOL_COMMIT


def test_one_node_equals_the_single_token_step():
    c = make([1] * 6, 2, 4, 128, 128, dtype=BF16, seed=3)
    out, deltas = decode(c, F32)
    pool = commit(c, deltas, [0] * 6)
    pool2 = c["pool"].cuda()
    out2 = kda.kda_decode(*gpu(c, "q", "k", "v", "raw", "beta", "a_log", "dt_bias"), pool2, c["idx"].cuda(), output_dtype=F32)
    assert R.rel(out, out2) < TOL and R.rel(pool, pool2) < TOL


def test_chain_equals_prefill():
    c = make([50, 21], 1, 2, 64, 64, shape="chain", seed=4)
    out, deltas = decode(c, F32)
    pool = commit(c, deltas, [49, 20])
    pool2 = c["pool"].cuda()
    out2 = kda.kda_chunk_fwd(*gpu(c, "q", "k", "v", "raw", "beta", "a_log", "dt_bias", "cu"), pool2, c["idx"].cuda())
    assert R.rel(out, out2) < 2 * TOL and R.rel(pool, pool2) < 2 * TOL


def test_strong_and_saturated_gates():
    # decays that underflow along the path: nothing of the far ancestors or the state may come back
    c = make([24], 1, 1, 128, 128, shape="chain", seed=5)
    c["raw"][:, 0, :40] = 30.0
    c["raw"][3, 0, 40:60] = float("inf")
    c["raw"][:, 0, 60:80] = float("-inf")
    ref, ref_deltas, nodes = reference(c)
    out, deltas = decode(c, F32)
    assert R.rel(out, ref) < TOL and R.rel(deltas, ref_deltas) < TOL
    pool = commit(c, deltas, [23])
    assert R.rel(pool[int(c["idx"][0])], nodes[0][23]) < TOL


def test_siblings_do_not_see_each_other():
    c = make([9], 1, 1, 128, 128, dtype=BF16, shape="star", seed=6)
    out, _ = decode(c, F32)
    for i in range(9):
        one = {**c, "counts": [1], "cu": torch.tensor([0, 1], dtype=torch.int32), "parents": torch.tensor([-1], dtype=torch.int32)}
        for k in ("q", "k", "v", "raw", "beta"):
            one[k] = c[k][i:i + 1]
        alone, _ = decode(one, F32)
        assert R.rel(out[i:i + 1], alone) < TOL


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("node", [0, 3, 20])
def test_what_is_not_finite_stays_on_its_branch(bad, node):
    n = 40
    c = make([n], 1, 1, 128, 128, dtype=BF16, seed=10)
    ref, ref_deltas, _ = reference(c)
    par = c["parents"].tolist()
    hit = {node}
    for i in range(node + 1, n):
        if par[i] in hit:
            hit.add(i)
    clean = [i for i in range(n) if i not in hit]
    assert clean or node == 0
    c["v"][node, 0, 5] = bad
    out, deltas = decode(c, F32)
    # column 5 of the node and of what follows it; every other branch and every other column as before
    assert not bool(torch.isfinite(out[node, 0, 5])) and not bool(torch.isfinite(deltas[node, 0, 5]))
    assert R.rel(out[clean], ref[clean]) < TOL and R.rel(deltas[clean], ref_deltas[clean]) < TOL
    others = [j for j in range(128) if j != 5]
    assert R.rel(out[:, :, others], ref[:, :, others]) < TOL


@pytest.mark.parametrize("what", ["slot", "parent of its own", "parent ahead", "parent below -1", "too many", "decreasing",
                                  "past the end"])
def test_bad_trees_are_reported_and_skipped(what):
    c = make([4, 6, 3], 1, 1, 128, 128, seed=7)
    max_nodes = 6
    if what == "slot":
        c["idx"][1] = -1
    elif what == "parent of its own":
        c["parents"][4 + 2] = 2
    elif what == "parent ahead":
        c["parents"][4 + 2] = 5
    elif what == "parent below -1":
        c["parents"][4 + 2] = -2
    elif what == "too many":
        max_nodes = 5
    elif what == "decreasing":
        c["cu"] = torch.tensor([0, 4, 2, 3], dtype=torch.int32)
    else:
        c["cu"] = torch.tensor([0, 4, 14, 14], dtype=torch.int32)
        max_nodes = 64
    out, deltas = torch.full((13, 1, 128), 5.0, device="cuda"), torch.full((13, 1, 128), 6.0, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    pool = c["pool"].cuda()
    kda.kda_tree_decode(*gpu(c, "q", "k", "v", "raw", "beta", "a_log", "dt_bias", "cu", "parents"), pool, c["idx"].cuda(),
                        out, deltas, max_nodes=max_nodes, device_status=status)
    assert int(status) == kda.ERR_DEVICE_CHECK
    first = {**c, "counts": [4]}
    for k in ("q", "k", "v", "raw", "beta", "parents"):
        first[k] = c[k][:4]
    ref, ref_deltas, nodes = reference(first)
    own = 2 if what == "decreasing" else 4  # the third sequence then has node 2, the first one's row
    assert R.rel(out[:own], ref[:own]) < TOL and R.rel(deltas[:own], ref_deltas[:own]) < TOL
    if what not in ("decreasing",):
        assert bool((out[4:10] == 5.0).all()) and bool((deltas[4:10] == 6.0).all())
    status.zero_()
    deltas[:4] = ref_deltas.float().cuda()
    kda.kda_tree_commit(*gpu(c, "k", "raw", "a_log", "dt_bias"), deltas, *gpu(c, "cu", "parents"),
                        torch.tensor([3, 2, -1], dtype=torch.int32, device="cuda"), pool, c["idx"].cuda(),
                        max_nodes=max_nodes, device_status=status)
    assert int(status) == kda.ERR_DEVICE_CHECK
    expect = c["pool"].double()
    expect[int(c["idx"][0])] = nodes[0][3]
    assert R.rel(pool, expect) < TOL_COMMIT


def test_accepted_outside_the_tree_is_reported():
    c = make([3, 2], 1, 1, 128, 128, seed=8)
    _, deltas = decode(c)
    for bad in ([3, 1], [-2, 1]):
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        pool = commit(c, deltas, bad, status=status)
        assert int(status) == kda.ERR_DEVICE_CHECK
        slot = int(c["idx"][0])
        assert torch.equal(pool[slot].cpu(), c["pool"][slot])
        assert not torch.equal(pool[int(c["idx"][1])].cpu(), c["pool"][int(c["idx"][1])])


def test_unaligned_pool_and_other_stream_and_graph():
    c = make([12, 7], 1, 2, 128, 128, dtype=BF16, seed=9)
    out, deltas = decode(c, BF16)
    pool = commit(c, deltas, [5, 6])
    flat = torch.empty(c["pool"].numel() + 1, device="cuda")
    odd = flat[1:].view(c["pool"].shape)
    odd.copy_(c["pool"])
    out2, deltas2 = decode(c, BF16, pool=odd)
    assert torch.equal(out, out2) and torch.equal(deltas, deltas2)
    assert torch.equal(commit(c, deltas, [5, 6], pool=odd), pool)
    names = ("q", "k", "v", "raw", "beta", "a_log", "dt_bias", "cu", "parents")
    args = gpu(c, *names)
    idx, acc = c["idx"].cuda(), torch.tensor([5, 6], dtype=torch.int32, device="cuda")
    pool3 = c["pool"].cuda()

    def step(stream=None):
        o, dl = kda.kda_tree_decode(*args, pool3, idx, max_nodes=12, stream=stream)
        kda.kda_tree_commit(args[1], args[3], args[5], args[6], dl, args[7], args[8], acc, pool3, idx, max_nodes=12, stream=stream)
        return o

    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    o = step(side)
    side.synchronize()
    assert torch.equal(o, out) and torch.equal(pool3, pool)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o = step()
    for _ in range(2):  # a replay goes on from the state that the last one left
        pool3.copy_(c["pool"])
        graph.replay()
        assert torch.equal(o, out) and torch.equal(pool3, pool)
