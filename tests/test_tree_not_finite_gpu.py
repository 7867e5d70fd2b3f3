"""What is not finite in drafted trees: it stays on its branch, in every form of the kernel (state staged or not, every
output type), and a gate that is not a number is one for the commit as much as for the tree."""
import pytest
import torch

import kimi_delta_attention_23_b200 as kda
import test_tree_gpu as T
import state_ops_reference as R

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("dtype,out_dtype", [(BF16, BF16), (BF16, F32), (F32, F32)])
@pytest.mark.parametrize("nodes,node,dk,dv", [(7, 2, 128, 128), (16, 0, 128, 128), (16, 5, 128, 128), (30, 17, 128, 128),
                                              (60, 33, 128, 128), (14, 3, 72, 45), (50, 20, 72, 45)])
@pytest.mark.parametrize("layout", ["K_FIRST", "V_FIRST"])
def test_a_value_that_is_not_finite_stays_on_its_branch(bad, dtype, out_dtype, nodes, node, dk, dv, layout):
    c = T.make([nodes], 1, 1, dk, dv, dtype=dtype, layout=layout, seed=nodes + node)
    ref, ref_deltas, _ = T.reference(c)
    par, hit = c["parents"].tolist(), {node}
    for i in range(node + 1, nodes):
        if par[i] in hit:
            hit.add(i)
    clean = [i for i in range(nodes) if i not in hit]
    c["v"][node, 0, 5] = bad
    out, deltas = T.decode(c, out_dtype)
    assert not bool(torch.isfinite(out[sorted(hit), 0, 5]).any()) and not bool(torch.isfinite(deltas[sorted(hit), 0, 5]).any())
    # the tolerance of the trees' own tests, and half a step of a bf16 output
    tol = T.TOL + (2.0 ** -8 if out_dtype == BF16 else 0.0)
    if clean:
        assert R.rel(out[clean], ref[clean]) < tol and R.rel(deltas[clean], ref_deltas[clean]) < T.TOL
    others = [j for j in range(dv) if j != 5]
    assert R.rel(out[:, :, others], ref[:, :, others]) < tol
    assert R.rel(deltas[:, :, others], ref_deltas[:, :, others]) < T.TOL


@pytest.mark.parametrize("modes", [dict(), dict(gate_mode="safe", gate_lower_bound=-0.5)])
@pytest.mark.parametrize("nodes,dk,dv", [(6, 128, 128), (40, 128, 128), (6, 24, 40)])
def test_a_gate_that_is_not_a_number(modes, nodes, dk, dv):
    c = T.make([nodes], 1, 1, dk, dv, shape="chain", seed=nodes)
    c["raw"][3, 0, 7] = float("nan")
    out, deltas = T.decode(c, F32, **modes)
    assert bool(torch.isnan(out[3:]).all()) and bool(torch.isfinite(out[:3]).all())
    ref, ref_deltas, nodes_of = T.reference(c, **modes)
    assert R.rel(out[:3], ref[:3]) < T.TOL
    slot = int(c["idx"][0])
    good = T.commit(c, ref_deltas.float().cuda(), [2], **modes)
    assert R.rel(good[slot], nodes_of[0][2]) < T.TOL_COMMIT
    # committed with deltas that are all numbers, so that nothing but the gate says so
    spoilt = T.commit(c, torch.zeros_like(deltas), [4], **modes)[slot, 0]
    assert bool(torch.isnan(spoilt[7]).all())
    kept = [j for j in range(dk) if j != 7]
    assert bool(torch.isfinite(spoilt[kept]).all())
