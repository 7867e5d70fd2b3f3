"""Drafted trees where the value is all but predicted: v = k^T S rounded to bf16, so a delta is what is left of
the two after they cancel, and every bit that the product with the state loses shows in it.

Tolerance, relative to the size of what cancels (L2).  Each factor is held in two tf32 parts, which miss at
most 2^-22 of it, and the product of the two low parts (2^-22) is left out: 3 * 2^-22 = 7.2e-7 of a term.
The 128 terms are summed 8 at a time in fp32, each sum off by at most 2^-23 and on average half of that, the
running sum being no more than its end on average: 16 * 2^-24 = 9.5e-7.  The decay of one token is off by
1.5e-7 (slow gates: the polynomial's) and a rounding, the fp32 steps after the product by 2^-24 each: 3.5e-7.
In all 2e-6, which two bf16 parts (4e-6) exceed.  Trees of depth one, so that no path adds to it.
"""
import pytest
import torch

import kimi_delta_attention_23_b200 as kda

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
TOL = 2e-6


@pytest.mark.parametrize("layout", ["K_FIRST", "V_FIRST"])
@pytest.mark.parametrize("dtype,out_dtype", [(BF16, BF16), (BF16, F32), (F32, F32)])
@pytest.mark.parametrize("nodes,dk,dv", [(8, 128, 128), (16, 128, 128), (32, 128, 128), (64, 128, 128), (16, 96, 80), (40, 96, 80)])
def test_deltas_beside_a_good_prediction(layout, dtype, out_dtype, nodes, dk, dv):
    B, H = 3, 2
    g = torch.Generator().manual_seed(nodes + dk)
    M = B * nodes
    k = torch.randn(M, H, dk, generator=g)
    k = (k / k.norm(dim=-1, keepdim=True)).to(dtype)
    q = torch.randn(M, H, dk, generator=g).to(dtype)
    S = torch.randn(B, H, dk, dv, generator=g)
    raw, a_log, bias = torch.randn(M, H, dk, generator=g), torch.zeros(H), torch.full((H, dk), -5.0)
    beta = torch.ones(M, H)
    decay = (-torch.logaddexp(raw.double() - 5.0, torch.zeros((), dtype=torch.float64))).exp()
    seq = torch.arange(M) // nodes
    predicted = torch.einsum("mhc,mhcv->mhv", k.double() * decay, S.double()[seq])
    v = predicted.to(dtype)
    want = v.double() - predicted
    pool = S if layout == "K_FIRST" else S.transpose(2, 3).contiguous()
    cu = torch.arange(0, M + 1, nodes, dtype=torch.int32)
    out, deltas = kda.kda_tree_decode(
        *(t.cuda() for t in (q, k, v, raw, beta, a_log, bias, cu, torch.full((M,), -1, dtype=torch.int32), pool,
                             torch.arange(B, dtype=torch.int32))),
        max_nodes=nodes, output_dtype=out_dtype, beta_mode="probability", state_layout=layout)
    # sibling nodes do not see each other, so out = (q o decay)^T S + (q . k) delta
    assert float((deltas.double().cpu() - want).norm() / predicted.norm()) < TOL
    ref = torch.einsum("mhc,mhcv->mhv", q.double() * decay, S.double()[seq]) + \
        (q.double() * k.double()).sum(-1, keepdim=True) * want
    err = float((out.double().cpu() - ref).norm() / ref.norm())
    assert err < TOL + (2.0 ** -8 if out_dtype == BF16 else 0.0)


def test_the_outputs_type_does_not_change_what_is_committed():
    g = torch.Generator().manual_seed(1)
    M, H, d = 24, 2, 128
    t = lambda *s: torch.randn(*s, generator=g).cuda()  # noqa: E731
    q, k, v = (t(M, H, d).to(BF16) for _ in range(3))
    rest = (t(M, H, d), t(M, H), t(H), t(H, d), torch.tensor([0, 14, 24], dtype=torch.int32).cuda(),
            torch.tensor([i // 2 - 1 for i in range(14)] + [i // 2 - 1 for i in range(10)], dtype=torch.int32).cuda(),
            t(2, H, d, d), torch.tensor([1, 0], dtype=torch.int32).cuda())
    for nodes in (16, 64):
        a = kda.kda_tree_decode(q, k, v, *rest, max_nodes=nodes, output_dtype=BF16)
        b = kda.kda_tree_decode(q, k, v, *rest, max_nodes=nodes, output_dtype=F32)
        assert torch.equal(a[1], b[1]) and torch.equal(a[0], b[0].to(BF16))
