"""Sequences that a cluster finishes in one step, or in one and a bit: every CTA of the cluster then reads the
starting state about when the first of them writes the final one.  Long runs of such calls on the same slots
must go on from exactly the state that the last one left."""
import pytest
import torch

import kimi_delta_attention_23_b200 as kda
import state_ops_reference as R

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("tokens", [1, 64, 65, 512, 513, 1024])
@pytest.mark.parametrize("heads", [1, 7])
def test_runs_of_short_sequences_carry_their_state(tokens, heads):
    g = torch.Generator().manual_seed(tokens)
    d, calls = 128, 12
    n = lambda *s, m=0.0: torch.randn(*s, generator=g) + m  # noqa: E731
    x, raw, beta = n(calls * tokens, heads, d), n(calls * tokens, heads, d), n(calls * tokens, heads)
    a_log, bias, pool = torch.rand(heads, generator=g), n(heads, d, m=-1.5), n(1, heads, d)
    gx, graw, gbeta, ga, gb = (t.cuda() for t in (x, raw, beta, a_log, bias))
    idx = torch.zeros(1, dtype=torch.int32, device="cuda")
    cu = torch.tensor([0, tokens], dtype=torch.int32, device="cuda")
    whole, apart = pool.cuda(), pool.cuda()
    outs = []
    for i in range(calls):
        s = slice(i * tokens, (i + 1) * tokens)
        outs.append(kda.kda_glr_fwd(gx[s], graw[s], gbeta[s], ga, gb, cu, apart, idx))
    one = kda.kda_glr_fwd(gx, graw, gbeta, ga, gb, cu * calls, whole, idx)
    ref, final = R.glr(x.double(), raw.double(), beta.double(), a_log.double(), bias.double(), [calls * tokens], pool.double())
    # 5e-5, as of the recurrence's own tests: decays off by 2^-21 on one side over a memory of 50 tokens
    assert R.rel(torch.cat(outs), ref) < 5e-5 and R.rel(one, ref) < 5e-5
    assert R.rel(apart, final) < 5e-5 and R.rel(whole, final) < 5e-5
