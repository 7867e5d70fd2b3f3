"""A serving step of a stack that mixes KDA and the gated linear recurrence, its operators together:
prefill both, fork every request into two samples, check drafted trees, commit different paths, free
some samples, pack the pools, decode on.  Checked against each sample run alone, token by token in
64 bits.  Tolerance: the prefill's fp32 kernel and the tree's products are each within 4e-5 of their
inputs' sizes, and the later steps contract; 1e-4 as the other fp32 parity tests.
"""
import pytest
import torch

import kimi_delta_attention_23_b200 as kda
import state_ops_reference as R

pytestmark = pytest.mark.gpu
TOL = 1e-4


def test_serving_step():
    g = torch.Generator().manual_seed(0)
    B, H, dk, dv, d, slots = 3, 2, 64, 64, 48, 12
    n = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    unit = lambda t: t / t.norm(dim=-1, keepdim=True)  # noqa: E731
    a_log, bias, a_log2, bias2 = torch.rand(H, generator=g), n(H, dk) * 0.3, torch.rand(H, generator=g), n(H, d) - 2

    def tokens(m):
        return dict(q=unit(n(m, H, dk)), k=unit(n(m, H, dk)), v=n(m, H, dv), raw=n(m, H, dk), beta=n(m, H),
                    x=n(m, H, d), raw2=n(m, H, d), beta2=n(m, H))

    def on_gpu(t, *names):
        return [t[k].cuda() for k in names]

    kda_par, glr_par = [a_log.cuda(), bias.cuda()], [a_log2.cuda(), bias2.cuda()]
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    lengths = [70, 5, 33]
    prompt = tokens(sum(lengths))
    cu = torch.tensor([0] + lengths, dtype=torch.int32).cumsum(0).int().cuda()
    pool, pool2 = torch.zeros(slots, H, dk, dv, device="cuda"), torch.zeros(slots, H, d, device="cuda")
    live = torch.zeros(slots, dtype=torch.int32, device="cuda")
    first = torch.tensor([7, 2, 10], dtype=torch.int32, device="cuda")
    live[first.long()] = 1
    kda.kda_chunk_fwd(*on_gpu(prompt, "q", "k", "v", "raw", "beta"), *kda_par, cu, pool, first, device_status=st)
    kda.kda_glr_fwd(*on_gpu(prompt, "x", "raw2", "beta2"), *glr_par, cu, pool2, first, input_mode="norm", device_status=st)

    # a second sample of every request; both pools share the slots' numbers
    live2 = live.clone()
    second = kda.kda_pool_fork(pool, live, first, device_status=st)
    assert torch.equal(second, kda.kda_pool_fork(pool2, live2, first, device_status=st))
    assert second.tolist() == [0, 1, 3] and torch.equal(live, live2)
    idx = torch.cat([first, second])

    counts = [4, 0, 6, 3, 5, 1]
    draft = tokens(sum(counts))
    parents = [-1, 0, 0, 1] + [-1, 0, 1, 1, -1, 4] + [-1, -1, 0] + [-1, 0, 1, 2, 3] + [-1]
    cun = torch.tensor([0] + counts, dtype=torch.int32).cumsum(0).int().cuda()
    par = torch.tensor(parents, dtype=torch.int32, device="cuda")
    accepted = [3, -1, 2, 2, 4, -1]
    out, deltas = kda.kda_tree_decode(*on_gpu(draft, "q", "k", "v", "raw", "beta"), *kda_par, cun, par, pool, idx,
                                      max_nodes=6, device_status=st)
    kda.kda_tree_commit(*on_gpu(draft, "k", "raw"), *kda_par, deltas, cun, par,
                        torch.tensor(accepted, dtype=torch.int32, device="cuda"), pool, idx, max_nodes=6, device_status=st)
    # the recurrence takes the accepted tokens as a short prefill
    paths, m0 = [], 0
    for b, c in enumerate(counts):
        path, a = [], accepted[b]
        while a >= 0:
            path.insert(0, m0 + a)
            a = parents[m0 + a]
        paths.append(path)
        m0 += c
    flat = [m for p in paths for m in p]
    taken = {k: draft[k][flat] for k in draft}
    cut = torch.tensor([0] + [len(p) for p in paths], dtype=torch.int32).cumsum(0).int().cuda()
    kda.kda_glr_fwd(*on_gpu(taken, "x", "raw2", "beta2"), *glr_par, cut, pool2, idx, input_mode="norm", device_status=st)

    # two samples end; what is left is packed, in both pools alike
    gone = idx[[0, 4]].contiguous()
    stay = idx[[1, 2, 3, 5]].contiguous()
    live2.copy_(live)
    stay2 = stay.clone()
    kda.kda_pool_free(pool, live, gone, device_status=st)
    kda.kda_pool_free(pool2, live2, gone, device_status=st)
    assert int(kda.kda_pool_compact(pool, live, stay, device_status=st)) == 4
    assert int(kda.kda_pool_compact(pool2, live2, stay2, device_status=st)) == 4
    assert torch.equal(stay, stay2) and sorted(stay.tolist()) == [0, 1, 2, 3]

    last = tokens(4)
    o = kda.kda_decode(*on_gpu(last, "q", "k", "v", "raw", "beta"), *kda_par, pool, stay, device_status=st)
    y = kda.kda_glr_decode(*on_gpu(last, "x", "raw2", "beta2"), *glr_par, pool2, stay, input_mode="norm", device_status=st)
    assert int(st) == 0

    # every sample alone
    def run(seq, t, ms):
        for m in ms:
            gt = R.gate(t["raw"][m].double(), a_log.double(), bias.double(), "original", 0)
            seq[0], seq[2], _ = R.kda_step(seq[0], *(t[k][m].double() for k in ("q", "k", "v")), gt,
                                           torch.sigmoid(t["beta"][m].double()))
            gy, seq[1] = R.glr(*(t[k][m:m + 1].double() for k in ("x", "raw2", "beta2")), a_log2.double(), bias2.double(), [1],
                               seq[1], input_mode="norm")
            seq[3] = gy[0]
        return seq

    ends = [0] + torch.tensor(lengths).cumsum(0).tolist()
    for row, b in enumerate([1, 2, 3, 5]):
        r = b % 3
        seq = [torch.zeros(H, dk, dv, dtype=torch.float64), torch.zeros(1, H, d, dtype=torch.float64), None, None]
        run(seq, prompt, range(ends[r], ends[r + 1]))
        run(seq, draft, paths[b])
        run(seq, last, [row])
        assert R.rel(o[row], seq[2]) < TOL and R.rel(y[row], seq[3]) < TOL
        assert R.rel(pool[int(stay[row])], seq[0]) < TOL and R.rel(pool2[int(stay[row])], seq[1][0]) < TOL
