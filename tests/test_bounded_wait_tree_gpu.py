"""The wait for a tree's state, made to run out on purpose without a fault or a hang: with the test hook the copy
is not started.  Every sequence then gives up after its limits (about two seconds, all at once), reports it and
writes nothing, and the next call on the same context is right."""
import ctypes
import time

import pytest
import torch

import kimi_delta_attention_23_b200 as kda
import state_ops_reference as R

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("max_nodes", [32, 64])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_a_state_that_never_comes(dtype, max_nodes):
    lib, M, H, d = kda.load_library(), 20, 2, 128
    g = torch.Generator().manual_seed(3)
    n = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    host = [(n(M, H, d) / 11.3).to(dtype) for _ in range(2)] + [n(M, H, d).to(dtype), n(M, H, d), n(M, H), torch.rand(H, generator=g),
                                                                n(H, d)]
    parents = torch.tensor([(i - 1) // 2 for i in range(M)], dtype=torch.int32)
    parents[0] = -1
    pool = n(1, H, d, d) * 0.3
    c = [t.cuda() for t in (*host, torch.tensor([0, M], dtype=torch.int32), parents)]
    gpool, idx, status = pool.cuda(), torch.zeros(1, dtype=torch.int32).cuda(), torch.zeros(1, dtype=torch.int32).cuda()
    out, deltas = torch.full((M, H, d), 5.0, device="cuda"), torch.full((M, H, d), 6.0, device="cuda")
    at = lambda t: ctypes.c_void_p(t.data_ptr())  # noqa: E731

    def call(flags):
        status.zero_()
        stream = ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
        kind = 1 if dtype == torch.bfloat16 else 0
        assert lib.kda_tree_decode(*(at(t) for t in c[:3]), kind, *(at(t) for t in c[3:]), 1, M, max_nodes, H, H, d, d, at(gpool), 1,
                                   at(idx), at(out), 0, at(deltas), flags, -5.0, at(status), stream) == 0
        torch.cuda.synchronize()
        return int(status)

    t0 = time.monotonic()
    assert call(kda.DEBUG_WITHHOLD_HANDOFF) == kda.ERR_DEVICE_TIMEOUT
    assert time.monotonic() - t0 < 30.0
    assert bool((out == 5.0).all()) and bool((deltas == 6.0).all())
    assert call(0) == 0
    ref, ref_deltas, _ = R.tree(*(t.double() for t in host), [M], parents, pool.double())
    # 4e-5, as of the trees' own tests
    assert R.rel(out, ref) < 4e-5 and R.rel(deltas, ref_deltas) < 4e-5
    assert torch.equal(gpool.cpu(), pool)
