"""The recurrence's bounded waits, made to run out on purpose without a fault or a hang.

The test hook has the last CTA of every chain's cluster withhold its first map, so the others (and it
itself) wait for something that never comes.  Each gives up after about a second, sends and fetches nothing
more, waits for the copies it has under way and meets the others at the cluster's closing barrier, so that no CTA
ends while another may still write to its shared memory.  The call must come back with the status, and the next
call on the same context must be right."""
import ctypes
import time

import pytest
import torch

import kimi_delta_attention_23_b200 as kda
import state_ops_reference as R

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16


@pytest.mark.parametrize("lengths", [[2600, 300], [50]])
@pytest.mark.parametrize("dtype,d", [(BF16, 128), (F32, 128), (F32, 37)])
def test_withheld_map_times_out_and_the_context_stays_usable(dtype, d, lengths):
    lib, H, B, T = kda.load_library(), 1, len(lengths), sum(lengths)
    g = torch.Generator().manual_seed(d)
    n = lambda *s, m=0.0: torch.randn(*s, generator=g) + m  # noqa: E731
    host = dict(x=n(T, H, d).to(dtype), raw=n(T, H, d).to(dtype), beta=n(T, H), a_log=torch.rand(H, generator=g),
                bias=n(H, d, m=-1.5), dout=n(T, H, d).to(dtype), pool=n(B, H, d))
    c = {k: v.cuda() for k, v in host.items()}
    cu = torch.tensor([0] + lengths, dtype=torch.int32).cumsum(0).to(torch.int32).cuda()
    idx, status = torch.arange(B, dtype=torch.int32).cuda(), torch.zeros(1, dtype=torch.int32).cuda()
    kept = torch.zeros(kda.kda_glr_checkpoint_shape(T, B, H, d)).cuda()
    out, dx, draw = (torch.empty_like(c["x"]) for _ in range(3))
    sums = [torch.empty(s, device="cuda") for s in ((T, H), (H,), (H, d), (B, H, d))]
    work = torch.empty(kda.kda_glr_bwd_workspace_size(T, B, H, d), dtype=torch.uint8, device="cuda")
    kind = 1 if dtype == BF16 else 0

    def at(t):
        return ctypes.c_void_p(t.data_ptr())

    def forward(flags):
        status.zero_()
        c["pool"].copy_(host["pool"])
        stream = ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
        assert lib.kda_glr_fwd(at(c["x"]), kind, at(c["raw"]), kind, at(c["beta"]), at(c["a_log"]), at(c["bias"]), at(cu), B, T,
                               H, d, at(c["pool"]), B, at(idx), at(out), kind, at(kept), flags, -5.0, at(status), stream) == 0
        torch.cuda.synchronize()
        return int(status)

    def backward(flags):
        status.zero_()
        stream = ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
        assert lib.kda_glr_bwd(at(c["dout"]), kind, at(c["x"]), kind, at(c["raw"]), kind, at(c["beta"]), at(c["a_log"]),
                               at(c["bias"]), at(cu), B, T, H, d, at(kept), None, at(dx), at(draw), *(at(t) for t in sums),
                               flags, -5.0, at(work), work.numel(), at(status), stream) == 0
        torch.cuda.synchronize()
        return int(status)

    for call in (forward, backward):
        t0 = time.monotonic()
        assert call(kda.DEBUG_WITHHOLD_HANDOFF) == kda.ERR_DEVICE_TIMEOUT
        assert time.monotonic() - t0 < 30.0  # about a second per wait, all at once
        assert forward(0) == 0 and backward(0) == 0
        leaves = {k: host[k].double().requires_grad_() for k in ("x", "raw", "beta", "a_log", "bias", "pool")}
        ref, final = R.glr(leaves["x"], leaves["raw"], leaves["beta"], leaves["a_log"], leaves["bias"], lengths, leaves["pool"])
        grads = torch.autograd.grad((ref * host["dout"].double()).sum(), [leaves["x"], leaves["pool"]])
        # the tolerances of the recurrence's own tests: 5e-5 and, of gradients, 1e-4; half a bf16 step more
        step = 2.0 ** -8 if dtype == BF16 else 0.0
        assert R.rel(out, ref.detach()) < 5e-5 + step and R.rel(c["pool"], final.detach()) < 5e-5
        assert R.rel(dx, grads[0]) < 1e-4 + step and R.rel(sums[3], grads[1]) < 1e-4
