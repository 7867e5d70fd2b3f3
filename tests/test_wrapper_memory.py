"""What a wrapper allocates itself belongs to the stream its kernels run on.

The allocator hands a block out again as soon as it is freed on the stream it belongs to, without waiting
for what still runs there; a kernel on another stream that got such a block would write into memory still
in use.  On the CPU the rule is checked with a stand-in for the streams and by reading the wrappers; on a
GPU the allocator itself says whose each result is."""
import ast
import contextlib
import glob
import os

import pytest
import torch

import kimi_delta_attention_23_b200 as kda

PACKAGE = os.path.dirname(os.path.abspath(kda.__file__))


class Streams:
    """Stands in for torch.cuda's current stream."""

    def __init__(self, monkeypatch):
        self.now, self.made, self.recorded = "own", [], []
        monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: self.now)
        monkeypatch.setattr(torch.cuda, "stream", self.on)

    @contextlib.contextmanager
    def on(self, stream):
        before, self.now = self.now, stream
        yield
        self.now = before

    def empty(self, n, device=None, dtype=None):
        self.made.append(self.now)
        outer = self

        class Tensor:
            def numel(self):
                return n

            def record_stream(self, stream):
                outer.recorded.append(stream)

            def is_contiguous(self):
                return False

            def contiguous(self):
                return outer.empty(n)
        return Tensor()


def test_made_on_the_calls_stream_and_handed_over(monkeypatch):
    s = Streams(monkeypatch)
    for stream, on, told in ((None, "own", []), ("own", "own", []), ("side", "side", ["own"])):
        s.made, s.recorded = [], []
        t = kda._make(stream, 0, s.empty, 4, device="cuda")
        kda._hand_over(stream, 0, t, None, s.empty(0))
        assert s.made[0] == on and s.recorded == told and s.now == "own"


def test_the_older_wrappers_tensors_too(monkeypatch):
    s = Streams(monkeypatch)
    monkeypatch.setattr(torch, "empty", s.empty)
    own = kda._Owned("side", 0)
    own.empty(4, dtype=torch.float32, device="cuda")
    own.contiguous(s.empty(4))
    assert s.made == ["side", "own", "side"]  # the second: the caller's own tensor
    own.launched()
    assert s.recorded == ["own"]


def test_no_wrapper_allocates_on_its_own():
    makers = {"empty", "empty_like", "zeros", "zeros_like", "ones", "full", "new_empty", "new_zeros"}
    for path in glob.glob(os.path.join(PACKAGE, "*.py")):
        if os.path.basename(path) in ("build.py", "distributed.py"):  # the latter runs whole with its stream current
            continue
        for node in ast.walk(ast.parse(open(path).read())):
            if not (isinstance(node, ast.Call) and isinstance(node.func, ast.Attribute) and node.func.attr in makers):
                continue
            if isinstance(node.func.value, ast.Name) and node.func.value.id == "own":
                continue
            on_host = any(k.arg == "pin_memory" for k in node.keywords) or not any(k.arg == "device" for k in node.keywords) \
                and node.func.attr == "zeros"
            assert on_host, f"{os.path.basename(path)}:{node.lineno} allocates device memory outside _make"


def _owner(t):
    """The stream whose memory a CUDA tensor is."""
    for seg in torch.cuda.memory_snapshot():
        if seg["address"] <= t.data_ptr() < seg["address"] + seg["total_size"]:
            return seg["stream"]
    raise AssertionError("not the allocator's")


@pytest.mark.gpu
def test_results_are_the_side_streams_memory():
    f = lambda *s, dtype=torch.float32: torch.zeros(*s, dtype=dtype, device="cuda")  # noqa: E731
    ints = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    T, H, d = 70, 2, 16
    glr = (f(T, H, d), f(T, H, d), f(T, H), f(H), f(H, d))
    kept, cu = f(*kda.kda_glr_checkpoint_shape(T, 1, H, d)), ints(0, T)
    tree = (f(5, 1, d), f(5, 1, d), f(5, H, d), f(5, H, d), f(5, H), f(H), f(H, d), ints(0, 5), ints(-1, 0, 1, 0, 0))
    pool = f(4, H, d, d)
    calls = [
        (kda.kda_glr_fwd, (*glr, cu, f(1, H, d), ints(0)), dict(checkpoints=kept)),
        (kda.kda_glr_decode, (*(t[:3] for t in glr[:3]), *glr[3:], f(3, H, d), ints(0, 1, 2)), {}),
        (kda.kda_glr_bwd, (glr[0], *glr, cu, kept), {}),
        (kda.kda_tree_decode, (*tree, pool, ints(1)), {}),
        (kda.kda_pool_fork, (pool, ints(1, 1, 0, 0), ints(0, 1)), {}),
        (kda.kda_pool_compact, (pool, ints(1, 0, 1, 0), ints(0, 2)), {}),
        (kda.kda_chunk_fwd, (*tree[:7], ints(0, 5), pool, ints(1)), {}),
        (kda.kda_decode, (*(t[:4] for t in tree[:5]), *tree[5:7], pool, ints(0, 1, 2, 3)), {}),
    ]
    side = torch.cuda.Stream()
    for call, args, kw in calls:
        # blocks of the current stream that were freed a moment ago: what must not be handed out here
        del [f(64) for _ in range(64)][:]
        torch.cuda.synchronize()
        for stream, owner in ((side, side.cuda_stream), (None, torch.cuda.current_stream().cuda_stream)):
            got = call(*args, stream=stream, **kw)
            got = got.values() if isinstance(got, dict) else got if isinstance(got, tuple) else (got,)
            torch.cuda.synchronize()
            assert all(_owner(t) == owner for t in got)
