"""What the build needs, and what it makes do without.  Nothing is compiled here: the compilers are stand-ins."""
import os
import subprocess
import warnings

import pytest
import torch

import kimi_delta_attention_23_b200 as kda
from kimi_delta_attention_23_b200 import build as kbuild


@pytest.fixture
def tree(tmp_path, monkeypatch):
    """A build into an empty folder, by compilers that write down what they are asked."""
    for name in ("LIB", "CHECK_LIB", "CHECK_FOR", "BUILD"):
        monkeypatch.setattr(kbuild, name, str(tmp_path / os.path.basename(getattr(kbuild, name))))
    asked, missing = [], set()

    def run(cmd, **kw):
        tool = os.path.basename(cmd[0])
        if tool in missing:
            raise FileNotFoundError(cmd[0])
        asked.append(tool)
        open(cmd[cmd.index("-o") + 1], "w").close()
        return subprocess.CompletedProcess(cmd, 0, "", "")

    monkeypatch.setattr(kbuild.subprocess, "run", run)
    return asked, missing


def test_the_library_is_built_without_a_host_compiler_for_the_binding(tree):
    asked, missing = tree
    missing.add("g++")
    with warnings.catch_warnings(record=True) as said:
        warnings.simplefilter("always")
        assert kbuild.build() == kbuild.LIB
    assert os.path.exists(kbuild.LIB) and not os.path.exists(kbuild.CHECK_LIB) and not kbuild.check_fits()
    assert any("checked in Python" in str(w.message) for w in said)
    # without it the checks in Python are asked
    look = kda._checker("x v T,H,d")
    assert look(torch.zeros(1, 1, 1)) is None


def test_the_library_is_still_required(tree):
    tree[1].add(os.path.basename(kbuild.NVCC))
    with pytest.raises(OSError):
        kbuild.build()


def test_the_checks_are_built_again_for_another_torch(tree, monkeypatch):
    asked, _ = tree
    kbuild.build()
    assert kbuild.check_fits() and asked.count("g++") == 1
    kbuild.build()
    assert asked.count("g++") == 1
    monkeypatch.setattr(torch, "__version__", "0.0.0")
    assert not kbuild.check_fits()  # and so it is not loaded
    assert kda._checker("x v T,H,d")(torch.zeros(1, 1, 1)) is None
    kbuild.build()
    assert kbuild.check_fits() and asked.count("g++") == 2


@pytest.mark.gpu
def test_calls_without_the_compiled_checks(monkeypatch):
    from kimi_delta_attention_23_b200 import glr, tree
    f = lambda *s: torch.randn(*s, device="cuda", generator=torch.Generator("cuda").manual_seed(sum(s)))  # noqa: E731
    ints = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    T, H, d = 9, 2, 16

    def calls():
        pools = [f(3, H, d), f(3, H, d), f(3, H, d, d)]
        yield kda.kda_glr_fwd(f(T, H, d), f(T, H, d), f(T, H), f(H), f(H, d), ints(0, 4, 9), pools[0], ints(2, 0))
        yield kda.kda_glr_decode(f(2, H, d), f(2, H, d), f(2, H), f(H), f(H, d), pools[1], ints(2, 0))
        k, raw, a_log, bias, cu, parents = f(T, 1, d), f(T, H, d), f(H), f(H, d), ints(0, 4, 9), ints(-1, 0, 0, 2, -1, 0, 1, 1, -1)
        out, deltas = kda.kda_tree_decode(f(T, 1, d), k, f(T, H, d), raw, f(T, H), a_log, bias, cu, parents, pools[2], ints(1, 2))
        kda.kda_tree_commit(k, raw, a_log, bias, deltas, cu, parents, ints(3, -1), pools[2], ints(1, 2))
        yield from (out, deltas, *pools)

    want = list(calls())
    monkeypatch.setattr(glr, "_FWD", lambda *t: None)
    monkeypatch.setattr(glr, "_DECODE", lambda *t: None)
    for checkers in (tree._TREE, tree._COMMIT):
        for layout in checkers:
            monkeypatch.setitem(checkers, layout, lambda *t: None)
    assert all(torch.equal(a, b) for a, b in zip(want, calls(), strict=True))
