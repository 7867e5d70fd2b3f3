"""Host-side refusals of the operators around the state pools: return codes of the C ABI before any
launch, and the binding's own checks.  No GPU: the pointers are never followed."""
import ctypes

import pytest
import torch

import kimi_delta_attention_23_b200 as kda
from kimi_delta_attention_23_b200 import build as kbuild

OK, INVALID, UNSUPPORTED, WORKSPACE = 0, 1, 2, 3


@pytest.fixture(scope="module")
def lib():
    kbuild.build()
    return kda.load_library()


def p(x):
    return ctypes.c_void_p(x) if x else None


def glr_fwd(lib, **over):
    a = dict(x=16, xt=1, raw=16, rt=1, beta=16, a_log=16, bias=16, cu=16, batch=1, T=16, H=2, d=128, pool=16, slots=4,
             idx=16, out=16, ot=1, ck=0, flags=0)
    a.update(over)
    return lib.kda_glr_fwd(p(a["x"]), a["xt"], p(a["raw"]), a["rt"], p(a["beta"]), p(a["a_log"]), p(a["bias"]), p(a["cu"]),
                           a["batch"], a["T"], a["H"], a["d"], p(a["pool"]), a["slots"], p(a["idx"]), p(a["out"]), a["ot"],
                           p(a["ck"]), a["flags"], -5.0, None, None)


@pytest.mark.parametrize("over,code", [
    (dict(batch=-1), INVALID), (dict(T=-1), INVALID), (dict(T=2 ** 31), INVALID), (dict(H=0), INVALID), (dict(d=0), INVALID),
    (dict(slots=0), INVALID), (dict(x=0), INVALID), (dict(raw=0), INVALID), (dict(beta=0), INVALID), (dict(a_log=0), INVALID),
    (dict(bias=0), INVALID), (dict(cu=0), INVALID), (dict(pool=0), INVALID), (dict(idx=0), INVALID), (dict(out=0), INVALID),
    (dict(flags=1 << 2), INVALID), (dict(flags=1 << 20), INVALID), (dict(xt=5), UNSUPPORTED), (dict(rt=5), UNSUPPORTED),
    (dict(ot=5), UNSUPPORTED), (dict(xt=0), UNSUPPORTED), (dict(xt=0, rt=0), UNSUPPORTED), (dict(d=129), UNSUPPORTED),
    (dict(batch=2 ** 30, H=64), INVALID), (dict(batch=0, T=0), OK),
])
def test_glr_fwd(lib, over, code):
    assert glr_fwd(lib, **over) == code


@pytest.mark.parametrize("over,code", [
    (dict(batch=-1), INVALID), (dict(H=0), INVALID), (dict(d=0), INVALID), (dict(slots=0), INVALID), (dict(x=0), INVALID),
    (dict(pool=0), INVALID), (dict(flags=4), INVALID), (dict(d=129), UNSUPPORTED), (dict(xt=0), UNSUPPORTED), (dict(batch=0), OK),
])
def test_glr_decode(lib, over, code):
    a = dict(x=16, xt=1, raw=16, rt=1, beta=16, a_log=16, bias=16, batch=1, H=2, d=128, pool=16, slots=4, idx=16, out=16,
             ot=1, flags=0)
    a.update(over)
    assert lib.kda_glr_decode(p(a["x"]), a["xt"], p(a["raw"]), a["rt"], p(a["beta"]), p(a["a_log"]), p(a["bias"]), a["batch"],
                              a["H"], a["d"], p(a["pool"]), a["slots"], p(a["idx"]), p(a["out"]), a["ot"], a["flags"], -5.0,
                              None, None) == code


@pytest.mark.parametrize("over,code", [
    (dict(batch=-1), INVALID), (dict(T=-1), INVALID), (dict(T=2 ** 31), INVALID), (dict(H=0), INVALID), (dict(d=0), INVALID),
    (dict(dout=0), INVALID), (dict(x=0), INVALID), (dict(cu=0), INVALID), (dict(ck=0), INVALID), (dict(dx=0), INVALID),
    (dict(draw=0), INVALID), (dict(dbeta=0), INVALID), (dict(da=0), INVALID), (dict(db=0), INVALID), (dict(di=0), INVALID),
    (dict(flags=4), INVALID), (dict(d=129), UNSUPPORTED), (dict(ot=3), UNSUPPORTED), (dict(xt=0, rt=0), UNSUPPORTED),
    (dict(ws=0), WORKSPACE), (dict(ws=16), WORKSPACE), (dict(short=1), WORKSPACE),
])
def test_glr_bwd(lib, over, code):
    a = dict(dout=16, ot=1, x=16, xt=1, raw=16, rt=1, beta=16, a_log=16, bias=16, cu=16, batch=1, T=16, H=2, d=128, ck=16,
             df=0, dx=16, draw=16, dbeta=16, da=16, db=16, di=16, flags=0, ws=256, short=0)
    a.update(over)
    need = lib.kda_glr_bwd_workspace_size(16, 1, 2, 128)
    assert need > 0
    assert lib.kda_glr_bwd(p(a["dout"]), a["ot"], p(a["x"]), a["xt"], p(a["raw"]), a["rt"], p(a["beta"]), p(a["a_log"]),
                           p(a["bias"]), p(a["cu"]), a["batch"], a["T"], a["H"], a["d"], p(a["ck"]), p(a["df"]), p(a["dx"]),
                           p(a["draw"]), p(a["dbeta"]), p(a["da"]), p(a["db"]), p(a["di"]), a["flags"], -5.0, p(a["ws"]),
                           need - a["short"], None, None) == code


def test_glr_sizes(lib):
    assert lib.kda_glr_checkpoints(0, 0) == 0 and lib.kda_glr_checkpoints(1000, 3) == 18
    assert lib.kda_glr_checkpoints(-1, 3) == 0
    assert lib.kda_glr_bwd_workspace_size(100, 0, 2, 8) == 0 and lib.kda_glr_bwd_workspace_size(100, 1, 2, 200) == 0
    # the kept states of two sequences never share an entry, whatever their lengths
    for lengths in ([1, 1, 1], [64, 64], [63, 65, 0, 1], [0, 0, 128], [127, 1, 64]):
        cu = [sum(lengths[:i]) for i in range(len(lengths) + 1)]
        used = [cu[b] // 64 + b + j for b, n in enumerate(lengths) for j in range(-(-n // 64))]
        assert len(set(used)) == len(used) and all(0 <= u < lib.kda_glr_checkpoints(cu[-1], len(lengths)) for u in used)


TREE = dict(q=16, k=16, v=16, t=1, raw=16, beta=16, a_log=16, bias=16, cu=16, par=16, batch=1, M=8, most=8, Hk=2, Hv=4, dk=128,
            dv=128, pool=16, slots=4, idx=16, out=16, ot=1, dl=16, acc=16, flags=0)


@pytest.mark.parametrize("over,code", [
    (dict(batch=-1), INVALID), (dict(M=-1), INVALID), (dict(M=2 ** 31), INVALID), (dict(most=0), INVALID),
    (dict(most=65), UNSUPPORTED), (dict(Hk=0), INVALID), (dict(Hv=3), INVALID), (dict(dk=0), INVALID), (dict(dv=0), INVALID),
    (dict(dk=129), UNSUPPORTED), (dict(dv=129), UNSUPPORTED), (dict(slots=0), INVALID), (dict(q=0), INVALID),
    (dict(par=0), INVALID), (dict(cu=0), INVALID), (dict(out=0), INVALID), (dict(dl=0), INVALID), (dict(pool=0), INVALID),
    (dict(flags=1 << 4), INVALID), (dict(t=4), UNSUPPORTED), (dict(t=0), UNSUPPORTED), (dict(ot=4), UNSUPPORTED),
    (dict(batch=2 ** 30, Hv=4), INVALID), (dict(batch=0, M=0), OK), (dict(M=0, q=0, k=0, v=0, par=0, out=0), OK),
])
def test_tree_decode(lib, over, code):
    a = {**TREE, **over}
    assert lib.kda_tree_decode(p(a["q"]), p(a["k"]), p(a["v"]), a["t"], p(a["raw"]), p(a["beta"]), p(a["a_log"]), p(a["bias"]),
                               p(a["cu"]), p(a["par"]), a["batch"], a["M"], a["most"], a["Hk"], a["Hv"], a["dk"], a["dv"],
                               p(a["pool"]), a["slots"], p(a["idx"]), p(a["out"]), a["ot"], p(a["dl"]), a["flags"], -5.0, None,
                               None) == code


@pytest.mark.parametrize("over,code", [
    (dict(batch=-1), INVALID), (dict(most=65), UNSUPPORTED), (dict(acc=0), INVALID), (dict(k=0), INVALID), (dict(dl=0), INVALID),
    (dict(Hv=3), INVALID), (dict(dk=129), UNSUPPORTED), (dict(t=7), UNSUPPORTED), (dict(idx=0), INVALID), (dict(batch=0), OK),
])
def test_tree_commit(lib, over, code):
    a = {**TREE, **over}
    assert lib.kda_tree_commit(p(a["k"]), a["t"], p(a["raw"]), p(a["a_log"]), p(a["bias"]), p(a["dl"]), p(a["cu"]), p(a["par"]),
                               p(a["acc"]), a["batch"], a["M"], a["most"], a["Hk"], a["Hv"], a["dk"], a["dv"], p(a["pool"]),
                               a["slots"], p(a["idx"]), a["flags"], -5.0, None, None) == code


@pytest.mark.parametrize("over,code", [
    (dict(pool=0), INVALID), (dict(layers=0), INVALID), (dict(slots=0), INVALID), (dict(elems=0), INVALID), (dict(n=-1), INVALID),
    (dict(elems=2 ** 62), INVALID), (dict(src=0), INVALID), (dict(ws=0), WORKSPACE), (dict(ws=128), WORKSPACE),
    (dict(short=1), WORKSPACE), (dict(n=0, src=0, dst=0, ws=0), OK),
])
def test_pool_calls(lib, over, code):
    a = dict(pool=16, layers=1, slots=8, elems=64, src=16, dst=16, n=3, ws=256, short=0, live=16, count=16)
    a.update(over)
    need = lib.kda_pool_workspace_size(max(a["n"], 0), max(a["slots"], 1)) - a["short"]
    head = (p(a["pool"]), a["layers"], a["slots"], a["elems"])
    tail = (p(a["ws"]), need, None, None)
    if code != WORKSPACE:  # a copy of this few pairs needs none
        assert lib.kda_pool_copy(*head, p(a["src"]), p(a["dst"]), a["n"], *tail) == code
    assert lib.kda_pool_fork(*head, p(a["live"]), p(a["src"]), p(a["dst"]), a["n"], *tail) == code
    assert lib.kda_pool_free(*head, p(a["live"]), p(a["src"]), a["n"], *tail) == code
    if a["n"]:  # without a list, packing still moves the slots
        assert lib.kda_pool_compact(*head, p(a["live"]), p(a["src"]), a["n"], p(a["count"]), *tail) == code


def test_pool_limits(lib):
    assert lib.kda_pool_copy(p(16), 1, 8, 64, p(16), p(16), 257, None, 0, None, None) == WORKSPACE
    assert lib.kda_pool_workspace_size(-1, 4) == 0 and lib.kda_pool_workspace_size(4, 0) == 0
    assert lib.kda_pool_copy(p(16), 1, 8, 64, p(16), p(16), kda.MAX_POOL_COPIES + 1, p(256), 1 << 30, None, None) == UNSUPPORTED
    assert lib.kda_pool_fork(p(16), 1, 8, 64, None, p(16), p(16), 3, p(256), 1 << 30, None, None) == INVALID
    assert lib.kda_pool_compact(p(16), 1, 8, 64, p(16), p(16), 3, None, p(256), 1 << 30, None, None) == INVALID


def test_binding_refuses_cpu_tensors():
    f, i = torch.zeros(2, 1, 4), torch.zeros(2, dtype=torch.int32)
    par = (torch.zeros(1), torch.zeros(1, 4))
    calls = [
        lambda: kda.kda_glr_fwd(f, f, torch.zeros(2, 1), *par, i, torch.zeros(1, 1, 4), i[:1]),
        lambda: kda.kda_glr_decode(f, f, torch.zeros(2, 1), *par, torch.zeros(2, 1, 4), i),
        lambda: kda.kda_glr_bwd(f, f, f, torch.zeros(2, 1), *par, i, torch.zeros(1, 1, 4)),
        lambda: kda.kda_tree_decode(f, f, f, f, torch.zeros(2, 1), *par, i, i, torch.zeros(1, 1, 4, 4), i[:1]),
        lambda: kda.kda_tree_commit(f, f, *par, f, i, i, i[:1], torch.zeros(1, 1, 4, 4), i[:1]),
        lambda: kda.kda_pool_copy(f, i, i), lambda: kda.kda_pool_fork(f, i, i), lambda: kda.kda_pool_free(f, i, i),
        lambda: kda.kda_pool_compact(f, i, i),
    ]
    for call in calls:
        with pytest.raises(ValueError, match="CUDA"):
            call()
