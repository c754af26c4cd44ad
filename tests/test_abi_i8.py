"""The INT8 operators and the MoE router refuse bad arguments on the host,
before touching the GPU (no GPU needed)."""
import ctypes
import os
import re

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE = 0x1000           # 256-byte aligned, never dereferenced
ODD = 0x1002


@pytest.fixture(scope="module")
def cq():
    from bit_non_uniform_b200 import build
    build.build()
    import bit_non_uniform_b200 as cq
    cq.lib()
    return cq


def test_declared_and_exported(cq):
    with open(os.path.join(ROOT, "include", "cq.h")) as f:
        text = f.read()
    for s in ("cq_gemm_i8", "cq_linear_i8", "cq_gemm_i8_workspace_size", "cq_moe_i8",
              "cq_moe_i8_workspace_size", "cq_moe_route"):
        assert re.search(rf"^CQ_API \w+ {s}\(", text, re.M), s
        assert hasattr(cq.lib(), s)


def product(cq, codes, **kw):
    a = dict(x=FAKE, am=FAKE, M=4, w=FAKE, s=FAKE, N=64, K=128, epi=0, dt=0, y=FAKE, ws=FAKE,
             nws=1 << 40)
    a.update(kw)
    tail = (a["M"], a["w"], a["s"], a["N"], a["K"], a["epi"], a["dt"], a["y"], a["ws"], a["nws"],
            None)
    if codes:
        return cq.lib().cq_gemm_i8(a["x"], a["am"], *tail)
    return cq.lib().cq_linear_i8(a["x"], *tail)


@pytest.mark.parametrize("codes", [True, False])
def test_products_refuse_bad_arguments(cq, codes):
    def call(**kw):
        return product(cq, codes, **kw)
    for bad in (dict(M=-1), dict(N=-1), dict(K=0), dict(K=-16), dict(epi=2), dict(dt=2),
                dict(x=None), dict(w=None), dict(s=None), dict(y=None)):
        assert call(**bad) == 1, bad
    for bad in (dict(K=24), dict(K=131088), dict(N=63, epi=1), dict(x=ODD), dict(w=ODD),
                dict(s=ODD), dict(y=ODD), dict(M=(1 << 24) + 1), dict(N=(1 << 24) + 2)):
        assert call(**bad) == 2, bad
    assert call(M=0) == 0 and call(N=0) == 0
    if codes:
        assert call(am=None) == 1 and call(am=ODD) == 2


def test_product_workspace(cq):
    f = cq.lib().cq_gemm_i8_workspace_size
    for bad in ((-1, 64, 128, 0), (4, -1, 128, 0), (4, 64, 24, 0), (4, 64, 0, 0), (4, 63, 128, 1),
                (4, 64, 128, 5), (0, 64, 128, 0), (4, 0, 128, 0)):
        assert f(*bad) == 0


def moe(cq, **kw):
    a = dict(x=FAKE, T=2, ids=FAKE, w=FAKE, k=2, E=4, wg=FAKE, sg=FAKE, wd=FAKE, sd=FAKE, H=64,
             I=32, dt=0, ro=FAKE, out=FAKE, ws=FAKE, nws=1 << 40)
    a.update(kw)
    return cq.lib().cq_moe_i8(a["x"], a["T"], a["ids"], a["w"], a["k"], a["E"], a["wg"], a["sg"],
                              a["wd"], a["sd"], a["H"], a["I"], a["dt"], a["ro"], a["out"],
                              a["ws"], a["nws"], None)


def test_moe_refuses_bad_arguments(cq):
    for bad in (dict(T=-1), dict(k=0), dict(E=0), dict(H=0), dict(I=-16), dict(dt=3),
                dict(x=None), dict(ids=None), dict(w=None), dict(wg=None), dict(sg=None),
                dict(wd=None), dict(sd=None), dict(ws=None)):
        assert moe(cq, **bad) == 1, bad
    for bad in (dict(E=16385), dict(k=1025), dict(H=72), dict(I=40), dict(H=131088),
                dict(I=131088), dict(x=ODD), dict(ids=ODD), dict(w=ODD), dict(wg=ODD),
                dict(sg=ODD), dict(wd=ODD), dict(sd=ODD), dict(ro=ODD), dict(out=ODD),
                dict(ws=FAKE + 16), dict(T=(1 << 24) + 1)):
        assert moe(cq, **bad) == 2, bad
    assert moe(cq, T=0) == 0


@pytest.mark.parametrize("k,E,H,I", [(8, 64, 7168, 2048), (2, 4, 64, 32), (16, 1000, 512, 256),
                                     (1, 1, 16, 16), (7, 40, 4096, 1536), (1000, 16384, 16, 32)])
def test_moe_workspace_serves_fewer_tokens(cq, k, E, H, I):
    """Whichever kernels a number of tokens takes: no fewer tokens need more."""
    f = cq.lib().cq_moe_i8_workspace_size
    sizes = [f(T, k, E, H, I) for T in list(range(300)) + list(range(300, 20000, 37)) + [1 << 20]]
    assert sizes == sorted(sizes) and sizes[1] > 0


def test_moe_workspace(cq):
    f = cq.lib().cq_moe_i8_workspace_size
    assert f(2, 2, 4, 64, 32) >= 2 * 2 * (64 + 32) * 4
    # one launch's routes bound the size
    assert f(100000, 8, 4, 64, 32) == f(2048, 8, 4, 64, 32)
    for bad in ((-1, 2, 4, 64, 32), (2, 0, 4, 64, 32), (2, 2, 0, 64, 32), (2, 2, 4, 72, 32),
                (2, 2, 4, 64, 40), (2, 1025, 4, 64, 32)):
        assert f(*bad) == 0, bad


def route(cq, **kw):
    a = dict(l=FAKE, ldt=0, T=3, E=8, k=2, b=FAKE, sc=0, rn=1, ids=FAKE, w=FAKE)
    a.update(kw)
    return cq.lib().cq_moe_route(a["l"], a["ldt"], a["T"], a["E"], a["k"], a["b"], a["sc"],
                                 a["rn"], ctypes.c_float(1.0), a["ids"], a["w"], None)


def test_route_refuses_bad_arguments(cq):
    for bad in (dict(T=-1), dict(E=0), dict(k=0), dict(k=9), dict(ldt=2), dict(sc=2), dict(rn=2),
                dict(l=None), dict(ids=None), dict(w=None)):
        assert route(cq, **bad) == 1, bad
    for bad in (dict(E=1025), dict(E=64, k=33), dict(l=ODD), dict(l=0x1001, ldt=1), dict(b=ODD),
                dict(ids=ODD), dict(w=ODD)):
        assert route(cq, **bad) == 2, bad
    assert route(cq, T=0) == 0


def test_binding_refuses_cpu_tensors(cq):
    x = torch.zeros((2, 64), dtype=torch.bfloat16)
    w = torch.zeros((8, 64), dtype=torch.int8)
    with pytest.raises(ValueError):
        cq.cq_linear_i8(x, w, torch.ones(8))
    with pytest.raises(ValueError):
        cq.cq_gemm_i8(w[:2], torch.ones(2), w, torch.ones(8))
    with pytest.raises(ValueError):
        cq.cq_gemm_i8(w[:2], None, w, torch.ones(8))
    with pytest.raises(ValueError):
        cq.cq_moe_route(torch.zeros((2, 8)), 2)
    with pytest.raises(ValueError):
        cq.cq_moe_i8(x, torch.zeros((2, 1), dtype=torch.int32), torch.ones((2, 1)),
                     torch.zeros((1, 32, 64), dtype=torch.int8), torch.ones((1, 32)),
                     torch.zeros((1, 64, 16), dtype=torch.int8), torch.ones((1, 64)))


def test_compiled_calls_leave_everything_unusual_to_the_binding(cq):
    """The compiled module is built beside libcq and answers None (the general
    path then says what is wrong) for tensors it does not take."""
    from bit_non_uniform_b200 import _cq_torch as direct
    x = torch.zeros((2, 64), dtype=torch.bfloat16)
    w, s = torch.zeros((8, 64), dtype=torch.int8), torch.ones(8)
    ids, tw = torch.zeros((2, 1), dtype=torch.int32), torch.ones((2, 1))
    lw = (torch.zeros((1, 32, 64), dtype=torch.int8), torch.ones((1, 32)),
          torch.zeros((1, 64, 16), dtype=torch.int8), torch.ones((1, 64)))
    for args in ((x, None, w, s, 0, 0, None), (1, None, w, s, 0, 0, None), (), (x,),
                 (x, None, None, None, 0, 0, None), (x[0], None, w, s, 0, 0, None),
                 (x, None, w, s, "0", 1 << 80, None)):
        assert direct.product(*args) is None, args
    for args in ((x, ids, tw, *lw, 0, None), (x, ids, None, *lw, 0, None), (x, 3), ()):
        assert direct.moe(*args) is None, args
    for args in ((tw, 1, None, 0, True, 1.0), (None, 1, None, 0, True, 1.0), (tw,)):
        assert direct.route(*args) is None, args
