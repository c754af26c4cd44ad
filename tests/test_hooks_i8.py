"""The test hooks of the INT8 operators (include/cq_hooks_i8.h): declared,
exported, and refusing what the calls they stand for refuse (no GPU needed)."""
import ctypes
import os
import re

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE = 0x1000           # 256-byte aligned, never dereferenced
AUTO, STREAM, SPLIT, PAIR, SORTED = range(5)


@pytest.fixture(scope="module")
def lib():
    from bit_non_uniform_b200 import build
    build.build()
    import bit_non_uniform_b200 as cq
    return cq.lib()


def test_hooks_are_declared_and_exported(lib):
    with open(os.path.join(ROOT, "include", "cq_hooks_i8.h")) as f:
        names = re.findall(r"^CQ_API \w+ (cq_\w+)\(", f.read(), re.M)
    assert sorted(names) == ["cq_test_moe_i8", "cq_test_moe_i8_path",
                             "cq_test_moe_i8_workspace_size", "cq_test_product_i8",
                             "cq_test_product_i8_path"]
    for s in names:
        assert hasattr(lib, s), s


def product(lib, path, **kw):
    a = dict(x=FAKE, am=FAKE, M=4, K=128, N=64, epi=0)
    a.update(kw)
    return lib.cq_test_product_i8(a["x"], a["am"], a["M"], FAKE, FAKE, a["N"], a["K"], a["epi"], 0,
                                  FAKE, FAKE, 1 << 40, path, 0, 0, None)


def test_products_refuse_bad_arguments(lib):
    for path in (-1, SORTED, 5):
        assert product(lib, path) == 1
    assert product(lib, AUTO, M=-1) == 1 and product(lib, AUTO, x=None) == 1
    assert product(lib, SPLIT, K=24) == 2
    assert product(lib, PAIR, M=0) == 0


def test_layers_refuse_bad_arguments(lib):
    def call(path, T=2, H=64):
        return lib.cq_test_moe_i8(FAKE, T, FAKE, FAKE, 2, 4, FAKE, FAKE, FAKE, FAKE, H, 32, 0, None,
                                  FAKE, FAKE, 1 << 40, path, 0, 0, None)
    for path in (-1, SPLIT, PAIR, 5):
        assert call(path) == 1
        assert lib.cq_test_moe_i8_workspace_size(2, 2, 4, 64, 32, path) == 0
    assert call(SORTED, H=72) == 2 and call(STREAM, T=-1) == 1 and call(SORTED, T=0) == 0


def test_paths(lib):
    f = lib.cq_test_product_i8_path
    assert f(1, 1000, 512, 0) == f(8, 6144, 7168, 1) == STREAM
    assert f(8, 6144, 131072, 1) == SPLIT                    # the rows do not fit
    assert f(37, 7168, 2048, 0) == SPLIT and f(4096, 6144, 7168, 1) == PAIR
    assert f(0, 64, 128, 0) == f(4, 64, 24, 0) == 0
    g, n = lib.cq_test_moe_i8_path, ctypes.c_int64(0)
    assert g(16, 8, 64, 7168, 2048, n) == STREAM and n.value == 16
    assert g(2048, 8, 64, 7168, 2048, n) == SORTED and n.value == 2048
    assert g(4096, 8, 64, 7168, 2048, n) == SORTED and n.value == 2048
    assert g(2, 0, 64, 7168, 2048, n) == 0
    for T in (16, 2048):
        sizes = [lib.cq_test_moe_i8_workspace_size(T, 8, 64, 7168, 2048, p)
                 for p in (AUTO, STREAM, SORTED)]
        auto = lib.cq_moe_i8_workspace_size(T, 8, 64, 7168, 2048)
        assert sizes[0] == auto == sizes[1 if T == 16 else 2] and sizes[1] < sizes[2]


def moe_path(lib, T, k, E, H, I):
    n = ctypes.c_int64(0)
    return lib.cq_test_moe_i8_path(T, k, E, H, I, n), n.value


def test_no_layer_is_streamed_in_several_launches(lib):
    """A streamed launch holds 1024 routes, and a second one would read most
    experts again: 256 tokens of 896 experts, top 16, would read them 2.8 times."""
    for k, E, H, I in ((16, 896, 7168, 2048), (8, 256, 7168, 2048), (8, 2048, 2048, 1024),
                       (8, 16384, 512, 512), (7, 1000, 4096, 1536), (1000, 4000, 2048, 1024)):
        for T in (1, 2, 3, 60, 64, 72, 128, 129, 146, 147, 160, 256, 300, 512, 4096):
            path, per = moe_path(lib, T, k, E, H, I)
            assert path == SORTED or per == T, (T, k, E)
    assert moe_path(lib, 64, 16, 896, 7168, 2048) == (STREAM, 64)
    assert moe_path(lib, 65, 16, 896, 7168, 2048) == (SORTED, 65)
    assert moe_path(lib, 128, 8, 256, 7168, 2048)[0] == STREAM
    assert moe_path(lib, 129, 8, 256, 7168, 2048)[0] == SORTED


def test_small_experts_are_streamed_for_few_routes_only(lib):
    """Whatever their number: staging activations for every chunk of routes costs
    more than its rows' weights."""
    for E, H, I in ((4, 512, 256), (16, 512, 256), (128, 256, 128), (512, 512, 256),
                    (1024, 64, 80)):
        assert moe_path(lib, 16, 2, E, H, I)[0] == STREAM, E
        assert moe_path(lib, 17, 2, E, H, I)[0] == SORTED, E
    # middling ones up to 128 routes, 5 each
    assert moe_path(lib, 16, 8, 128, 1024, 512)[0] == STREAM
    assert moe_path(lib, 17, 8, 128, 1024, 512)[0] == SORTED
    assert moe_path(lib, 20, 2, 8, 1024, 512)[0] == STREAM
    assert moe_path(lib, 21, 2, 8, 1024, 512)[0] == SORTED
    # large ones while their weights bound both
    assert moe_path(lib, 40, 4, 32, 2048, 1024)[0] == STREAM
    assert moe_path(lib, 41, 4, 32, 2048, 1024)[0] == SORTED


def test_a_sorted_launch_holds_more_routes_of_more_experts(lib):
    """Every further launch reads the experts again: 2048 tokens of 896 experts,
    top 16, are 37 routes each and took two."""
    assert moe_path(lib, 2048, 16, 896, 7168, 2048) == (SORTED, 2048)
    assert moe_path(lib, 100000, 16, 896, 7168, 2048) == (SORTED, 4096)
    assert moe_path(lib, 100000, 8, 256, 7168, 2048) == (SORTED, 4096)
    assert moe_path(lib, 100000, 8, 64, 7168, 2048) == (SORTED, 2048)
    assert lib.cq_moe_i8_workspace_size(1 << 20, 16, 896, 7168, 2048) < 3 << 30
