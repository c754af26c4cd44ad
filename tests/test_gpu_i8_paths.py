"""The INT8 layer and product on each of their kernels, whatever a call of that
size picks: sizes at which a kernel's plan takes its longer ways (several
launches, more than 32 routes or experts in use, more than 1024 experts,
several passes over a CTA's rows), against the FP64 forms and bounds of
test_gpu_i8.py."""
import ctypes

import pytest
import torch
from test_gpu_i8 import (check_moe, check_product, codes, cq, distinct_ids, gen, layer,  # noqa: F401
                         moe_ref, product_ref, scales, tokens)

pytestmark = pytest.mark.gpu
AUTO, STREAM, SPLIT, PAIR, SORTED = range(5)


def stream():
    return torch.cuda.current_stream().cuda_stream


def moe_on(cq, path, x, ids, w, lw):
    T, H = x.shape
    k = ids.shape[1]
    E, _, I = lw[2].shape
    n = cq.lib().cq_test_moe_i8_workspace_size(T, k, E, H, I, path)
    ws = torch.empty(max(n, 256), dtype=torch.uint8, device="cuda")
    ro = torch.full((T * k, H), 7.0, device="cuda")
    out = torch.full((T, H), 7.0, device="cuda")
    st = cq.lib().cq_test_moe_i8(x.data_ptr(), T, ids.data_ptr(), w.data_ptr(), k, E,
                                 *(t.data_ptr() for t in lw), H, I, cq.F32, ro.data_ptr(),
                                 out.data_ptr(), ws.data_ptr(), ws.numel(), path, 0, 0, stream())
    assert st == 0
    return ro, out


LAYERS = [
    # T,   k,  E,     H,    I,   dropped
    (300,  5,  128,   48,   32,  0.1),     # streamed: two launches, the second shorter
    (1100, 2,  7,     32,   16,  0.0),     # ... three
    (40,   2,  2,     160,  96,  0.0),     # several chunks of an expert
    (20,   1,  1,     16400, 32, 0.0),     # long rows: fewer routes in a pass
    (9,    2,  3,     9216, 9232, 0.0),
    (100,  3,  90,    144,  80,  0.2),     # more than 32 experts in use
    (40,   4,  2000,  32,   48,  0.0),     # more than 1024 experts
    (30,   1,  16384, 16,   16,  0.3),     # as many as there can be
    (300,  2,  16384, 16,   32,  0.0),
    (70,   16, 896,   64,   32,  0.0),
    (260,  8,  256,   64,   48,  0.5),
    (2,    1,  3,     512,  256, 0.0),     # fewer routes than experts
]


@pytest.mark.parametrize("T,k,E,H,I,dropped", LAYERS)
def test_layers_on_both_paths(cq, T, k, E, H, I, dropped):  # noqa: F811
    g = gen(T + E)
    x, lw = tokens(g, T, H), layer(g, E, H, I)
    ids = distinct_ids(g, T, E, k)
    if dropped:
        ids = torch.where(torch.rand(T, k, generator=g, device="cuda") < dropped, -1, ids)
    w = torch.randn(T, k, generator=g, device="cuda")
    ref = moe_ref(x, ids, w, *lw)
    got = [moe_on(cq, path, x, ids, w, lw) for path in (STREAM, SORTED)]
    for ro, out in got:
        check_moe(ro, out, ref, k, False)
    assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[1][1])
    ro, out = cq.cq_moe_i8(x, ids, w, *lw)
    assert torch.equal(ro, got[0][0]) and torch.equal(out, got[0][1])
    assert cq.device_error() == (0, 0)


def test_sorted_layer_of_many_experts(cq):  # noqa: F811
    """More routes than a launch of 2000 experts holds, most experts with a full
    tile; the tokens' outputs are those of few."""
    T, k, E, H, I = 8500, 8, 2000, 16, 16
    g = gen(3)
    x, lw = tokens(g, T, H), layer(g, E, H, I)
    ids = distinct_ids(g, T, E, k)
    w = torch.rand(T, k, generator=g, device="cuda")
    n = ctypes.c_int64(0)
    assert cq.lib().cq_test_moe_i8_path(T, k, E, H, I, n) == SORTED and n.value < T
    ro, out = cq.cq_moe_i8(x, ids, w, *lw)
    for t in (0, n.value - 5, n.value, T - 9):
        few = moe_on(cq, STREAM, x[t:t + 9].contiguous(), ids[t:t + 9].contiguous(),
                     w[t:t + 9].contiguous(), lw)
        assert torch.equal(few[0], ro[t * k:(t + 9) * k]) and torch.equal(few[1], out[t:t + 9])
    assert cq.device_error() == (0, 0)


PRODUCTS = [
    # path,   M,    N,     K,    swiglu
    (STREAM,  8,    80000, 64,   False),    # several passes over a CTA's rows
    (STREAM,  8,    160000, 64,  True),
    (STREAM,  3,    129,   16384, False),
    (STREAM,  1,    100,   131072, True),
    (SPLIT,   1,    300,   272,  False),
    (SPLIT,   200,  1003,  1040, False),
    (SPLIT,   130,  514,   4112, True),
    (PAIR,    1,    300,   272,  True),
    (PAIR,    129,  260,   784,  False),
    (PAIR,    700,  4100,  528,  True),     # tiles cut along their tokens
]


@pytest.mark.parametrize("path,M,N,K,swiglu", PRODUCTS)
def test_products_on_a_chosen_path(cq, path, M, N, K, swiglu):  # noqa: F811
    g = gen(M + N)
    x, wq, ws = tokens(g, M, K), codes(g, N, K), scales(g, N, K=K)
    xq, am = cq.cq_quant_rows(x)
    epi = cq.EPI_SWIGLU if swiglu else cq.EPI_NONE
    ref = product_ref(xq, am, wq, ws)
    got = []
    buf = torch.empty(M * K + 4 * M + 4096, dtype=torch.uint8, device="cuda")
    for a, b in ((xq, am), (x, None)):
        y = torch.full((M, N // 2 if swiglu else N), 7.0, device="cuda")
        st = cq.lib().cq_test_product_i8(a.data_ptr(), None if b is None else b.data_ptr(), M,
                                         wq.data_ptr(), ws.data_ptr(), N, K, epi, cq.F32,
                                         y.data_ptr(), buf.data_ptr(), buf.numel(), path, 0, 0,
                                         stream())
        assert st == 0
        check_product(y, ref, swiglu, False)
        got.append(y)
    assert torch.equal(got[0], got[1])
    assert torch.equal(cq.cq_linear_i8(x, wq, ws, epilogue=epi), got[0])
    assert cq.device_error() == (0, 0)


@pytest.mark.parametrize("M,N,K,epi,path", [
    (1, 1000, 512, 0, STREAM), (8, 6144, 7168, 1, STREAM), (8, 300, 16384, 0, SPLIT),
    (9, 333, 4096, 0, SPLIT), (37, 7168, 2048, 0, SPLIT), (128, 6144, 7168, 1, SPLIT),
    (1000, 7163, 7168, 0, PAIR), (4096, 6144, 7168, 1, PAIR), (2049, 1281, 96, 0, PAIR),
])
def test_which_kernel_a_product_takes(cq, M, N, K, epi, path):  # noqa: F811
    assert cq.lib().cq_test_product_i8_path(M, N, K, epi) == path


@pytest.mark.parametrize("path", [STREAM, SORTED])
def test_nan_activations_have_code_0(cq, path):  # noqa: F811
    """A NaN activation does not raise its row's maximum and contributes nothing;
    a row of NaN is a row of zeros."""
    T, k, E, H, I = 12, 2, 4, 512, 96
    g = gen(8)
    x, lw = tokens(g, T, H), layer(g, E, H, I)
    ids, w = distinct_ids(g, T, E, k), torch.ones(T, k, device="cuda")
    x[1, 5] = 0.0
    x[2] = 0.0
    clean = moe_on(cq, path, x, ids, w, lw)
    x[1, 5] = float("nan")
    x[2] = float("nan")
    ro, out = moe_on(cq, path, x, ids, w, lw)
    assert torch.equal(ro, clean[0]) and torch.equal(out, clean[1])
    assert bool((out[2] == 0).all())
