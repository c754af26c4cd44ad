"""Failure detection in the INT8 kernels without a GPU fault: every wait is
bounded.  A test hook withholds an arrival on each CTA's first piece of
operands, so that the waits for it can never complete; the kernel must give up after the (short)
limit, record CQ_ERR_TIMEOUT with the site of the first wait that gave up,
tear down (its other copies land, tensor memory is freed, whole warps leave
together) and leave the context usable: a normal call right after gives the
bits of one before."""
import pytest
import torch

pytestmark = pytest.mark.gpu

ERR_TIMEOUT = 4
STREAM, SPLIT, PAIR, SORTED = 1, 2, 3, 4
LIMIT = 20_000_000                   # 20 ms
STREAM_SITES = (54, 55)              # a slot of the ring that stays full, or empty
SECOND = 2                           # added by the layer's second launch
TC_SITES = (50, 51, 52, 53)


@pytest.fixture(scope="module")
def cq():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import bit_non_uniform_b200 as cq
    cq.lib()
    return cq


def codes(g, *shape):
    return torch.randint(-127, 128, shape, generator=g, device="cuda", dtype=torch.int8)


def stream():
    return torch.cuda.current_stream().cuda_stream


@pytest.mark.parametrize("codes_given", [True, False])
@pytest.mark.parametrize("path,M,N,K,swiglu", [
    (STREAM, 4, 2000, 4096, False),
    (STREAM, 6, 600, 16384, True),           # more units than the ring holds
    (SPLIT, 37, 1024, 4096, False),          # K over a cluster
    (SPLIT, 100, 514, 7168, True),
    (PAIR, 300, 1003, 2048, False),
    (PAIR, 1000, 2048, 1040, True),
])
def test_withheld_operands_of_a_product_time_out(cq, path, M, N, K, swiglu, codes_given):
    g = torch.Generator(device="cuda").manual_seed(M + N)
    x = torch.randn(M, K, generator=g, device="cuda").to(torch.bfloat16)
    wq, ws = codes(g, N, K), torch.rand(N, generator=g, device="cuda") / K
    epi = cq.EPI_SWIGLU if swiglu else cq.EPI_NONE
    xq, am = cq.cq_quant_rows(x)
    want = cq.cq_gemm_i8(xq, am, wq, ws, epilogue=epi)
    buf = torch.zeros(M * K + 4 * M + 4096, dtype=torch.uint8, device="cuda")
    y = torch.zeros_like(want)

    def call(limit, withhold):
        return cq.lib().cq_test_product_i8(
            (xq if codes_given else x).data_ptr(), am.data_ptr() if codes_given else None, M,
            wq.data_ptr(), ws.data_ptr(), N, K, epi, cq.F32, y.data_ptr(), buf.data_ptr(),
            buf.numel(), path, limit, withhold, stream())

    assert cq.device_error() == (0, 0)
    assert call(LIMIT, 1) == 0                              # the launch itself succeeds
    status, site = cq.device_error()                        # synchronises, reads, clears
    assert status == ERR_TIMEOUT
    assert site in (STREAM_SITES if path == STREAM else TC_SITES)
    assert cq.device_error() == (0, 0)
    # the same kernel, nothing withheld: every path gives the call's bits
    y.zero_()
    assert call(0, 0) == 0
    assert cq.device_error() == (0, 0)
    assert torch.equal(y, want)
    assert torch.equal(cq.cq_gemm_i8(xq, am, wq, ws, epilogue=epi), want)


def test_a_path_that_does_not_take_the_product_is_refused(cq):
    """8 rows of 16384 do not fit beside 12 units of the ring (6 do), and the
    streaming kernel takes 8 rows at most."""
    fake = 0x1000
    for M, K in ((8, 16384), (9, 512)):
        assert cq.lib().cq_test_product_i8(fake, fake, M, fake, fake, 600, K, 1, cq.F32, fake, None,
                                           0, STREAM, LIMIT, 1, stream()) == 2


def layer_call(cq, T, k, E, H, I, path):
    g = torch.Generator(device="cuda").manual_seed(T * H + I)
    x = torch.randn(T, H, generator=g, device="cuda").to(torch.bfloat16)
    ids = torch.rand(T, E, generator=g, device="cuda").topk(k, dim=1).indices.to(torch.int32)
    w = torch.rand(T, k, generator=g, device="cuda")
    lw = (codes(g, E, 2 * I, H), torch.rand(E, 2 * I, generator=g, device="cuda") / H,
          codes(g, E, H, I), torch.rand(E, H, generator=g, device="cuda") / I)
    n = cq.lib().cq_test_moe_i8_workspace_size(T, k, E, H, I, path)
    buf = torch.zeros(max(n, 256), dtype=torch.uint8, device="cuda")
    out = torch.zeros(T, H, device="cuda")

    def call(limit, withhold):
        return cq.lib().cq_test_moe_i8(
            x.data_ptr(), T, ids.data_ptr(), w.data_ptr(), k, E, *(t.data_ptr() for t in lw), H, I,
            cq.F32, None, out.data_ptr(), buf.data_ptr(), buf.numel(), path, limit, withhold,
            stream())

    return call, out, cq.cq_moe_i8(x, ids, w, *lw)[1]


@pytest.mark.parametrize("stage", [1, 2])
@pytest.mark.parametrize("path,T,k,E,H,I", [
    (STREAM, 3, 4, 6, 2064, 1040),
    (STREAM, 16, 2, 3, 4096, 272),           # two blocks of columns
    (STREAM, 40, 3, 50, 528, 400),           # more than 32 routes
    (SORTED, 300, 2, 5, 1040, 528),          # tiles of 128 routes
    (SORTED, 70, 2, 4, 2064, 1040),          # ... and of 64
])
def test_withheld_operands_of_a_layer_time_out(cq, path, T, k, E, H, I, stage):
    call, out, want = layer_call(cq, T, k, E, H, I, path)
    assert cq.device_error() == (0, 0)
    assert call(LIMIT, stage) == 0
    status, site = cq.device_error()
    assert status == ERR_TIMEOUT
    if path == STREAM:
        assert site in [s + SECOND * (stage - 1) for s in STREAM_SITES]
    else:
        assert site in TC_SITES
    assert cq.device_error() == (0, 0)
    out.zero_()
    assert call(0, 0) == 0
    assert cq.device_error() == (0, 0)
    assert torch.equal(out, want)


def test_the_second_launch_does_not_count_the_first_ones_time(cq):
    """One expert of 16 gate/up pairs keeps 16 CTAs busy, so that the down
    launch starts on the other SMs at once, fills its ring (28 units a CTA, more
    than fit) and waits.  The gate/up launch is held for 40 ms; the down
    launch's limit of 10 ms must not begin before that one has ended."""
    T, k, E, H, I = 1, 1, 1, 65536, 16
    call, out, want = layer_call(cq, T, k, E, H, I, STREAM)
    assert cq.device_error() == (0, 0)
    assert call(40_000_000, 1) == 0
    status, site = cq.device_error()
    assert status == ERR_TIMEOUT and site in STREAM_SITES
    assert call(0, 0) == 0
    assert cq.device_error() == (0, 0)
    assert torch.equal(out, want)
