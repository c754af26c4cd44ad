"""A stream of another device than the tensors' is refused (it would be dropped
silently: entering it makes its own device the current one).  A stand-in takes
the place of a second GPU."""
import pytest
import torch


class Stream:
    device = torch.device("cuda", 5)
    device_index = 5
    cuda_stream = 0


def test_another_devices_stream_is_refused_before_anything_is_entered():
    import bit_non_uniform_b200 as cq
    with pytest.raises(ValueError, match="stream is on cuda:5"):
        cq._on_device(0, Stream())


@pytest.mark.gpu
def test_calls_refuse_another_devices_stream():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import bit_non_uniform_b200 as cq
    x = torch.randn(2, 64, device="cuda").to(torch.bfloat16)
    wq, ws = torch.ones(32, 64, dtype=torch.int8, device="cuda"), torch.ones(32, device="cuda")
    xq, am = cq.cq_quant_rows(x)
    ids, w = cq.cq_moe_route(torch.randn(2, 3, device="cuda"), 1)
    lw = (torch.ones(3, 64, 64, dtype=torch.int8, device="cuda"), torch.ones(3, 64, device="cuda"),
          torch.ones(3, 64, 32, dtype=torch.int8, device="cuda"), torch.ones(3, 64, device="cuda"))
    s = Stream()
    for call in (lambda: cq.cq_linear_i8(x, wq, ws, stream=s),
                 lambda: cq.cq_gemm_i8(xq, am, wq, ws, stream=s),
                 lambda: cq.cq_moe_i8(x, ids, w, *lw, stream=s),
                 lambda: cq.cq_moe_route(torch.randn(2, 3, device="cuda"), 1, stream=s)):
        with pytest.raises(ValueError, match="stream is on cuda:5"):
            call()
