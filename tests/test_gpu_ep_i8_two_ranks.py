"""Expert parallelism of an INT8 layer with cq_moe_i8 as every rank's expert
compute: two ranks (processes) over gloo, both on cuda:0.

The exchange runs on the host; each rank's expert compute copies the rows it
received to the GPU, runs cq_moe_i8 over its own block of experts (ids of the
other rank are -1) and copies the combined partial rows back.  No kernel waits
on another process.  A route's output does not depend on the call it is in, so
each rank's rows are the weighted sums of the single-process layer's routes;
only the order of at most k + 1 FP32 additions differs.
"""
import os
import socket

import pytest
import torch
import torch.multiprocessing as mp

pytestmark = pytest.mark.gpu

H, I, E, K_TOP = 512, 208, 8, 4
U = 2.0 ** -24


def _layer():
    g = torch.Generator().manual_seed(11)
    return (torch.randint(-127, 128, (E, 2 * I, H), generator=g, dtype=torch.int8),
            (0.5 + torch.rand(E, 2 * I, generator=g)) / (73 * H ** 0.5),
            torch.randint(-127, 128, (E, H, I), generator=g, dtype=torch.int8),
            (0.5 + torch.rand(E, H, generator=g)) / (73 * I ** 0.5))


def _inputs(rank, T):
    """This rank's tokens, ids and weights; rank 1 also drops a route and has a
    token whose routes all land on one rank and one without routes."""
    g = torch.Generator().manual_seed(20 + rank)
    x = torch.randn(T, H, generator=g).to(torch.bfloat16)
    ids = torch.rand(T, E, generator=g).topk(K_TOP, dim=1).indices.to(torch.int32)
    w = torch.rand(T, K_TOP, generator=g)
    if rank == 1 and T >= 3:
        ids[0, 1] = -1
        ids[1] = torch.tensor([4, 5, 6, 7], dtype=torch.int32)
        ids[2] = -1
    return x, ids, w


def _free_port():
    with socket.socket() as s:
        s.bind(("127.0.0.1", 0))
        return s.getsockname()[1]


def _rank_main(rank, world, port, tokens_per_rank, q):
    import datetime
    import torch.distributed as dist
    os.environ.update(MASTER_ADDR="127.0.0.1", MASTER_PORT=str(port),
                      RANK=str(rank), WORLD_SIZE=str(world))
    dist.init_process_group("gloo", rank=rank, world_size=world,
                            timeout=datetime.timedelta(seconds=120))
    try:
        import bit_non_uniform_b200 as cq
        from bit_non_uniform_b200.ep import MoeExpertParallel, experts_per_rank, libcq_i8_compute
        torch.cuda.set_device(0)
        el = experts_per_rank(E, world)
        on_gpu = libcq_i8_compute(*(t[rank * el:(rank + 1) * el].cuda() for t in _layer()))

        def compute(tokens, ids, w):          # host rows in, host partial rows out
            return on_gpu(tokens.cuda(), ids.cuda(), w.cuda()).cpu()

        layer = MoeExpertParallel(E, H, compute)
        got = layer.forward(*_inputs(rank, tokens_per_rank[rank])).numpy()
        torch.cuda.synchronize()
        q.put((rank, got, cq.device_error()))
    finally:
        dist.destroy_process_group()


@pytest.mark.parametrize("tokens_per_rank", [(5, 6), (0, 4), (40, 33)])
def test_two_ranks_give_the_layers_sums(tokens_per_rank):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import bit_non_uniform_b200 as cq
    world = 2
    ctx = mp.get_context("spawn")
    q = ctx.Queue()
    port = _free_port()
    procs = [ctx.Process(target=_rank_main, args=(r, world, port, tokens_per_rank, q))
             for r in range(world)]
    for p in procs:
        p.start()
    # read before joining: a rank ends only once its rows have gone through the pipe
    results = sorted((q.get(timeout=200) for _ in range(world)), key=lambda r: r[0])
    for p in procs:
        p.join(60)
    exits = [p.exitcode for p in procs]
    for p in procs:
        if p.is_alive():
            p.kill()
    assert exits == [0, 0], exits
    lw = [t.cuda() for t in _layer()]
    for rank, got, dev_err in results:
        T = tokens_per_rank[rank]
        assert got.shape == (T, H) and dev_err == (0, 0)
        if T == 0:
            continue
        x, ids, w = _inputs(rank, T)
        ro, _ = cq.cq_moe_i8(x.cuda(), ids.cuda(), w.cuda(), *lw)
        terms = ro.cpu().double().view(T, K_TOP, H) * w.double()[:, :, None]
        # an FP32 multiply-add per route, and the sum of the two ranks' partials
        tol = (K_TOP + 2) * 1.01 * U * terms.abs().sum(dim=1)
        err = (torch.from_numpy(got).double() - terms.sum(dim=1)).abs()
        assert bool((err <= tol).all()), (rank, float((err - tol).max()))
