"""GPU parity of the INT8 operators (cq_gemm_i8, cq_linear_i8, cq_moe_i8) and
of the MoE router (cq_moe_route) against plain FP64 forms of their
definitions.

Bars.  The integer sums are exact, so a product carries the roundings of its
scaling only: RN(RN(sx ws) RN(acc)) is within 3 half steps of 2^-24 (relative)
of the value; SwiGLU adds expf (2 units in the last place), an add, a division
and two products, and carries the errors of g and u through silu, whose
relative condition number is at most 1 + |g|; BF16 output adds half a step,
2^-8.  The MoE layer's codes are decided from FP64 values and equal the
reference's; a route carries the 3 half steps and the weighted sum one product
and one add per route.  A router's ids are equal; its weights are FP64 values
rounded once, except for the FP32 softmax sum (at most 31 adds per lane, expf,
a rounded difference)."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu
U = 2.0 ** -24                       # half a step of FP32
UB = 2.0 ** -8                       # half a step of BF16


@pytest.fixture(scope="module")
def cq():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import bit_non_uniform_b200 as cq
    cq.lib()
    return cq


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def tokens(g, M, K):
    return (torch.randn(M, K, generator=g, device="cuda") * 1.7).to(torch.bfloat16)


def codes(g, *shape):
    return torch.randint(-127, 128, shape, generator=g, device="cuda", dtype=torch.int8)


def scales(g, *shape, K):
    return (0.5 + torch.rand(*shape, generator=g, device="cuda")) / (73.0 * K ** 0.5)


def quant_ref(v):
    """Codes and maxima of FP32 rows, decided in FP32 (numpy divides and rounds to nearest even)."""
    a = v.detach().cpu().to(torch.float32).numpy()
    top = np.abs(a).max(axis=1)
    with np.errstate(divide="ignore"):
        inv = np.where(top > 0, np.float32(127.0) / top, np.float32(0)).astype(np.float32)
    q = np.clip(np.rint((a * inv[:, None]).astype(np.float32)), -127, 127)
    return torch.from_numpy(q).double().cuda(), torch.from_numpy(top).cuda()


def sx_of(absmax):
    """RN(absmax / 127) as FP64."""
    q = (absmax.cpu().numpy() / np.float32(127.0)).astype(np.float32)
    return torch.from_numpy(q).double().cuda()


def product_ref(xq, absmax, wq, ws):
    return (xq.double() @ wq.double().t()) * sx_of(absmax)[:, None] * ws.double()[None, :]


def silu_ref(v):
    return v * torch.sigmoid(v)


def check_product(y, ref, swiglu, bf16):
    if swiglu:
        g, u = ref.chunk(2, dim=1)
        ref = silu_ref(g) * u
        tol = (3 * (1 + g.abs()) + 3 + 4 + 1 + 1 + 2) * 1.01 * U * ref.abs() + 1e-30
    else:
        tol = 3.01 * U * ref.abs()
    if bf16:
        tol = tol + 1.01 * UB * ref.abs()
    err = (y.double() - ref).abs()
    assert y.shape == ref.shape
    assert bool((err <= tol).all()), float((err - tol).max())


PRODUCTS = [
    # M,    N,    K,    swiglu, bf16
    (1,     1,    16,   False, False),
    (1,     1000, 512,  False, True),
    (1,     770,  7168, True,  True),
    (2,     7,    48,   False, False),
    (8,     334,  272,  True,  False),
    (9,     333,  4096, False, False),
    (16,    50,   2064, True,  False),
    (16,    6144, 1040, False, True),
    (17,    129,  144,  False, False),
    (33,    2,    1008, True,  False),
    (64,    1024, 512,  True,  True),
    (100,   517,  1552, False, False),
    (129,   260,  4112, True,  False),
    (256,   256,  128,  False, True),
    (300,   1003, 2048, False, False),
    (1025,  514,  784,  True,  True),
    (2049,  1281, 96,   False, False),
    (16,  300,  8208, False, False),       # long rows
    (11,  40,   14000, True, False),
    (2,   100,  99984, False, False),
]


@pytest.mark.parametrize("M,N,K,swiglu,bf16", PRODUCTS)
def test_products_match_fp64(cq, M, N, K, swiglu, bf16):
    g = gen(M * 7 + N)
    x, wq, ws = tokens(g, M, K), codes(g, N, K), scales(g, N, K=K)
    epi = cq.EPI_SWIGLU if swiglu else cq.EPI_NONE
    dt = cq.BF16 if bf16 else cq.F32
    y = cq.cq_linear_i8(x, wq, ws, epilogue=epi, out_dtype=dt)
    xq, am = cq.cq_quant_rows(x)
    rq, ra = quant_ref(x)
    assert torch.equal(xq.double(), rq) and torch.equal(am, ra)
    check_product(y, product_ref(xq, am, wq, ws), swiglu, bf16)
    # rows quantized before give the same bits, and so does a second call on a kept workspace
    wsp = cq.gemm_i8_workspace(M, N, K, epi)
    for _ in range(2):
        z = cq.cq_gemm_i8(xq, am, wq, ws, epilogue=epi, out_dtype=dt, workspace=wsp)
        assert torch.equal(z, y)
    assert cq.device_error() == (0, 0)


@pytest.mark.parametrize("M", [1, 16, 40, 200])
def test_largest_sums_are_exact(cq, M):
    """K = 131072 with every code at the end of its range: the sums reach
    +-127^2 K = +-2,114,060,288 and stay exact in INT32."""
    K, N = 131072, 130
    xq = torch.full((M, K), 127, dtype=torch.int8, device="cuda")
    wq = torch.full((N, K), 127, dtype=torch.int8, device="cuda")
    wq[1::2] = -127
    wq[2, ::2] = -127
    am = torch.full((M,), 127.0, device="cuda")
    y = cq.cq_gemm_i8(xq, am, wq, torch.ones(N, device="cuda"))
    ref = (127.0 * 127.0 * K) * torch.ones(N, dtype=torch.float64, device="cuda")
    ref[1::2] *= -1
    ref[2] = 0.0
    assert torch.equal(y.double(), ref.float().double().expand(M, N))


@pytest.mark.parametrize("M", [3, 70])
def test_code_minus_128_counts_as_such(cq, M):
    g = gen(4)
    N, K = 66, 512
    xq = torch.randint(-128, 128, (M, K), generator=g, device="cuda", dtype=torch.int8)
    wq = torch.randint(-128, 128, (N, K), generator=g, device="cuda", dtype=torch.int8)
    am, ws = torch.full((M,), 127.0, device="cuda"), torch.ones(N, device="cuda")
    y = cq.cq_gemm_i8(xq, am, wq, ws)
    assert torch.equal(y.double(), xq.double() @ wq.double().t())


@pytest.mark.parametrize("M", [4, 50])
def test_zero_infinite_and_nan_rows(cq, M):
    g = gen(5)
    N, K = 96, 256
    x, wq, ws = tokens(g, M, K), codes(g, N, K), scales(g, N, K=K)
    x[0] = 0.0
    x[1, 3] = float("inf")
    x[2, 5] = float("nan")
    y = cq.cq_linear_i8(x, wq, ws)
    assert bool((y[0] == 0).all())
    assert not bool(torch.isfinite(y[1]).any())
    z = x[2:].clone()
    z[0, 5] = 0.0                                # a NaN activation has code 0
    assert torch.equal(y[2:], cq.cq_linear_i8(z, wq, ws))
    assert bool(torch.isfinite(y[2:]).all())


@pytest.mark.parametrize("M", [0, 5])
def test_empty_products(cq, M):
    x = torch.zeros((M, 64), dtype=torch.bfloat16, device="cuda")
    wq = torch.zeros((0, 64), dtype=torch.int8, device="cuda")
    y = cq.cq_linear_i8(x, wq, torch.zeros(0, device="cuda"))
    assert y.shape == (M, 0)
    y = cq.cq_linear_i8(x[:0], torch.zeros((8, 64), dtype=torch.int8, device="cuda"),
                        torch.zeros(8, device="cuda"))
    assert y.shape == (0, 8)


# ---------------------------------------------------------------------------
# the MoE layer
# ---------------------------------------------------------------------------

def layer(g, E, H, I):
    return (codes(g, E, 2 * I, H), scales(g, E, 2 * I, K=H), codes(g, E, H, I),
            scales(g, E, H, K=I))


def moe_ref(x, ids, w, w_gu, s_gu, w_dn, s_dn):
    """Per-route outputs, their weighted sum and the sum of its magnitudes, in FP64."""
    T, k = ids.shape
    E, H, I = w_dn.shape
    xq, am = quant_ref(x)
    routes = torch.zeros(T * k, H, dtype=torch.float64, device="cuda")
    flat = ids.reshape(-1).tolist()
    for e in sorted(set(v for v in flat if 0 <= v < E)):
        rs = [r for r, v in enumerate(flat) if v == e]
        ts = [r // k for r in rs]
        gu = (xq[ts] @ w_gu[e].double().t()) * (sx_of(am)[ts][:, None] * s_gu[e].double()[None])
        h = (silu_ref(gu[:, :I]) * gu[:, I:]).float()
        hq, hm = quant_ref(h)
        routes[rs] = product_ref(hq, hm, w_dn[e], s_dn[e])
    terms = routes.view(T, k, H) * w.double()[:, :, None]
    live = ((ids >= 0) & (ids < E))[:, :, None]
    terms = torch.where(live, terms, torch.zeros_like(terms))
    return routes, terms.sum(dim=1), terms.abs().sum(dim=1)


def distinct_ids(g, T, E, k):
    return torch.rand(T, E, generator=g, device="cuda").topk(k, dim=1).indices.to(torch.int32)


def check_moe(ro, out, ref, k, bf16):
    routes, total, mag = ref
    if ro is not None:
        assert bool(((ro.double() - routes).abs() <= 3.01 * U * routes.abs()).all())
    if out is not None:
        tol = (3 + 2 * k) * 1.01 * U * mag
        if bf16:
            tol = tol + 1.01 * UB * total.abs()
        err = (out.double() - total).abs()
        assert bool((err <= tol).all()), float((err - tol).max())


MOE = [
    # T,  k, E,  H,    I,   dropped, bf16
    (1,   2, 8,  512,  256, 0.0, False),
    (1,   1, 1,  16,   16,  0.0, False),
    (3,   4, 6,  2064, 48,  0.0, True),
    (5,   6, 40, 272,  1040, 0.4, False),
    (8,   8, 16, 1024, 144, 0.0, False),
    (16,  4, 5,  528,  272, 0.2, True),
    (40,  2, 2,  160,  96,  0.0, False),
    (300, 5, 7,  48,   32,  0.1, False),
    (2,   3, 3,  16,   4096, 0.0, False),
    (20,  1, 1,  16400, 32, 0.0, False),      # long rows
    (16,  4, 5,  7168, 48,  0.0, False),
    (14,  3, 4,  64,   8208, 0.3, False),
    (9,   2, 3,  9216, 9232, 0.0, True),
    (16,  1, 1,  16400, 32, 0.0, False),
    (9,   1, 2,  9216, 9232, 0.0, False),
]


@pytest.mark.parametrize("T,k,E,H,I,dropped,bf16", MOE)
def test_moe_matches_fp64(cq, T, k, E, H, I, dropped, bf16):
    g = gen(T * 31 + H)
    x, lw = tokens(g, T, H), layer(g, E, H, I)
    ids = distinct_ids(g, T, E, k)
    if dropped:
        gone = torch.rand(T, k, generator=g, device="cuda") < dropped
        ids = torch.where(gone, torch.where(gone.cumsum(1) % 2 == 0, -1, E).to(torch.int32), ids)
    w = torch.randn(T, k, generator=g, device="cuda")
    w[ids < 0] = float("nan")                    # weights of dropped routes are not read
    ws = cq.moe_i8_workspace(T, k, E, H, I)
    dt = cq.BF16 if bf16 else cq.F32
    ro, out = cq.cq_moe_i8(x, ids, w, *lw, out_dtype=dt, workspace=ws)
    check_moe(ro, out, moe_ref(x, ids, torch.nan_to_num(w), *lw), k, bf16)
    # without the per-route output, and on the kept workspace: the same bits
    for _ in range(2):
        none, again = cq.cq_moe_i8(x, ids, w, *lw, out_dtype=dt, route_out=False, workspace=ws)
        assert none is None and torch.equal(again, out)
    only, none = cq.cq_moe_i8(x, ids, None, *lw, combine=False, workspace=ws)
    assert none is None and torch.equal(only, ro)
    assert cq.device_error() == (0, 0)


# more than 16 routes per expert: the tensor cores, with tiles of 64 and 128
# routes
MOE_MANY = [
    (33,   1, 2,  16,   16,  0.0, False),      # one 16-byte block of K each
    (100,  2, 5,  528,  272, 0.2, True),       # up to 64 routes a tile
    (101,  3, 3,  400,  144, 0.0, False),      # 101 routes: one tile, not full
    (257,  2, 2,  272,  80,  0.3, False),      # several tiles of an expert
    (129,  1, 4,  4112, 48,  0.0, True),       # rows longer than a thread keeps
    (40,   2, 2,  64,   8208, 0.0, False),
    (700,  2, 70, 64,   64,  0.5, False),      # many experts, tiles nearly empty
    (4200, 4, 40, 32,   16,  0.1, False),      # more routes than one launch takes
]


@pytest.mark.parametrize("T,k,E,H,I,dropped,bf16", MOE_MANY)
def test_moe_many_routes_match_fp64(cq, T, k, E, H, I, dropped, bf16):
    assert T * k > 16 * E
    test_moe_matches_fp64(cq, T, k, E, H, I, dropped, bf16)


@pytest.mark.parametrize("T", [30, 80, 200])
def test_moe_many_routes_give_the_bits_of_a_few(cq, T):
    """A token's outputs do not depend on how many others share the call; all
    to one expert, dropped routes between, other experts empty."""
    g = gen(T)
    k, E, H, I = 2, 3, 640, 208
    x, lw = tokens(g, T, H), layer(g, E, H, I)
    ids = torch.full((T, k), 1, dtype=torch.int32, device="cuda")
    ids[::3, 0] = -1
    ids[::7] = E
    w = torch.randn(T, k, generator=g, device="cuda")
    ro, out = cq.cq_moe_i8(x, ids, w, *lw)
    for t in range(0, T, 9):
        few = cq.cq_moe_i8(x[t:t + 9].contiguous(), ids[t:t + 9].contiguous(),
                           w[t:t + 9].contiguous(), *lw)
        assert torch.equal(few[0], ro[t * k:(t + 9) * k]) and torch.equal(few[1], out[t:t + 9])
    assert bool((ro.view(T, k, H)[::7] == 0).all()) and bool((out[::7] == 0).all())
    ids.fill_(-1)
    ro, out = cq.cq_moe_i8(x, ids, w, *lw)
    assert bool((ro == 0).all()) and bool((out == 0).all())
    assert cq.device_error() == (0, 0)


def test_moe_many_routes_hide_no_overflow(cq):
    g = gen(21)
    T, k, E, H, I = 60, 2, 4, 512, 64
    x, lw = tokens(g, T, H), layer(g, E, H, I)
    ids, w = distinct_ids(g, T, E, k), torch.ones(T, k, device="cuda")
    clean = cq.cq_moe_i8(x, ids, w, *lw)[0]
    for bad_row in (torch.full((H,), float("inf"), device="cuda"), x[1].float() * 1e30):
        bad = x.clone()
        bad[1] = bad_row.to(torch.bfloat16)
        ro, out = cq.cq_moe_i8(bad, ids, w, *lw)
        assert not bool(torch.isfinite(ro[k:2 * k]).any())
        assert torch.equal(ro[:k], clean[:k]) and torch.equal(ro[2 * k:], clean[2 * k:])


def test_moe_many_routes_captured_and_on_another_stream(cq):
    g = gen(22)
    T, k, E, H, I = 70, 2, 3, 256, 96
    lw = layer(g, E, H, I)
    xs = [tokens(g, T, H) for _ in range(2)]
    ids = [distinct_ids(g, T, E, k) for _ in range(2)]
    w = torch.rand(T, k, generator=g, device="cuda")
    want = [cq.cq_moe_i8(xs[i], ids[i], w, *lw, route_out=False)[1] for i in range(2)]
    ws = cq.moe_i8_workspace(T, k, E, H, I)
    x, i = xs[0].clone(), ids[0].clone()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        out = cq.cq_moe_i8(x, i, w, *lw, route_out=False, workspace=ws)[1]
        twice = cq.cq_moe_i8(x, i, w, *lw, route_out=False, workspace=ws)[1]
    for n in (0, 1, 0):
        x.copy_(xs[n])
        i.copy_(ids[n])
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want[n]) and torch.equal(twice, want[n])
    with torch.cuda.stream(s):
        other = cq.cq_moe_i8(xs[1], ids[1], w, *lw, route_out=False)[1]
    s.synchronize()
    assert torch.equal(other, want[1])


def test_moe_all_routes_dropped(cq):
    g = gen(8)
    T, k, E, H, I = 3, 4, 5, 512, 64
    x, lw = tokens(g, T, H), layer(g, E, H, I)
    ids = torch.full((T, k), -1, dtype=torch.int32, device="cuda")
    w = torch.ones(T, k, device="cuda")
    ws = cq.moe_i8_workspace(T, k, E, H, I)
    ro = torch.full((T * k, H), 7.0, device="cuda")
    for dt in (cq.F32, cq.BF16):
        _, out = cq.cq_moe_i8(x, ids, w, *lw, out_dtype=dt, route_out=ro, workspace=ws)
        assert bool((out == 0).all()) and bool((ro == 0).all())
    ids[1, 2] = 4
    ro, out = cq.cq_moe_i8(x, ids, w, *lw, workspace=ws)
    check_moe(ro, out, moe_ref(x, ids, w, *lw), k, False)
    assert bool((out[0] == 0).all()) and bool((out[2] == 0).all())


@pytest.mark.parametrize("T", [2, 12])
def test_moe_infinite_token_and_overflow_are_not_hidden(cq, T):
    """An infinite activation, or gate and up values whose product overflows
    FP32, leave outputs that are not finite; other tokens keep their bits."""
    g = gen(13)
    k, E, H, I = 2, 4, 512, 64
    x, lw = tokens(g, T, H), layer(g, E, H, I)
    ids, w = distinct_ids(g, T, E, k), torch.ones(T, k, device="cuda")
    clean = cq.cq_moe_i8(x, ids, w, *lw)[0]
    bad = x.clone()
    bad[1, 7] = float("inf")
    ro, out = cq.cq_moe_i8(bad, ids, w, *lw)
    assert not bool(torch.isfinite(ro[k:2 * k]).any()) and not bool(torch.isfinite(out[1]).any())
    assert torch.equal(ro[:k], clean[:k]) and torch.equal(ro[2 * k:], clean[2 * k:])
    bad = x.clone()
    bad[1] = (x[1].float() * 1e30).to(torch.bfloat16)          # g and u near 1e30
    ro, out = cq.cq_moe_i8(bad, ids, w, *lw)
    assert not bool(torch.isfinite(ro[k:2 * k]).any())
    assert torch.equal(ro[:k], clean[:k])


def test_moe_the_same_expert_twice(cq):
    g = gen(9)
    T, k, E, H, I = 12, 3, 4, 256, 96
    x, lw = tokens(g, T, H), layer(g, E, H, I)
    ids = torch.full((T, k), 2, dtype=torch.int32, device="cuda")
    w = torch.rand(T, k, generator=g, device="cuda")
    ro, out = cq.cq_moe_i8(x, ids, w, *lw)
    check_moe(ro, out, moe_ref(x, ids, w, *lw), k, False)


def test_moe_no_tokens(cq):
    g = gen(10)
    lw = layer(g, 2, 64, 32)
    ro, out = cq.cq_moe_i8(tokens(g, 0, 64), torch.zeros((0, 2), dtype=torch.int32, device="cuda"),
                           torch.zeros((0, 2), device="cuda"), *lw)
    assert ro.shape == (0, 64) and out.shape == (0, 64)


def test_moe_matches_the_products_it_is_made_of(cq):
    """One route: the layer's gate/up codes and sums are those of
    cq_linear_i8, and its down product is cq_gemm_i8 on the codes of h."""
    g = gen(11)
    E, H, I = 3, 768, 160
    x, (w_gu, s_gu, w_dn, s_dn) = tokens(g, 1, H), layer(g, E, H, I)
    ids = torch.tensor([[1]], dtype=torch.int32, device="cuda")
    ro, _ = cq.cq_moe_i8(x, ids, torch.ones(1, 1, device="cuda"), w_gu, s_gu, w_dn, s_dn)
    gu = cq.cq_linear_i8(x, w_gu[1], s_gu[1]).double()
    h = (silu_ref(gu[:, :I]) * gu[:, I:]).float()
    hq, hm = quant_ref(h)
    y = cq.cq_gemm_i8(hq.to(torch.int8), hm, w_dn[1], s_dn[1])
    # FP32 g and u move a few values of h by an FP32 step; a code that flips moves y by hm/127 ws 127
    tol = 2 * float(hm) * float(s_dn[1].max())
    assert float((ro - y).abs().max()) <= tol


# ---------------------------------------------------------------------------
# the router
# ---------------------------------------------------------------------------

def route_ref(logits, k, bias, sigmoid, renorm, scale):
    l = logits.double()
    live = ~(torch.isnan(l) | torch.isneginf(l))
    if sigmoid:
        score = 1.0 / (1.0 + torch.exp(-l))
    else:
        top = torch.where(live, l, torch.full_like(l, -np.inf)).amax(dim=1, keepdim=True)
        e = torch.where(l == top, torch.ones_like(l), torch.exp(l - top))
        e = torch.where(live, e, torch.zeros_like(e))
        score = e / e.sum(dim=1, keepdim=True)
    pick = l if bias is None else score + bias.double()
    live = live & ~torch.isnan(pick) & ~torch.isneginf(pick)
    pick = torch.where(live, pick, torch.full_like(pick, -np.inf))
    order = torch.sort(pick, dim=1, descending=True, stable=True).indices[:, :k]
    ok = torch.gather(live, 1, order)
    w = torch.where(ok, torch.gather(score, 1, order), torch.zeros_like(score[:, :k]))
    if renorm:
        s = w.sum(dim=1, keepdim=True)
        w = torch.where(s > 0, w / s, torch.zeros_like(w))
    return torch.where(ok, order, torch.full_like(order, -1)).to(torch.int32), w * scale


def check_route(cq, logits, k, bias, sigmoid, renorm, scale=1.0):
    scoring = cq.SCORE_SIGMOID if sigmoid else cq.SCORE_SOFTMAX
    ids, w = cq.cq_moe_route(logits, k, bias=bias, scoring=scoring, renorm=renorm, scale=scale)
    ri, rw = route_ref(logits, k, bias, sigmoid, renorm, scale)
    assert torch.equal(ids, ri)
    # FP64 values rounded once; the plain softmax divides by an FP32 sum: expf and its rounded
    # argument (at most 20 half steps while the sum's terms lie within 16 of the top), 31 adds
    tol = (1.01 if sigmoid or renorm or bias is not None else 64) * U
    assert bool(((w.double() - rw).abs() <= tol * rw.abs() + 1e-45).all())
    return ids, w


ROUTES = [
    # T,   E,    k
    (1,    896,  16),
    (5,    8,    2),
    (1,    1,    1),
    (7,    33,   33 - 1),
    (64,   128,  6),
    (65,   129,  8),
    (130,  512,  32),
    (33,   1024, 32),
    (1000, 700,  1),
]


@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("T,E,k", ROUTES)
def test_route_matches_fp64(cq, T, E, k, sigmoid, bias):
    for bf16 in (False, True):
        g = gen(T + E)
        logits = torch.randn(T, E, generator=g, device="cuda") * 1.5
        logits = logits.to(torch.bfloat16) if bf16 else logits
        b = torch.randn(E, generator=g, device="cuda") * 0.1 if bias else None
        for renorm in (False, True):
            check_route(cq, logits, k, b, sigmoid, renorm, 2.5)


@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("sigmoid", [False, True])
def test_route_masks(cq, sigmoid, bias):
    g = gen(3)
    E, k = 200, 8
    b = torch.randn(E, generator=g, device="cuda") * 0.1 if bias else None
    logits = torch.randn(9, E, generator=g, device="cuda")
    logits[0] = float("-inf")                               # nothing left
    logits[1, 5:] = float("-inf")                           # fewer than k left
    logits[2, 3:] = torch.finfo(torch.float32).min          # the type's lowest value
    logits[3] = torch.finfo(torch.float32).min
    logits[4, ::2] = float("nan")
    logits[5] = 0.25                                        # all equal: the lowest ids
    logits[6, 17] = float("inf")
    logits[7, ::3] = logits[7, 0].item()                    # many ties
    for renorm in (False, True):
        ids, w = check_route(cq, logits, k, b, sigmoid, renorm)
        assert ids[0].tolist() == [-1] * k and w[0].tolist() == [0.0] * k
        assert sorted(ids[1].tolist())[:3] == [-1] * 3
        if not bias:
            assert ids[5].tolist() == list(range(k))


@pytest.mark.parametrize("E,k", [(1024, 32), (896, 16), (300, 5)])
def test_route_more_equal_picks_than_are_ranked_at_once(cq, E, k):
    logits = torch.full((3, E), -1.0, device="cuda")
    logits[1, E // 2:] = 2.0
    bias = torch.zeros(E, device="cuda")
    bias[::7] = 1e-9
    for b in (None, bias):
        for sigmoid in (False, True):
            check_route(cq, logits, k, b, sigmoid, True)


def test_route_picks_closer_than_fp32_resolves(cq):
    """Scores that differ below FP32's resolution are ordered as in FP64."""
    E = 256
    logits = torch.zeros(1, E, device="cuda")
    logits[0] = torch.arange(E, device="cuda") * 1e-7 + 0.5
    bias = torch.zeros(E, device="cuda")
    for sigmoid in (False, True):
        ids, _ = check_route(cq, logits, 12, bias, sigmoid, True)
        assert ids[0, 0].item() == E - 1
    bias = -torch.arange(E, device="cuda").float() * 1e-8
    check_route(cq, logits, 12, bias, True, True)


def test_route_extreme_biases(cq):
    g = gen(6)
    E, k = 100, 6
    logits = torch.randn(4, E, generator=g, device="cuda")
    for values in ([float("inf"), float("-inf"), float("nan")], [3e38, -3e38, 1e6],
                   [-3.4e38, 3.4e38, 0.0]):
        bias = torch.zeros(E, device="cuda")
        bias[11], bias[12], bias[13] = values
        check_route(cq, logits, k, bias, True, True)
        check_route(cq, logits, k, bias, False, False)
    check_route(cq, logits, k, torch.full((E,), float("-inf"), device="cuda"), True, True)


def test_route_no_tokens(cq):
    ids, w = cq.cq_moe_route(torch.zeros((0, 8), device="cuda"), 2)
    assert ids.shape == (0, 2) and w.shape == (0, 2)


# ---------------------------------------------------------------------------
# together, on streams and in graphs
# ---------------------------------------------------------------------------

def moe_block(cq, x, w_router, lw, shared, k, bufs):
    """A decode step's MoE block: router, routed experts, a shared expert."""
    logits = x.float() @ w_router.t()
    ids, w = cq.cq_moe_route(logits, k, scoring=cq.SCORE_SIGMOID, scale=2.5)
    _, routed = cq.cq_moe_i8(x, ids, w, *lw, route_out=False, workspace=bufs["moe"])
    s_gu, c_gu, s_dn, c_dn = shared
    h = cq.cq_linear_i8(x, s_gu, c_gu, epilogue=cq.EPI_SWIGLU, out_dtype=cq.BF16,
                        workspace=bufs["gu"])
    y = cq.cq_linear_i8(h, s_dn, c_dn, workspace=bufs["dn"])
    return routed + y, ids, w, logits, routed, h, y


def block_inputs(cq, seed, T, H, I, E, k):
    g = gen(seed)
    x = tokens(g, T, H)
    w_router = torch.randn(E, H, generator=g, device="cuda") / H ** 0.5
    lw = layer(g, E, H, I)
    shared = (codes(g, 2 * I, H), scales(g, 2 * I, K=H), codes(g, H, I), scales(g, H, K=I))
    bufs = dict(moe=cq.moe_i8_workspace(T, k, E, H, I),
                gu=cq.gemm_i8_workspace(T, 2 * I, H, cq.EPI_SWIGLU),
                dn=cq.gemm_i8_workspace(T, H, I))
    return x, w_router, lw, shared, bufs


@pytest.mark.parametrize("T", [1, 6, 48])
def test_router_experts_and_shared_expert_together(cq, T):
    H, I, E, k = 1024, 208, 24, 4
    x, w_router, lw, shared, bufs = block_inputs(cq, 20 + T, T, H, I, E, k)
    total, ids, w, logits, routed, h, y = moe_block(cq, x, w_router, lw, shared, k, bufs)
    ri, rw = route_ref(logits, k, None, True, True, 2.5)
    assert torch.equal(ids, ri)
    assert bool(((w.double() - rw).abs() <= 1.01 * U * rw.abs()).all())
    check_moe(None, routed, moe_ref(x, ids, w, *lw), k, False)
    xq, am = cq.cq_quant_rows(x)
    check_product(h, product_ref(xq, am, shared[0], shared[1]), True, True)
    hq, hm = cq.cq_quant_rows(h)
    check_product(y, product_ref(hq, hm, shared[2], shared[3]), False, False)
    assert torch.equal(total, routed + y)


@pytest.mark.parametrize("T", [2, 48])
def test_captured_block_replays_on_new_inputs(cq, T):
    """Two graphs that share the workspaces, replayed in turn with new inputs,
    give the bits of eager calls."""
    H, I, E, k = 512, 144, 12, 3
    x, w_router, lw, shared, bufs = block_inputs(cq, 30, T, H, I, E, k)
    x2 = x.clone()
    moe_block(cq, x, w_router, lw, shared, k, bufs)                  # warm-up
    graphs = []
    side = torch.cuda.Stream()
    for inp in (x, x2):
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr, stream=side):
            out = moe_block(cq, inp, w_router, lw, shared, k, bufs)
        graphs.append((gr, inp, out))
    for turn in range(4):
        gr, inp, out = graphs[turn % 2]
        inp.copy_(tokens(gen(40 + turn), T, H))
        gr.replay()
        gr.replay()
        got = [t.clone() for t in out]
        want = moe_block(cq, inp, w_router, lw, shared, k, bufs)
        for a, b in zip(got, want):
            assert torch.equal(a, b)
    assert cq.device_error() == (0, 0)


@pytest.mark.parametrize("T", [3, 100])
def test_calls_on_another_stream(cq, T):
    """`stream` orders a call (its own buffers included) on that stream."""
    g = gen(50)
    H, I, E, k = 512, 96, 6, 2
    x, lw = tokens(g, T, H), layer(g, E, H, I)
    logits = torch.randn(T, E, generator=g, device="cuda")
    wq, ws = codes(g, 300, H), scales(g, 300, K=H)
    ids, w = cq.cq_moe_route(logits, k)
    _, out = cq.cq_moe_i8(x, ids, w, *lw)
    y = cq.cq_linear_i8(x, wq, ws)
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    with torch.cuda.stream(st):
        torch.cuda._sleep(2_000_000)
    i2, w2 = cq.cq_moe_route(logits, k, stream=st)
    _, o2 = cq.cq_moe_i8(x, i2, w2, *lw, stream=st)
    y2 = cq.cq_linear_i8(x, wq, ws, stream=st)
    st.synchronize()
    assert torch.equal(i2, ids) and torch.equal(w2, w)
    assert torch.equal(o2, out) and torch.equal(y2, y)


def test_two_streams_at_once(cq):
    """Calls with their own workspaces may overlap."""
    g = gen(60)
    T, H, I, E, k = 8, 1024, 256, 16, 4
    x, lw = tokens(g, T, H), layer(g, E, H, I)
    ids, w = distinct_ids(g, T, E, k), torch.rand(T, k, generator=g, device="cuda")
    wq, ws = codes(g, 1000, H), scales(g, 1000, K=H)
    xm = tokens(g, 90, H)
    want = cq.cq_moe_i8(x, ids, w, *lw)[1]
    y = cq.cq_linear_i8(xm, wq, ws)
    streams = [torch.cuda.Stream() for _ in range(2)]
    moe_ws = [cq.moe_i8_workspace(T, k, E, H, I) for _ in streams]
    lin_ws = [cq.gemm_i8_workspace(90, 1000, H) for _ in streams]
    torch.cuda.synchronize()
    got = []
    for _ in range(20):
        for s, mw, lw_ in zip(streams, moe_ws, lin_ws):
            got.append((cq.cq_moe_i8(x, ids, w, *lw, route_out=False, workspace=mw, stream=s)[1],
                        cq.cq_linear_i8(xm, wq, ws, workspace=lw_, stream=s)))
    torch.cuda.synchronize()
    for o, z in got:
        assert torch.equal(o, want) and torch.equal(z, y)
    assert cq.device_error() == (0, 0)


def test_binding_refuses_mismatched_tensors(cq):
    g = gen(70)
    x, wq, ws = tokens(g, 4, 64), codes(g, 32, 64), scales(g, 32, K=64)
    xq, am = cq.cq_quant_rows(x)
    bad = [
        lambda: cq.cq_linear_i8(x.float(), wq, ws),
        lambda: cq.cq_linear_i8(x[:, :48], wq[:, :48].contiguous(), ws),       # strided rows
        lambda: cq.cq_linear_i8(x, wq.t().contiguous().t(), ws),
        lambda: cq.cq_linear_i8(x, wq, ws[:31]),
        lambda: cq.cq_linear_i8(x, wq, ws.cpu()),
        lambda: cq.cq_linear_i8(x, wq, ws, out_dtype=5),
        lambda: cq.cq_linear_i8(x, wq, ws, out=torch.empty(4, 31, device="cuda")),
        lambda: cq.cq_gemm_i8(xq, am[:3], wq, ws),
        lambda: cq.cq_gemm_i8(x, am, wq, ws),
        lambda: cq.cq_moe_route(torch.zeros(2, 8, device="cuda", dtype=torch.float16), 2),
        lambda: cq.cq_moe_route(torch.zeros(8, 2, device="cuda").t(), 2),
        lambda: cq.cq_moe_route(torch.zeros(2, 8, device="cuda"), 2,
                                bias=torch.zeros(7, device="cuda")),
    ]
    for f in bad:
        with pytest.raises(ValueError):
            f()
    for f in (lambda: cq.cq_moe_route(torch.zeros(2, 8, device="cuda"), 9),
              lambda: cq.cq_linear_i8(tokens(g, 2, 24), codes(g, 8, 24), scales(g, 8, K=24)),
              lambda: cq.cq_linear_i8(x, wq[:31], ws[:31], epilogue=cq.EPI_SWIGLU)):
        with pytest.raises(cq.CQError):
            f()
    lw = layer(g, 2, 64, 32)
    ids, w = torch.zeros((4, 1), dtype=torch.int32, device="cuda"), torch.ones(4, 1, device="cuda")
    for args in ((x, ids.long(), w, *lw), (x, ids, w.double(), *lw), (x, ids, None, *lw),
                 (x, ids, w, lw[0][:, :60], *lw[1:])):
        with pytest.raises(ValueError):
            cq.cq_moe_i8(*args)
    small = torch.zeros(256, dtype=torch.uint8, device="cuda")
    with pytest.raises(cq.CQError):
        cq.cq_moe_i8(x, ids, w, *lw, workspace=small)
    xm = tokens(g, 100, 64)
    with pytest.raises(cq.CQError):
        cq.cq_linear_i8(xm, wq, ws, workspace=small)
    with pytest.raises(cq.CQError):                  # not 256-byte aligned
        cq.cq_linear_i8(xm, wq, ws,
                        workspace=torch.zeros(1 << 20, dtype=torch.uint8, device="cuda")[16:])
    with pytest.raises(ValueError):
        cq.cq_linear_i8(xm, wq, ws, workspace=torch.zeros(1 << 20, dtype=torch.uint8))


def test_expert_parallel_layer_on_one_rank(cq):
    """The expert-parallel exchange around INT8 experts: on one rank the bits
    of the layer itself."""
    from bit_non_uniform_b200.ep import MoeExpertParallel, libcq_i8_compute
    g = gen(80)
    T, k, E, H, I = 6, 3, 8, 512, 96
    x, lw = tokens(g, T, H), layer(g, E, H, I)
    ids, w = distinct_ids(g, T, E, k), torch.rand(T, k, generator=g, device="cuda")
    ids[2] = -1                                      # a token without routes
    want = cq.cq_moe_i8(x, ids, w, *lw)[1]
    ep = MoeExpertParallel(E, H, libcq_i8_compute(*lw))
    assert torch.equal(ep.forward(x, ids, w), want)


def test_compiled_and_general_calls_agree(cq, monkeypatch):
    g = gen(90)
    H, I, E, k = 256, 96, 6, 2
    lw = layer(g, E, H, I)
    wq, ws = codes(g, 300, H), scales(g, 300, K=H)
    bias = torch.randn(E, generator=g, device="cuda")

    def calls(T):
        gg = gen(T)
        x = tokens(gg, T, H)
        xq, am = cq.cq_quant_rows(x)
        logits = torch.randn(T, E, generator=gg, device="cuda")
        ids, w = cq.cq_moe_route(logits, k, bias=bias, scale=1.5)
        bufs = (cq.gemm_i8_workspace(T, 300, H), cq.moe_i8_workspace(T, k, E, H, I))
        return (ids, w, cq.cq_linear_i8(x, wq, ws, epilogue=cq.EPI_SWIGLU),
                cq.cq_linear_i8(x, wq, ws, out_dtype=cq.BF16, workspace=bufs[0]),
                cq.cq_gemm_i8(xq, am, wq, ws),
                cq.cq_moe_i8(x, ids, w, *lw, route_out=False)[1],
                cq.cq_moe_i8(x, ids, w, *lw, out_dtype=cq.BF16, route_out=None,
                             workspace=bufs[1])[1])

    assert cq._direct is not None
    for T in (0, 1, 5, 70):
        fast = calls(T)
        with monkeypatch.context() as m:
            m.setattr(cq, "_direct", None)
            for a, b in zip(fast, calls(T)):
                assert a.dtype == b.dtype and a.shape == b.shape and torch.equal(a, b)


def test_route_refuses_more_experts_than_there_are_without_allocating(cq):
    logits = torch.randn(4096, 8, device="cuda")
    for k in (9, 2 ** 31 - 1):
        with pytest.raises((ValueError, RuntimeError)) as e:
            cq.cq_moe_route(logits, k)
        assert not isinstance(e.value, torch.OutOfMemoryError), k
    assert cq.cq_moe_route(logits, 8)[0].shape == (4096, 8)
