"""The 8-bit integer operators and the MoE router: cases, inputs and plain forms.

Three operators are covered:

* ``linear``: y = x W^T with x quantized to INT8 per token inside the call and W
  held as INT8 with a scale per output channel (``cq_linear_i8``), or the same
  product of rows quantized before (``cq_gemm_i8``); optionally with SwiGLU.
* ``moe``: the routed-expert FFN of one MoE layer on INT8 experts
  (``cq_moe_i8``): quantize, gate/up, SwiGLU, quantize, down, weighted sum.
* ``route``: a router's logits to the top-k expert ids and their weights
  (``cq_moe_route``).

With ``own`` false, ``run`` computes them from elementary torch operations.
"""
from __future__ import annotations

import math
import random

import torch

own = False

MIN_MASK = "lowest"          # masked experts get the type's lowest value
INF_MASK = "inf"             # masked experts get -inf


def _cq():
    import bit_non_uniform_b200 as cq
    return cq


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # a small projection for one token: the call's latency
        dict(name="linear_m1_small", op="linear", M=1, N=1000, K=512, swiglu=False, f32=False,
             quantized=False),
        # one decode step of a shared expert's gate/up: weights streamed once
        dict(name="linear_m1_gate_up", op="linear", M=1, N=6144, K=7168, swiglu=True, f32=False,
             quantized=False),
        # a decode batch of odd size through a projection, FP32 output
        dict(name="linear_m37", op="linear", M=37, N=7168, K=2048, swiglu=False, f32=True,
             quantized=False),
        # several projections share one quantized chunk of tokens: odd token and channel counts
        dict(name="gemm_m1000", op="linear", M=1000, N=7163, K=7168, swiglu=False, f32=False,
             quantized=True),
        # a prefill chunk through a shared expert's gate/up
        dict(name="linear_m4096_gate_up", op="linear", M=4096, N=6144, K=7168, swiglu=True,
             f32=False, quantized=False),
        # a tiny layer for one token: the call's latency
        dict(name="moe_t1_tiny", op="moe", T=1, k=2, E=8, H=512, I=256, dropped=0.0),
        # one token of the large layer: 16 of the resident experts are read
        dict(name="moe_t1", op="moe", T=1, k=16, E=64, H=7168, I=3072, dropped=0.0),
        # a decode batch of 16 sequences on the same layer: every resident expert is read
        dict(name="moe_t16", op="moe", T=16, k=16, E=64, H=7168, I=3072, dropped=0.0),
        # ragged sizes, a third of the routes owned by other ranks
        dict(name="moe_t5_ragged", op="moe", T=5, k=6, E=40, H=2064, I=1040, dropped=0.33),
        # one decode step's router: sigmoid scores with a selection bias
        dict(name="route_t1", op="route", T=1, E=896, k=16, sigmoid=True, bias=True, renorm=True,
             bf16=False, masked=0, mask=INF_MASK),
        # a prefill chunk's router, BF16 logits (many equal scores)
        dict(name="route_t4096", op="route", T=4096, E=896, k=16, sigmoid=True, bias=True,
             renorm=True, bf16=True, masked=0, mask=INF_MASK),
        # softmax scores over an odd number of experts, some of them masked
        dict(name="route_t333_masked", op="route", T=333, E=125, k=6, sigmoid=False, bias=False,
             renorm=False, bf16=False, masked=31, mask=MIN_MASK),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng: random.Random):
    op = rng.choice(["linear", "linear", "moe", "moe", "route"])
    if op == "linear":
        M = _log_int(rng, 1, 4096)
        K = 16 * _log_int(rng, 8, 512)
        N = _log_int(rng, 64, 8192)
        while M * N * K > 4096 * 6144 * 7168:
            N = max(64, N // 2)
        swiglu = rng.random() < 0.4
        if swiglu:
            N += N % 2
        return dict(op=op, M=M, N=N, K=K, swiglu=swiglu, f32=rng.random() < 0.4,
                    quantized=rng.random() < 0.4)
    if op == "moe":
        E = _log_int(rng, 4, 64)
        k = rng.randint(1, min(E, 16))
        T = _log_int(rng, 1, 16)
        H = 16 * _log_int(rng, 16, 448)
        I = 16 * _log_int(rng, 8, 192)
        return dict(op=op, T=T, k=k, E=E, H=H, I=I,
                    dropped=rng.choice([0.0, 0.0, 0.25, 0.75]))
    E = _log_int(rng, 8, 1024)
    return dict(op=op, T=_log_int(rng, 1, 4096), E=E, k=rng.randint(1, min(E, 16)),
                sigmoid=rng.random() < 0.6, bias=rng.random() < 0.6, renorm=rng.random() < 0.6,
                bf16=rng.random() < 0.5, masked=rng.choice([0, 0, E // 3]),
                mask=rng.choice([INF_MASK, MIN_MASK]))


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) & 0x7FFFFFFF)
    return g


def _tokens(g, rows, cols):
    """Activations after a norm: unit variance, a few channels several times larger."""
    x = torch.randn(rows, cols, generator=g, device="cuda")
    loud = torch.rand(cols, generator=g, device="cuda") < 0.005
    return (x * torch.where(loud, 6.0, 1.0)).to(torch.bfloat16)


def _int8_weights(g, rows, cols):
    """INT8 codes of Gaussian rows (the row's largest value near four deviations)."""
    w = torch.randn(rows, cols, generator=g, device="cuda")
    return w.mul_(127.0 / 4.2).round_().clamp_(-127, 127).to(torch.int8)


def _channel_scales(g, rows, cols):
    """Scales that give products of unit variance, spread over a factor of three."""
    s = 0.5 + torch.rand(rows, generator=g, device="cuda")
    return s * (4.2 / 127.0) / math.sqrt(cols)


def _quant_rows(x):
    """INT8 codes and row maxima; the decisions are taken in FP32."""
    x = x.float()
    amax = x.abs().amax(dim=1)
    # a true division: `127.0 / tensor` multiplies by a rounded reciprocal
    inv = torch.where(amax > 0, torch.full_like(amax, 127.0) / amax, torch.zeros_like(amax))
    q = torch.round(x * inv[:, None]).clamp(-127, 127)
    return q, amax


def _prepare_linear(c, g):
    st = dict(case=c)
    x = _tokens(g, c["M"], c["K"])
    if c["quantized"]:
        q, amax = _quant_rows(x)
        st["xq"], st["absmax"] = q.to(torch.int8), amax
    else:
        st["x"] = x
    st["wq"] = _int8_weights(g, c["N"], c["K"])
    st["ws"] = _channel_scales(g, c["N"], c["K"])
    if own:
        cq = _cq()
        epi = cq.EPI_SWIGLU if c["swiglu"] else cq.EPI_NONE
        st["workspace"] = cq.gemm_i8_workspace(c["M"], c["N"], c["K"], epi)
    return st


def _prepare_moe(c, g):
    T, k, E, H, I = c["T"], c["k"], c["E"], c["H"], c["I"]
    st = dict(case=c, tokens=_tokens(g, T, H))
    # popular experts take more routes; the ids of a token are distinct
    pop = torch.randn(E, generator=g, device="cuda") * 0.7
    logits = torch.randn(T, E, generator=g, device="cuda") + pop
    val, ids = torch.topk(logits, k, dim=1)
    st["w"] = torch.softmax(val, dim=1)
    ids = ids.to(torch.int32)
    if c["dropped"] > 0:
        gone = torch.rand(T, k, generator=g, device="cuda") < c["dropped"]
        ids = torch.where(gone, torch.full_like(ids, -1), ids)
    st["ids"] = ids.contiguous()
    w_gu = torch.empty((E, 2 * I, H), dtype=torch.int8, device="cuda")
    w_dn = torch.empty((E, H, I), dtype=torch.int8, device="cuda")
    for e in range(E):
        w_gu[e] = _int8_weights(g, 2 * I, H)
        w_dn[e] = _int8_weights(g, H, I)
    st["w_gu"], st["w_dn"] = w_gu, w_dn
    st["s_gu"] = _channel_scales(g, E * 2 * I, H).view(E, 2 * I)
    st["s_dn"] = _channel_scales(g, E * H, I).view(E, H)
    if own:
        st["workspace"] = _cq().moe_i8_workspace(T, k, E, H, I)
    return st


def _prepare_route(c, g):
    T, E = c["T"], c["E"]
    logits = torch.randn(T, E, generator=g, device="cuda") * 1.5
    logits = logits.to(torch.bfloat16) if c["bf16"] else logits
    if c["masked"]:
        low = -math.inf if c["mask"] == INF_MASK else torch.finfo(logits.dtype).min
        order = torch.argsort(torch.rand(T, E, generator=g, device="cuda"), dim=1)
        logits.scatter_(1, order[:, :c["masked"]], low)
    bias = torch.randn(E, generator=g, device="cuda") * 0.05 if c["bias"] else None
    return dict(case=c, logits=logits, bias=bias, scale=2.5 if c["sigmoid"] else 1.0)


def prepare(case, seed):
    g = _gen(seed)
    return {"linear": _prepare_linear, "moe": _prepare_moe,
            "route": _prepare_route}[case["op"]](case, g)


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def _plain_linear(st):
    c = st["case"]
    if c["quantized"]:
        xq, amax = st["xq"].float(), st["absmax"]
    else:
        xq, amax = _quant_rows(st["x"])
    y = (xq @ st["wq"].float().t()) * (amax / 127.0)[:, None] * st["ws"][None, :]
    if c["swiglu"]:
        h = c["N"] // 2
        gate, up = y[:, :h], y[:, h:]
        y = gate / (1.0 + torch.exp(-gate)) * up
    return y if c["f32"] else y.to(torch.bfloat16)


def _int_dot(xq, wq):
    """Exact integer dot products [rows][N] in FP64: every FP32 sum of 1024 products of
    INT8 codes stays below 2^24."""
    acc = torch.zeros(xq.shape[0], wq.shape[0], dtype=torch.float64, device=xq.device)
    w = wq.float()
    for k0 in range(0, w.shape[1], 1024):
        acc += xq[:, k0:k0 + 1024] @ w[:, k0:k0 + 1024].t()
    return acc


def _plain_expert(xq, sx, w_gu, s_gu, w_dn, s_dn):
    """Rows of one expert.  The SwiGLU values sit next to rounding borders of the second
    quantization, so they are computed in 64 bits and rounded once."""
    gu = _int_dot(xq, w_gu) * (sx.double()[:, None] * s_gu.double()[None, :])
    I = gu.shape[1] // 2
    gate, up = gu[:, :I], gu[:, I:]
    h = (gate / (1.0 + torch.exp(-gate)) * up).float()
    hq, hmax = _quant_rows(h)
    y = _int_dot(hq, w_dn) * ((hmax / 127.0).double()[:, None] * s_dn.double()[None, :])
    return y.float()


def _plain_moe(st):
    c = st["case"]
    T, k, E, H = c["T"], c["k"], c["E"], c["H"]
    xq, amax = _quant_rows(st["tokens"])
    sx = amax / 127.0
    ids = st["ids"].long()
    live = (ids >= 0) & (ids < E)
    w = torch.where(live, st["w"], torch.zeros_like(st["w"]))
    out = torch.zeros(T, H, device=xq.device)
    if T * k <= E:
        # few routes: fetch the expert of each
        flat = ids.clamp(0, E - 1).view(-1)
        for r in range(T * k):
            t, e = r // k, flat[r:r + 1]
            y = _plain_expert(xq[t:t + 1], sx[t:t + 1], st["w_gu"].index_select(0, e)[0],
                              st["s_gu"].index_select(0, e)[0],
                              st["w_dn"].index_select(0, e)[0],
                              st["s_dn"].index_select(0, e)[0])
            out[t] += w[t, r % k] * y[0]
    else:
        # many: every expert on every token, unselected ones with weight zero
        for e in range(E):
            we = torch.where(ids == e, w, torch.zeros_like(w)).sum(dim=1)
            y = _plain_expert(xq, sx, st["w_gu"][e], st["s_gu"][e], st["w_dn"][e],
                              st["s_dn"][e])
            out += we[:, None] * y
    return out.to(torch.bfloat16)


def _plain_route(st):
    c = st["case"]
    logits = st["logits"].double()              # scores lie next to the border of the selection
    k = c["k"]
    if c["sigmoid"]:
        score = 1.0 / (1.0 + torch.exp(-logits))
    else:
        e = torch.exp(logits - logits.amax(dim=1, keepdim=True))
        score = e / e.sum(dim=1, keepdim=True)
    # the scores grow with the logits; without a bias the logits order them exactly
    pick = score + st["bias"].double() if c["bias"] else logits
    pick = torch.where(logits > -math.inf, pick, torch.full_like(pick, -math.inf))
    order = torch.sort(pick, dim=1, descending=True, stable=True).indices[:, :k]
    live = torch.gather(logits, 1, order) > -math.inf
    w = torch.where(live, torch.gather(score, 1, order), torch.zeros_like(score[:, :k]))
    if c["renorm"]:
        total = w.sum(dim=1, keepdim=True)
        w = torch.where(total > 0, w / total, torch.zeros_like(w))
    ids = torch.where(live, order, torch.full_like(order, -1))
    return ids.to(torch.int32), (w * st["scale"]).float()


def _own(st):
    cq = _cq()
    c = st["case"]
    if c["op"] == "linear":
        epi = cq.EPI_SWIGLU if c["swiglu"] else cq.EPI_NONE
        dt = cq.F32 if c["f32"] else cq.BF16
        if c["quantized"]:
            return cq.cq_gemm_i8(st["xq"], st["absmax"], st["wq"], st["ws"], epilogue=epi,
                                 out_dtype=dt, workspace=st["workspace"])
        return cq.cq_linear_i8(st["x"], st["wq"], st["ws"], epilogue=epi, out_dtype=dt,
                               workspace=st["workspace"])
    if c["op"] == "moe":
        _, out = cq.cq_moe_i8(st["tokens"], st["ids"], st["w"], st["w_gu"], st["s_gu"],
                              st["w_dn"], st["s_dn"], out_dtype=cq.BF16, route_out=False,
                              workspace=st["workspace"])
        return out
    scoring = cq.SCORE_SIGMOID if c["sigmoid"] else cq.SCORE_SOFTMAX
    return cq.cq_moe_route(st["logits"], c["k"], bias=st["bias"], scoring=scoring,
                           renorm=c["renorm"], scale=st["scale"])


def run(state):
    if own:
        return _own(state)
    return {"linear": _plain_linear, "moe": _plain_moe,
            "route": _plain_route}[state["case"]["op"]](state)


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------

def work(case):
    c = case
    if c["op"] == "linear":
        M, N, K = c["M"], c["N"], c["K"]
        cols = N // 2 if c["swiglu"] else N
        x = M * K + 4 * M if c["quantized"] else 2 * M * K
        return {"bytes": x + N * K + 4 * N + M * cols * (4 if c["f32"] else 2),
                "flops": 2 * M * N * K}
    if c["op"] == "moe":
        T, k, E, H, I = c["T"], c["k"], c["E"], c["H"], c["I"]
        live = k * (1.0 - c["dropped"])
        active = E * (1.0 - (1.0 - live / E) ** T)        # distinct experts, routes spread evenly
        return {"bytes": int(active * (3 * H * I + 4 * (2 * I + H)) + T * (4 * H + 8 * k)),
                "flops": int(2 * T * live * 3 * H * I)}
    T, E, k = c["T"], c["E"], c["k"]
    return {"bytes": T * E * (2 if c["bf16"] else 4) + (4 * E if c["bias"] else 0) + T * k * 8,
            "flops": T * E * 4}


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------

def _exact_codes(v):
    """The codes' definition: RNE(RN32(v * RN32(127 / max|v|))), saturated; 0 for a zero row."""
    v32 = v.to(torch.float32)
    top = v32.abs().max(dim=1, keepdim=True).values
    factor = torch.full_like(top, 127.0) / top
    codes = (v32 * factor).nan_to_num(0.0).double().round().clamp(-127.0, 127.0)
    return codes, top.double()[:, 0]


def _exact_silu(v):
    return v * torch.sigmoid(v)


def _exact_linear(st):
    c = st["case"]
    codes, top = ((st["xq"].double(), st["absmax"].double()) if c["quantized"]
                  else _exact_codes(st["x"]))
    parts = []
    for n0 in range(0, c["N"], 2048):
        w = st["wq"][n0:n0 + 2048].double() * st["ws"][n0:n0 + 2048].double()[:, None]
        parts.append(torch.einsum("mk,nk->mn", codes * (top / 127.0)[:, None], w))
    y = torch.cat(parts, dim=1)
    if c["swiglu"]:
        gate, up = y.chunk(2, dim=1)
        y = _exact_silu(gate) * up
    return y


def _exact_moe(st):
    c = st["case"]
    codes, top = _exact_codes(st["tokens"])
    out = torch.zeros(c["T"], c["H"], dtype=torch.float64, device=codes.device)
    for e in range(c["E"]):
        t, j = torch.nonzero(st["ids"] == e, as_tuple=True)
        if t.numel() == 0:
            continue
        gu = torch.einsum("mk,nk->mn", codes[t], st["w_gu"][e].double())
        gu = gu * (top[t] / 127.0).float().double()[:, None] * st["s_gu"][e].double()
        gate, up = gu.chunk(2, dim=1)
        hc, htop = _exact_codes(_exact_silu(gate) * up)
        y = torch.einsum("mk,nk->mn", hc, st["w_dn"][e].double())
        y = y * (htop / 127.0)[:, None] * st["s_dn"][e].double()
        out.index_add_(0, t, y * st["w"][t, j].double()[:, None])
    return out


def _exact_route(st):
    c = st["case"]
    logits = st["logits"].double()
    score = torch.sigmoid(logits) if c["sigmoid"] else torch.softmax(logits, dim=1)
    alive = ~torch.isneginf(logits)
    key = logits if st["bias"] is None else score + st["bias"].double()
    key = key.masked_fill(~alive, -math.inf)
    chosen = torch.argsort(key, dim=1, descending=True, stable=True)[:, :c["k"]]
    w = score.gather(1, chosen) * alive.gather(1, chosen)
    if c["renorm"]:
        w = (w / w.sum(dim=1, keepdim=True)).nan_to_num(0.0)
    return None, w * st["scale"]


def exact(case, seed):
    global own
    keep, own = own, False                  # inputs only: no workspace of the framework
    try:
        st = prepare(case, seed)
    finally:
        own = keep
    return {"linear": _exact_linear, "moe": _exact_moe,
            "route": _exact_route}[case["op"]](st)
