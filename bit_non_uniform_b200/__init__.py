"""Python binding of libcq, the B200 CubicQuant weight-only GEMM library.

This module only marshals arguments: every step of the computation runs in
the CUDA kernels of ``libcq.so`` (built in-tree by ``build.py``).  There is
no CPU fallback; if the library is missing or a call fails, an exception is
raised.  PyTorch is used for device memory and streams.

The calls mirror ``include/cq.h``:

* ``cq_pack(codes, B)``                         -> packed [N][K*B/8] uint8
* ``cq_decode(packed, scales, ab, K, B, G)``    -> W [N][K] (float32 / bfloat16)
* ``cq_gemm(x, packed, scales, ab, N, K, B, G)`` -> y [M][N] (or [M][N/2])
* ``cq_moe_grouped_gemm(tokens, topk_ids, ...)`` -> per-route / combined outputs
* ``cq_linear_i8(x, wq, wscale)`` / ``cq_gemm_i8(xq, absmax, wq, wscale)`` -> y, INT8 weights
* ``cq_moe_i8(tokens, topk_ids, topk_w, w_gu, s_gu, w_dn, s_dn)`` -> the layer on INT8 experts
* ``cq_moe_route(logits, k)``                   -> (topk_ids, topk_w)
"""
from __future__ import annotations

import contextlib
import ctypes
import os

import torch

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libcq.so")

MIDRISE, MIDTREAD = 0, 1
F32, BF16 = 0, 1
EPI_NONE, EPI_SWIGLU = 0, 1
SCORE_SOFTMAX, SCORE_SIGMOID = 0, 1

_STATUS = {
    0: "ok", 1: "invalid argument", 2: "unsupported", 3: "CUDA runtime error",
    4: "a bounded device wait ran out", 5: "workspace missing or too small",
}


class CQError(RuntimeError):
    def __init__(self, status: int, where: str):
        super().__init__(f"{where}: libcq status {status} ({_STATUS.get(status, '?')})")
        self.status = status


_lib = None
_direct = None          # the compiled INT8 calls (_cq_torch), loaded with the library


class MatrixDesc(ctypes.Structure):
    _fields_ = [("packed", ctypes.c_void_p), ("scales", ctypes.c_void_p),
                ("ab", ctypes.c_void_p), ("B", ctypes.c_int32), ("reserved", ctypes.c_int32)]


class ExpertDesc(ctypes.Structure):
    _fields_ = [("gate_up", MatrixDesc), ("down", MatrixDesc)]


def lib():
    """Load libcq.so (raises if it has not been built), and the compiled calls
    that link against it.  Not before: a process that imports the package in
    order to build the library must not hold the one it replaces."""
    global _lib, _direct
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(
            f"libcq.so not found at {LIB_PATH}; build it with "
            "`python -m bit_non_uniform_b200.build`")
    L = ctypes.CDLL(LIB_PATH)
    P, i64, i32, sz, u64 = (ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_size_t,
                            ctypes.c_uint64)
    sigs = {
        "cq_version": (i32, []),
        "cq_status_string": (ctypes.c_char_p, [i32]),
        "cq_pack": (i32, [P, i64, i64, i32, P, P]),
        "cq_decode": (i32, [P, P, P, i64, i64, i32, i32, i32, i32, P, P]),
        "cq_gemm_workspace_size": (sz, [i64, i64, i64, i32, i32, i32]),
        "cq_gemm": (i32, [P, i64, P, P, P, i64, i64, i32, i32, i32, i32, i32, P, P, sz, P]),
        "cq_moe_layer_bytes": (sz, [i32]),
        "cq_moe_prepare_layer": (i32, [P, i32, i64, i64, i32, P]),
        "cq_moe_workspace_size": (sz, [i64, i32, i32, i64, i64, i32]),
        "cq_moe_grouped_gemm": (i32, [P, i64, P, P, i32, i32, P, i64, i64, i32, i32, i32,
                                      P, P, P, sz, P]),
        "cq_gemm_noalloc": (i32, [P, i64, P, P, P, i64, i64, i32, i32, i32, i32, i32, P, P]),
        "cq_gemm_host": (i32, [P, i64, P, P, P, i64, i64, i32, i32, i32, i32, i32, P, P, P, P,
                               sz, P]),
        "cq_get_device_error": (i32, [P, ctypes.POINTER(ctypes.c_int)]),
        "cq_test_gemm_bounded": (i32, [P, i64, P, P, P, i64, i64, i32, i32, P, P, sz, u64,
                                       i32, P]),
        "cq_test_gemm_path_workspace_size": (sz, [i64, i64, i64, i32, i32, i32, i32]),
        "cq_quant_rows": (i32, [P, i64, i64, P, P, P]),
        "cq_gemm_a8_workspace_size": (sz, [i64, i64, i64, i32, i32, i32]),
        "cq_gemm_a8": (i32, [P, i64, P, P, P, i64, i64, i32, i32, i32, i32, i32, P, P, sz, P]),
        "cq_gemm_i8_workspace_size": (sz, [i64, i64, i64, i32]),
        "cq_gemm_i8": (i32, [P, P, i64, P, P, i64, i64, i32, i32, P, P, sz, P]),
        "cq_linear_i8": (i32, [P, i64, P, P, i64, i64, i32, i32, P, P, sz, P]),
        "cq_moe_i8_workspace_size": (sz, [i64, i32, i32, i64, i64]),
        "cq_moe_i8": (i32, [P, i64, P, P, i32, i32, P, P, P, P, i64, i64, i32, P, P, P, sz, P]),
        "cq_moe_route": (i32, [P, i32, i64, i32, i32, P, i32, i32, ctypes.c_float, P, P, P]),
        "cq_test_product_i8_path": (i32, [i64, i64, i64, i32]),
        "cq_test_product_i8": (i32, [P, P, i64, P, P, i64, i64, i32, i32, P, P, sz, i32, u64, i32,
                                     P]),
        "cq_test_moe_i8_path": (i32, [i64, i32, i32, i64, i64, ctypes.POINTER(i64)]),
        "cq_test_moe_i8_workspace_size": (sz, [i64, i32, i32, i64, i64, i32]),
        "cq_test_moe_i8": (i32, [P, i64, P, P, i32, i32, P, P, P, P, i64, i64, i32, P, P, P, sz,
                                 i32, u64, i32, P]),
        "cq_test_gemm_path": (i32, [P, i64, P, P, P, i64, i64, i32, i32, i32, i32, i32, P, P,
                                    sz, i32, P]),
    }
    for name, (res, args) in sigs.items():
        f = getattr(L, name)
        f.restype = res
        f.argtypes = args
    from .build import built_for
    try:
        from . import _cq_torch as _direct
        if getattr(_direct, "built_for", None) != built_for():
            _direct = None
    except ImportError:                    # not built: the calls go through Python
        _direct = None
    _lib = L
    return L


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _on_stream(stream=None):
    """Allocations and fills of a binding call go on the call's stream, so
    that the buffers it creates are ready (and are recycled) in that
    stream's order."""
    return torch.cuda.stream(stream) if stream is not None else contextlib.nullcontext()


def _stream(stream=None):
    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


def _check(st: int, where: str):
    if st != 0:
        raise CQError(st, where)


def _need_cuda(*ts):
    for t in ts:
        if t is not None and not t.is_cuda:
            raise ValueError("libcq works on CUDA tensors only")


def version() -> int:
    return int(lib().cq_version())


def cq_pack(codes: torch.Tensor, B: int, out: torch.Tensor | None = None, stream=None):
    """codes uint8 [N][K] (CUDA) -> packed uint8 [N][K*B/8]."""
    with _on_stream(stream):
        _need_cuda(codes)
        codes = codes.contiguous()
        N, K = codes.shape
        if out is None:
            out = torch.empty((N, K * B // 8), dtype=torch.uint8, device=codes.device)
        _check(lib().cq_pack(_ptr(codes), N, K, B, _ptr(out), _stream(stream)), "cq_pack")
        return out


def cq_decode(packed, scales, ab, K: int, B: int, G: int, mode: int = MIDRISE,
              out_dtype: int = F32, stream=None):
    """Decode packed codes + (s, a, b) into W [N][K] (float32 or bfloat16)."""
    with _on_stream(stream):
        _need_cuda(packed, scales, ab)
        N = packed.shape[0]
        dt = torch.float32 if out_dtype == F32 else torch.bfloat16
        W = torch.empty((N, K), dtype=dt, device=packed.device)
        _check(lib().cq_decode(_ptr(packed), _ptr(scales), _ptr(ab), N, K, B, G, mode, out_dtype,
                               _ptr(W), _stream(stream)), "cq_decode")
        return W


def gemm_workspace_size(M, N, K, B, G, epilogue=EPI_NONE) -> int:
    return int(lib().cq_gemm_workspace_size(M, N, K, B, G, epilogue))


def gemm_workspace(M, N, K, B, G, epilogue=EPI_NONE, device="cuda"):
    """A zero-initialised workspace buffer for cq_gemm."""
    n = gemm_workspace_size(M, N, K, B, G, epilogue)
    return torch.zeros(max(n, 16), dtype=torch.uint8, device=device)


def cq_gemm(x, packed, scales, ab, N: int, K: int, B: int, G: int, mode: int = MIDRISE,
            epilogue: int = EPI_NONE, out_dtype: int = F32, workspace=None, out=None,
            stream=None):
    """y = x W^T with W given packed; x bfloat16 [M][K]."""
    with _on_stream(stream):
        _need_cuda(x, packed, scales, ab)
        assert x.dtype == torch.bfloat16 and x.is_contiguous()
        M = x.shape[0]
        ncol = N // 2 if epilogue == EPI_SWIGLU else N
        if out is None:
            dt = torch.float32 if out_dtype == F32 else torch.bfloat16
            out = torch.empty((M, ncol), dtype=dt, device=x.device)
        if workspace is None:
            workspace = gemm_workspace(M, N, K, B, G, epilogue, x.device)
        _check(lib().cq_gemm(_ptr(x), M, _ptr(packed), _ptr(scales), _ptr(ab), N, K, B, G, mode,
                             epilogue, out_dtype, _ptr(out), _ptr(workspace),
                             workspace.numel() * workspace.element_size(), _stream(stream)),
               "cq_gemm")
        return out


# kernels of cq_gemm (test hook cq_test_gemm_path)
PATH_AUTO, PATH_NARROW, PATH_GEMV, PATH_ENGINE = 0, 1, 2, 3


def gemm_on_path(path: int, x, packed, scales, ab, N: int, K: int, B: int, G: int,
                 mode: int = MIDRISE, epilogue: int = EPI_NONE, out_dtype: int = F32,
                 stream=None):
    """cq_gemm on a chosen kernel (a test hook); raises CQError with status 2
    when that kernel does not take the problem."""
    with _on_stream(stream):
        _need_cuda(x, packed, scales, ab)
        M = x.shape[0]
        ncol = N // 2 if epilogue == EPI_SWIGLU else N
        dt = torch.float32 if out_dtype == F32 else torch.bfloat16
        out = torch.empty((M, ncol), dtype=dt, device=x.device)
        n = int(lib().cq_test_gemm_path_workspace_size(M, N, K, B, G, epilogue, path))
        ws = torch.zeros(max(n, 16), dtype=torch.uint8, device=x.device)
        _check(lib().cq_test_gemm_path(_ptr(x), M, _ptr(packed), _ptr(scales), _ptr(ab), N, K, B, G,
                                       mode, epilogue, out_dtype, _ptr(out), _ptr(ws), ws.numel(),
                                       path, _stream(stream)), "cq_test_gemm_path")
        return out


def cq_gemm_host(x_host, packed, scales, ab, N: int, K: int, B: int, G: int,
                 mode: int = MIDRISE, epilogue: int = EPI_NONE, out_dtype: int = F32,
                 y_host=None, x_dev=None, y_dev=None, workspace=None, stream=None):
    """cq_gemm with x and y in host memory (pinned CPU tensors keep the
    copies asynchronous): the copies and the GEMM are queued on `stream`;
    synchronize it before reading y_host."""
    with _on_stream(stream):
        _need_cuda(packed, scales, ab)
        assert x_host.device.type == "cpu" and x_host.dtype == torch.bfloat16
        assert x_host.is_contiguous()
        M = x_host.shape[0]
        dev = packed.device
        ncol = N // 2 if epilogue == EPI_SWIGLU else N
        dt = torch.float32 if out_dtype == F32 else torch.bfloat16
        if y_host is None:
            y_host = torch.empty((M, ncol), dtype=dt).pin_memory()
        if x_dev is None:
            x_dev = torch.empty((M, K), dtype=torch.bfloat16, device=dev)
        if y_dev is None:
            y_dev = torch.empty((M, ncol), dtype=dt, device=dev)
        if workspace is None:
            workspace = gemm_workspace(M, N, K, B, G, epilogue, dev)
        _check(lib().cq_gemm_host(x_host.data_ptr(), M, _ptr(packed), _ptr(scales), _ptr(ab), N, K,
                                  B, G, mode, epilogue, out_dtype, y_host.data_ptr(), _ptr(x_dev),
                                  _ptr(y_dev), _ptr(workspace), workspace.numel(), _stream(stream)),
               "cq_gemm_host")
        return y_host


def cq_gemm_noalloc(x, packed, scales, ab, N: int, K: int, B: int, G: int,
                    mode: int = MIDRISE, epilogue: int = EPI_NONE, out_dtype: int = F32,
                    out=None, stream=None):
    """cq_gemm without a workspace (scratch in libcq's fixed array; M <= 16)."""
    with _on_stream(stream):
        _need_cuda(x, packed, scales, ab)
        M = x.shape[0]
        ncol = N // 2 if epilogue == EPI_SWIGLU else N
        if out is None:
            dt = torch.float32 if out_dtype == F32 else torch.bfloat16
            out = torch.empty((M, ncol), dtype=dt, device=x.device)
        _check(lib().cq_gemm_noalloc(_ptr(x), M, _ptr(packed), _ptr(scales), _ptr(ab), N, K, B, G,
                                     mode, epilogue, out_dtype, _ptr(out), _stream(stream)),
               "cq_gemm_noalloc")
        return out


def gemm_a8_workspace_size(M, N, K, B, G, epilogue=EPI_NONE) -> int:
    return int(lib().cq_gemm_a8_workspace_size(M, N, K, B, G, epilogue))


def cq_quant_rows(x, stream=None):
    """Per-row dynamic INT8 quantization: (xq int8 [M][K], absmax f32 [M])."""
    with _on_stream(stream):
        _need_cuda(x)
        assert x.dtype == torch.bfloat16 and x.is_contiguous()
        M, K = x.shape
        xq = torch.empty((M, K), dtype=torch.int8, device=x.device)
        absmax = torch.empty(M, dtype=torch.float32, device=x.device)
        _check(lib().cq_quant_rows(_ptr(x), M, K, _ptr(xq), _ptr(absmax), _stream(stream)),
               "cq_quant_rows")
        return xq, absmax


def cq_gemm_a8(x, packed, scales, ab, N: int, K: int, B: int, G: int, mode: int = MIDRISE,
               epilogue: int = EPI_NONE, out_dtype: int = F32, out=None, workspace=None,
               stream=None):
    """Dynamic-A8 y = x W^T: x quantized per row to INT8 inside the call."""
    with _on_stream(stream):
        _need_cuda(x, packed, scales, ab)
        assert x.dtype == torch.bfloat16 and x.is_contiguous()
        M = x.shape[0]
        ncol = N // 2 if epilogue == EPI_SWIGLU else N
        if out is None:
            dt = torch.float32 if out_dtype == F32 else torch.bfloat16
            out = torch.empty((M, ncol), dtype=dt, device=x.device)
        if workspace is None:
            n = gemm_a8_workspace_size(M, N, K, B, G, epilogue)
            workspace = torch.empty(max(n, 256), dtype=torch.uint8, device=x.device)
        _check(lib().cq_gemm_a8(_ptr(x), M, _ptr(packed), _ptr(scales), _ptr(ab), N, K, B, G, mode,
                                epilogue, out_dtype, _ptr(out), _ptr(workspace),
                                workspace.numel(), _stream(stream)), "cq_gemm_a8")
        return out


def moe_workspace_size(T, k, E, H, I, G) -> int:
    return int(lib().cq_moe_workspace_size(T, k, E, H, I, G))


def moe_prepare_layer(experts, H: int, I: int, G: int, device="cuda"):
    """Build the device-side layer table (TMA descriptors + operand
    descriptions) for a list of per-expert dicts with keys packed_gu,
    scales_gu, ab_gu, B_gu, packed_dn, scales_dn, ab_dn, B_dn (CUDA tensors).
    Returns the table (a uint8 CUDA tensor the caller keeps alive)."""
    E = len(experts)
    arr = (ExpertDesc * E)()
    for e, ex in enumerate(experts):
        for fld, key in (("gate_up", "gu"), ("down", "dn")):
            d = getattr(arr[e], fld)
            d.packed = ex[f"packed_{key}"].data_ptr()
            d.scales = ex[f"scales_{key}"].data_ptr()
            d.ab = ex[f"ab_{key}"].data_ptr()
            d.B = int(ex[f"B_{key}"])
            d.reserved = 0
    nbytes = int(lib().cq_moe_layer_bytes(E))
    table = torch.empty(nbytes + 64, dtype=torch.uint8, device=device)
    off = (-table.data_ptr()) % 64
    table = table[off:off + nbytes]
    _check(lib().cq_moe_prepare_layer(ctypes.cast(arr, ctypes.c_void_p), E, H, I, G,
                                      _ptr(table)), "cq_moe_prepare_layer")
    return table


def moe_workspace(T, k, E, H, I, G, device="cuda"):
    n = moe_workspace_size(T, k, E, H, I, G)
    return torch.empty(max(n, 256), dtype=torch.uint8, device=device)


def cq_moe_grouped_gemm(tokens, topk_ids, topk_w, layer, E: int, H: int, I: int, G: int,
                        mode: int = MIDRISE, out_dtype: int = F32, route_out=True,
                        combine=True, workspace=None, stream=None):
    """Routed-expert FFN of one MoE layer.  Returns (route_out, out)."""
    with _on_stream(stream):
        _need_cuda(tokens, topk_ids, layer)
        T, k = topk_ids.shape
        ro = None
        if route_out is True:
            ro = torch.empty((T * k, H), dtype=torch.float32, device=tokens.device)
        elif route_out is not None and route_out is not False:
            ro = route_out
        out = None
        if combine:
            dt = torch.float32 if out_dtype == F32 else torch.bfloat16
            out = torch.empty((T, H), dtype=dt, device=tokens.device)
        if workspace is None:
            workspace = moe_workspace(T, k, E, H, I, G, tokens.device)
        _check(lib().cq_moe_grouped_gemm(
            _ptr(tokens), T, _ptr(topk_ids), _ptr(topk_w) if topk_w is not None else None, k, E,
            _ptr(layer), H, I, G, mode, out_dtype, _ptr(ro), _ptr(out), _ptr(workspace),
            workspace.numel(), _stream(stream)), "cq_moe_grouped_gemm")
        return ro, out


# ---------------------------------------------------------------------------
# INT8 weights
# ---------------------------------------------------------------------------
# A decode step makes many of these calls, each a few microseconds long on the
# GPU, so the host side of a call is kept short.  The plain call (everything on
# the current device and stream, nothing to say about the arguments) is made by
# the compiled module, in about half the time; all others go through Python:
# one test per tensor, the current stream's handle without a Stream object, and
# no context manager where device and stream are the current ones already.

def _direct_result(r, where):
    if type(r) is int:
        raise CQError(r, where)
    return r


def _on_device(index: int, stream):
    """The call's device and stream as the current ones (libcq launches on the
    current device)."""
    if stream is not None and stream.device.index != index:
        raise ValueError(f"the stream is on {stream.device}, the tensors on cuda:{index}")
    stack = contextlib.ExitStack()
    stack.enter_context(torch.cuda.device(index))
    if stream is not None:
        stack.enter_context(torch.cuda.stream(stream))
    return stack


_current_device = torch._C._cuda_getDevice
_raw_stream = torch._C._cuda_getCurrentRawStream      # of a device's current stream


def _tensor(name, t, dtype, shape, index: int) -> int:
    """Check one argument of a call and return its address."""
    if (t.dtype is dtype and t.shape == shape and t.get_device() == index
            and t.is_contiguous()):
        return t.data_ptr()
    if t.get_device() != index:
        raise ValueError(f"{name} is on {t.device}, expected cuda:{index}")
    if t.dtype != dtype:
        raise ValueError(f"{name} is {t.dtype}, expected {dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    raise ValueError(f"{name} must be contiguous")


def _scratch(workspace, index: int):
    """(address, bytes) of a call's workspace."""
    if workspace is None:
        return None, 0
    if workspace.get_device() != index or not workspace.is_contiguous():
        raise ValueError(f"the workspace must be contiguous on cuda:{index}")
    return workspace.data_ptr(), workspace.nbytes


_DTYPES = {F32: torch.float32, BF16: torch.bfloat16}


def _out_dtype(out_dtype: int):
    dt = _DTYPES.get(out_dtype)
    if dt is None:
        raise ValueError(f"out_dtype must be F32 or BF16, not {out_dtype!r}")
    return dt


def gemm_i8_workspace_size(M, N, K, epilogue=EPI_NONE) -> int:
    return int(lib().cq_gemm_i8_workspace_size(M, N, K, epilogue))


def gemm_i8_workspace(M, N, K, epilogue=EPI_NONE, device="cuda"):
    """A workspace for cq_gemm_i8 and cq_linear_i8."""
    n = gemm_i8_workspace_size(M, N, K, epilogue)
    return torch.empty(max(n, 256), dtype=torch.uint8, device=device)


def _i8_product(where, x, absmax, wq, wscale, epilogue, out_dtype, out, workspace, stream):
    try:
        M, K = x.shape
        N, _ = wq.shape
    except ValueError:
        raise ValueError(f"{where}: activations [M][K] and weights [N][K] expected") from None
    index = x.get_device()
    if index < 0:
        _need_cuda(x)
    if stream is not None or index != _current_device():
        with _on_device(index, stream):
            return _i8_product(where, x, absmax, wq, wscale, epilogue, out_dtype, out, workspace,
                               None)
    L = _lib or lib()
    dt = _out_dtype(out_dtype)
    px = _tensor("x", x, torch.bfloat16 if absmax is None else torch.int8, (M, K), index)
    pw = _tensor("wq", wq, torch.int8, (N, K), index)
    ps = _tensor("wscale", wscale, torch.float32, (N,), index)
    shape = (M, N // 2 if epilogue == EPI_SWIGLU else N)
    if out is None:
        out = x.new_empty(shape, dtype=dt)
        py = out.data_ptr()
    else:
        py = _tensor("out", out, dt, shape, index)
    st = _raw_stream(index)
    if absmax is not None:
        pa = _tensor("absmax", absmax, torch.float32, (M,), index)
        _check(L.cq_gemm_i8(px, pa, M, pw, ps, N, K, epilogue, out_dtype, py, None, 0, st), where)
        return out
    if workspace is None:
        need = L.cq_gemm_i8_workspace_size(M, N, K, epilogue)
        if need:
            workspace = x.new_empty(need, dtype=torch.uint8)
    pws, nws = _scratch(workspace, index)
    _check(L.cq_linear_i8(px, M, pw, ps, N, K, epilogue, out_dtype, py, pws, nws, st), where)
    return out


def cq_gemm_i8(xq, absmax, wq, wscale, epilogue: int = EPI_NONE, out_dtype: int = F32, out=None,
               workspace=None, stream=None):
    """y = (absmax / 127) wscale (xq wq^T): INT8 activations (cq_quant_rows) times INT8
    weights [N][K] with one scale per output channel."""
    if absmax is None:
        raise ValueError("cq_gemm_i8 needs absmax (cq_quant_rows returns it)")
    if _direct is not None and out is None and stream is None:
        r = _direct.product(xq, absmax, wq, wscale, epilogue, out_dtype, workspace)
        if r is not None:
            return _direct_result(r, "cq_gemm_i8")
    return _i8_product("cq_gemm_i8", xq, absmax, wq, wscale, epilogue, out_dtype, out, workspace,
                       stream)


def cq_linear_i8(x, wq, wscale, epilogue: int = EPI_NONE, out_dtype: int = F32, out=None,
                 workspace=None, stream=None):
    """cq_gemm_i8 on bfloat16 activations, quantized per row inside the call."""
    if _direct is not None and out is None and stream is None:
        r = _direct.product(x, None, wq, wscale, epilogue, out_dtype, workspace)
        if r is not None:
            return _direct_result(r, "cq_linear_i8")
    return _i8_product("cq_linear_i8", x, None, wq, wscale, epilogue, out_dtype, out, workspace,
                       stream)


def moe_i8_workspace_size(T, k, E, H, I) -> int:
    return int(lib().cq_moe_i8_workspace_size(T, k, E, H, I))


def moe_i8_workspace(T, k, E, H, I, device="cuda"):
    """A workspace for cq_moe_i8."""
    n = moe_i8_workspace_size(T, k, E, H, I)
    return torch.empty(max(n, 256), dtype=torch.uint8, device=device)


def cq_moe_i8(tokens, topk_ids, topk_w, w_gu, s_gu, w_dn, s_dn, out_dtype: int = F32,
              route_out=True, combine=True, workspace=None, stream=None):
    """Routed-expert FFN of one MoE layer on INT8 experts:
    w_gu int8 [E][2I][H], s_gu [E][2I], w_dn int8 [E][H][I], s_dn [E][H].
    Returns (route_out, out) as cq_moe_grouped_gemm does."""
    if _direct is not None and combine and stream is None and (route_out is False
                                                               or route_out is None):
        r = _direct.moe(tokens, topk_ids, topk_w, w_gu, s_gu, w_dn, s_dn, out_dtype, workspace)
        if r is not None:
            return None, _direct_result(r, "cq_moe_i8")
    try:
        T, H = tokens.shape
        _, k = topk_ids.shape
        E, _, I = w_dn.shape
    except ValueError:
        raise ValueError("cq_moe_i8: tokens [T][H], topk_ids [T][k], w_gu [E][2I][H] and "
                         "w_dn [E][H][I] expected") from None
    index = tokens.get_device()
    if index < 0:
        _need_cuda(tokens)
    if stream is not None or index != _current_device():
        with _on_device(index, stream):
            return cq_moe_i8(tokens, topk_ids, topk_w, w_gu, s_gu, w_dn, s_dn, out_dtype,
                             route_out, combine, workspace)
    L = _lib or lib()
    dt = _out_dtype(out_dtype)
    pt = _tensor("tokens", tokens, torch.bfloat16, (T, H), index)
    pi = _tensor("topk_ids", topk_ids, torch.int32, (T, k), index)
    if topk_w is None and combine:
        raise ValueError("cq_moe_i8 needs topk_w to combine the routes")
    pk = None if topk_w is None else _tensor("topk_w", topk_w, torch.float32, (T, k), index)
    pgu = _tensor("w_gu", w_gu, torch.int8, (E, 2 * I, H), index)
    psg = _tensor("s_gu", s_gu, torch.float32, (E, 2 * I), index)
    pdn = _tensor("w_dn", w_dn, torch.int8, (E, H, I), index)
    psd = _tensor("s_dn", s_dn, torch.float32, (E, H), index)
    ro = pro = None
    if route_out is True:
        ro = tokens.new_empty((T * k, H), dtype=torch.float32)
        pro = ro.data_ptr()
    elif route_out is not None and route_out is not False:
        ro = route_out
        pro = _tensor("route_out", ro, torch.float32, (T * k, H), index)
    out = po = None
    if combine:
        out = tokens.new_empty((T, H), dtype=dt)
        po = out.data_ptr()
    if workspace is None:
        need = L.cq_moe_i8_workspace_size(T, k, E, H, I)
        workspace = tokens.new_empty(max(need, 256), dtype=torch.uint8)
    pws, nws = _scratch(workspace, index)
    _check(L.cq_moe_i8(pt, T, pi, pk, k, E, pgu, psg, pdn, psd, H, I, out_dtype, pro, po, pws, nws,
                       _raw_stream(index)), "cq_moe_i8")
    return ro, out


def cq_moe_route(logits, k: int, bias=None, scoring: int = SCORE_SOFTMAX, renorm: bool = True,
                 scale: float = 1.0, stream=None):
    """The k experts of each row of router logits [T][E] (float32 or bfloat16):
    (topk_ids int32 [T][k], topk_w float32 [T][k]), as the MoE layers take them."""
    if _direct is not None and stream is None:
        r = _direct.route(logits, k, bias, scoring, renorm, scale)
        if r is not None:
            return _direct_result(r, "cq_moe_route")
    try:
        T, E = logits.shape
    except ValueError:
        raise ValueError("cq_moe_route: logits [T][E] expected") from None
    dt = logits.dtype
    if dt is not torch.float32 and dt is not torch.bfloat16:
        raise ValueError(f"logits are {dt}, expected float32 or bfloat16")
    index = logits.get_device()
    if index < 0:
        _need_cuda(logits)
    if stream is not None or index != _current_device():
        with _on_device(index, stream):
            return cq_moe_route(logits, k, bias, scoring, renorm, scale)
    L = _lib or lib()
    pl = _tensor("logits", logits, dt, (T, E), index)
    pb = None if bias is None else _tensor("bias", bias, torch.float32, (E,), index)
    shape = (T, min(max(k, 0), E))               # a larger k is refused below
    ids = logits.new_empty(shape, dtype=torch.int32)
    w = logits.new_empty(shape, dtype=torch.float32)
    _check(L.cq_moe_route(pl, F32 if dt is torch.float32 else BF16, T, E, k, pb, scoring,
                          1 if renorm else 0, scale, ids.data_ptr(), w.data_ptr(),
                          _raw_stream(index)), "cq_moe_route")
    return ids, w


def device_error(stream=None) -> tuple[int, int]:
    """(status, site) of the device error word; clears it."""
    site = ctypes.c_int(0)
    st = lib().cq_get_device_error(_stream(stream), ctypes.byref(site))
    return int(st), int(site.value)
