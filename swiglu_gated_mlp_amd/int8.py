"""The gated MLP from int8 operands with a scale for each token and channel:
argument marshalling for the C entry points of the same names
(``include/swiglu.h``)."""
from __future__ import annotations

import torch

from . import _check, _empty, _raw_stream, _scratch, _shape, _stream, _tensor, lib

_need: dict = {}


def _cached(fn, *args):
    key = (fn, args)
    need = _need.get(key)
    if need is None:
        if len(_need) >= 4096:
            _need.clear()
        need = _need[key] = fn(*args)
    return need


def swiglu_packed_bytes_int8(K: int, N: int) -> int:
    return int(lib().swiglu_packed_bytes_int8(K, N))


def swiglu_gemm_packed_bytes_int8(K: int, N: int) -> int:
    return int(lib().swiglu_gemm_packed_bytes_int8(K, N))


def swiglu_workspace_bytes_int8(M: int, K: int, N: int) -> int:
    return int(lib().swiglu_workspace_bytes_int8(M, K, N))


def swiglu_gemm_workspace_bytes_int8(M: int, K: int, N: int) -> int:
    return int(lib().swiglu_gemm_workspace_bytes_int8(M, K, N))


def swiglu_mlp_workspace_bytes_int8(M: int, K: int, N: int) -> int:
    return int(lib().swiglu_mlp_workspace_bytes_int8(M, K, N))


# Small products are bound by the host (a launch 2.2 us, an output 1.3 us), so what a
# call asks of torch it asks once, and in its cheapest form: quantized rows and their
# product 15.3 us of host time, with general checks and torch.cuda's functions 19.6 us.
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _here() -> int:
    """The current GPU: plans, streams and launches are its own."""
    return _current_device() if torch.cuda.is_initialized() else -2   # a CPU tensor's is -1


def _stream_at(here: int, stream) -> int:
    return _raw_stream(here) if stream is None and _raw_stream is not None else _stream(stream)


def _dev(t, dtype, name: str, here: int) -> int:
    """A contiguous tensor of dtype on the current GPU."""
    if isinstance(t, torch.Tensor) and t.dtype is dtype and t.is_contiguous() and t.get_device() == here:
        return t.data_ptr()
    _tensor(t, name)
    if t.device.type != "cuda":
        raise ValueError("%s must be a GPU tensor (got %s)" % (name, t.device))
    if t.dtype != dtype:
        raise TypeError("%s must be %s (got %s)" % (name, str(dtype)[6:], t.dtype))
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)
    raise ValueError("%s is on %s, the current device is %d" % (name, t.device, here))


# What is no tensor lacks these attributes, or fails a comparison: only then is its type
# looked at (asked first, it took 0.4 us a call).
def _vector(t, n: int, name: str, here: int) -> int:
    try:
        if t.dtype is torch.float32 and t.shape == (n,) and t.is_contiguous() and t.get_device() == here:
            return t.data_ptr()
    except AttributeError:
        pass
    _shape(t, (n,), name)
    return _dev(t, torch.float32, name, here)


def _matrix(t, name: str):
    try:
        flat = t.dim() == 2
    except AttributeError:
        _tensor(t, name)
        raise
    if not flat:
        raise ValueError("%s must be a matrix (got %s)" % (name, list(t.shape)))
    return t.shape


def _length(t, name: str) -> int:
    try:
        n, = t.shape
    except (AttributeError, ValueError):
        _tensor(t, name)
        raise ValueError("%s must be a vector (got %s)" % (name, list(t.shape)))
    return n


def _space(workspace, need: int, device, s: int, here: int):
    """The workspace's address and bytes."""
    ws, ws_bytes = _scratch(workspace, need, device, s)
    if ws is None:
        return 0, 0
    if ws.get_device() != here:
        raise ValueError("the workspace is on %s, the current device is %d" % (ws.device, here))
    return ws.data_ptr(), ws_bytes


def _out(t, shape, dtype, device, s: int, stream):
    if t is not None:
        return t
    return torch.empty(*shape, dtype=dtype, device=device) if stream is None else _empty(shape, dtype, device, s)


def _quantize(fn: str, X, Q, scales, n: int, stream):
    R, C = X.shape
    _shape(Q, (R, C), "Q")
    _shape(scales, (n,), "scales")
    here = _here()
    x = _dev(X, torch.bfloat16, "A" if fn == "swiglu_quantize_rows_int8" else "W", here)
    s, device = _stream_at(here, stream), X.device
    Q = _out(Q, (R, C), torch.int8, device, s, stream)
    scales = _out(scales, (n,), torch.float32, device, s, stream)
    _check(fn, getattr(lib(), fn)(x, _dev(Q, torch.int8, "Q", here), _dev(scales, torch.float32, "scales", here), R, C,
                                  s))
    return Q, scales


def swiglu_quantize_rows_int8(A: torch.Tensor, Q: torch.Tensor | None = None, scales: torch.Tensor | None = None,
                              stream=None):
    """A [M,K] bf16 as (codes int8 [M,K], scales fp32 [M]), a scale for each row."""
    return _quantize("swiglu_quantize_rows_int8", A, Q, scales, _matrix(A, "A")[0], stream)


def swiglu_quantize_columns_int8(W: torch.Tensor, Q: torch.Tensor | None = None, scales: torch.Tensor | None = None,
                                 stream=None):
    """W [K,N] bf16 as (codes int8 [K,N], scales fp32 [N]), a scale for each column."""
    return _quantize("swiglu_quantize_columns_int8", W, Q, scales, _matrix(W, "W")[1], stream)


def _packed(fn: str, sizer, weights, Wp, name: str, stream):
    (W, first), *rest = weights
    K, N = _matrix(W, first)
    for t, n in rest:
        _shape(t, (K, N), n)
    nbytes = _cached(sizer, K, N)
    if nbytes == 0:
        raise ValueError("invalid int8 weight shape [%d,%d] (K must be a multiple of 16, N of 8)" % (K, N))
    here = _here()
    ptrs, s = [_dev(t, torch.int8, n, here) for t, n in weights], _stream_at(here, stream)
    if Wp is not None:
        _tensor(Wp, name)
        if Wp.numel() < nbytes:
            raise ValueError("%s too small: need %d bytes" % (name, nbytes))
    Wp = _out(Wp, (nbytes,), torch.int8, W.device, s, stream)
    _check(fn, getattr(lib(), fn)(*ptrs, _dev(Wp, torch.int8, name, here), K, N, s))
    return Wp


def swiglu_pack_weights_int8(W1: torch.Tensor, W2: torch.Tensor, Wp: torch.Tensor | None = None,
                             stream=None) -> torch.Tensor:
    """Pack the codes W1, W2 int8 [K,N] for swiglu_fused_packed_int8."""
    return _packed("swiglu_pack_weights_int8", swiglu_packed_bytes_int8, [(W1, "W1"), (W2, "W2")], Wp, "Wp", stream)


def swiglu_gemm_pack_weight_int8(W: torch.Tensor, Wg: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Pack one weight's codes W int8 [K,N] for swiglu_gemm_packed_int8."""
    return _packed("swiglu_gemm_pack_weight_int8", swiglu_gemm_packed_bytes_int8, [(W, "W")], Wg, "Wg", stream)


def _weight_at_least(W, need: int, K: int, N: int, name: str) -> None:
    try:
        n = W.numel()
    except AttributeError:
        _tensor(W, name)
        raise
    if need == 0:
        raise ValueError("invalid int8 weight shape [%d,%d]" % (K, N))
    if n < need:
        raise ValueError("%s holds %d codes; a packed int8 [%d,%d] weight needs %d" % (name, n, K, N, need))


def _sizes(weights, need, M: int, K: int, N: int, here: int):
    """(codes of the packed weights, workspace bytes on this device) of a call."""
    key = (need, M, K, N, here)
    sizes = _need.get(key)
    if sizes is None:
        if len(_need) >= 4096:
            _need.clear()
        sizes = _need[key] = (weights(K, N), need(M, K, N))
    return sizes


def swiglu_fused_packed_int8(A: torch.Tensor, sa: torch.Tensor, Wp: torch.Tensor, s1: torch.Tensor, s2: torch.Tensor,
                             Y: torch.Tensor | None = None, workspace=None, stream=None) -> torch.Tensor:
    """Y = SiLU(G) * U bf16 [M,N] from the codes A int8 [M,K], their rows' scales sa
    [M], the packed codes of W1 and W2 and their columns' scales s1, s2 [N] (fp32)."""
    (M, K), N, here = _matrix(A, "A"), _length(s1, "s1"), _here()
    least, need = _sizes(swiglu_packed_bytes_int8, swiglu_workspace_bytes_int8, M, K, N, here)
    _weight_at_least(Wp, least, K, N, "Wp")
    _shape(Y, (M, N), "Y")
    a, r, w = _dev(A, torch.int8, "A", here), _vector(sa, M, "sa", here), _dev(Wp, torch.int8, "Wp", here)
    p1, p2 = _vector(s1, N, "s1", here), _vector(s2, N, "s2", here)
    s, device = _stream_at(here, stream), A.device
    Y = _out(Y, (M, N), torch.bfloat16, device, s, stream)
    ws, ws_bytes = _space(workspace, need, device, s, here)
    _check("swiglu_fused_packed_int8", lib().swiglu_fused_packed_int8(
        a, r, w, p1, p2, _dev(Y, torch.bfloat16, "Y", here), M, K, N, ws, ws_bytes, s))
    return Y


def swiglu_gemm_packed_int8(A: torch.Tensor, sa: torch.Tensor, Wg: torch.Tensor, sw: torch.Tensor,
                            C: torch.Tensor | None = None, workspace=None, stream=None) -> torch.Tensor:
    """C = A @ W bf16 [M,N] from the codes A int8 [M,K], sa [M], one weight's packed
    codes and its columns' scales sw [N] (fp32)."""
    (M, K), N, here = _matrix(A, "A"), _length(sw, "sw"), _here()
    least, need = _sizes(swiglu_gemm_packed_bytes_int8, swiglu_gemm_workspace_bytes_int8, M, K, N, here)
    _weight_at_least(Wg, least, K, N, "Wg")
    _shape(C, (M, N), "C")
    a, r, w = _dev(A, torch.int8, "A", here), _vector(sa, M, "sa", here), _dev(Wg, torch.int8, "Wg", here)
    p = _vector(sw, N, "sw", here)
    s, device = _stream_at(here, stream), A.device
    C = _out(C, (M, N), torch.bfloat16, device, s, stream)
    ws, ws_bytes = _space(workspace, need, device, s, here)
    _check("swiglu_gemm_packed_int8", lib().swiglu_gemm_packed_int8(
        a, r, w, p, _dev(C, torch.bfloat16, "C", here), M, K, N, ws, ws_bytes, s))
    return C


def swiglu_mlp_packed_int8(A: torch.Tensor, Wp: torch.Tensor, s1: torch.Tensor, s2: torch.Tensor, W3g: torch.Tensor,
                           s3: torch.Tensor, Y: torch.Tensor | None = None, Z: torch.Tensor | None = None,
                           workspace=None, stream=None):
    """The gated MLP block from A bf16 [M,K]: its rows quantized, Y = SiLU(G) * U
    (bf16), Y's rows quantized, Z = Y @ W3.  Returns (Y, Z)."""
    (M, K), N, here = _matrix(A, "A"), _length(s1, "s1"), _here()
    least, need = _sizes(swiglu_packed_bytes_int8, swiglu_mlp_workspace_bytes_int8, M, K, N, here)
    _weight_at_least(Wp, least, K, N, "Wp")
    _weight_at_least(W3g, _cached(swiglu_gemm_packed_bytes_int8, N, K), N, K, "W3g")
    _shape(Y, (M, N), "Y")
    _shape(Z, (M, K), "Z")
    bf16 = torch.bfloat16
    a, wp, w3 = _dev(A, bf16, "A", here), _dev(Wp, torch.int8, "Wp", here), _dev(W3g, torch.int8, "W3g", here)
    p1, p2, p3 = _vector(s1, N, "s1", here), _vector(s2, N, "s2", here), _vector(s3, K, "s3", here)
    s, device = _stream_at(here, stream), A.device
    Y = _out(Y, (M, N), bf16, device, s, stream)
    Z = _out(Z, (M, K), bf16, device, s, stream)
    ws, ws_bytes = _space(workspace, need, device, s, here)
    st = lib().swiglu_mlp_packed_int8(a, wp, p1, p2, w3, p3, _dev(Y, bf16, "Y", here), _dev(Z, bf16, "Z", here), M, K,
                                      N, ws, ws_bytes, s)
    _check("swiglu_mlp_packed_int8", st)
    return Y, Z
