"""Training entry points of the gated MLP: the forward pass that keeps Gate and
Up, the gradients of the SwiGLU product and of the whole block, and autograd
functions on top of them.

The swiglu_* functions marshal arguments for the C entry points of the same
names (``include/swiglu.h``).  ``swiglu`` and ``swiglu_mlp`` are differentiable:
their forward and backward passes are those entry points.

Capturing a backward pass into a graph: take the gradients with
``torch.autograd.grad``, or let no eager graph of the same leaves live.  The
accumulation into a leaf runs on the stream where it was first recorded, and a
capture that has to wait for that stream ends the process.
"""
from __future__ import annotations

import torch

from . import (_check, _dev_bf16, _new, _ptr, _scratch, _shape, _stream, lib, swiglu_fused,
               swiglu_gemm_bf16)

_need: dict = {}


def swiglu_train_workspace_bytes(M: int, K: int, N: int) -> int:
    return int(lib().swiglu_train_workspace_bytes(M, K, N))


def swiglu_train_forward_workspace_bytes(M: int, K: int, N: int) -> int:
    return int(lib().swiglu_train_forward_workspace_bytes(M, K, N))


def _cached(fn, M: int, K: int, N: int, device) -> int:
    key = (fn, M, K, N, device.index)
    need = _need.get(key)
    if need is None:
        if len(_need) >= 4096:
            _need.clear()
        need = _need[key] = fn(M, K, N)
    return need


def _weights(A, W1, W2):
    if A.dim() != 2 or W1.dim() != 2:
        raise ValueError("A must be [M,K] and W1, W2 [K,N]")
    M, K = A.shape
    N = W1.shape[1]
    _shape(W1, (K, N), "W1")
    _shape(W2, (K, N), "W2")
    return M, K, N


def swiglu_train_forward(A: torch.Tensor, W1: torch.Tensor, W2: torch.Tensor, Y: torch.Tensor | None = None,
                         G: torch.Tensor | None = None, U: torch.Tensor | None = None, workspace=None, stream=None):
    """Y = SiLU(G) * U with G = A @ W1, U = A @ W2 kept: returns (Y, G, U), bf16 [M,N]."""
    M, K, N = _weights(A, W1, W2)
    for t, name in ((Y, "Y"), (G, "G"), (U, "U")):
        _shape(t, (M, N), name)
    a, w1, w2 = _dev_bf16(A, "A"), _dev_bf16(W1, "W1"), _dev_bf16(W2, "W2")
    s = _stream(stream)
    Y = _new((M, N), A.device, s, stream) if Y is None else Y
    G = _new((M, N), A.device, s, stream) if G is None else G
    U = _new((M, N), A.device, s, stream) if U is None else U
    ws, ws_bytes = _scratch(workspace, _cached(swiglu_train_forward_workspace_bytes, M, K, N, A.device), A.device, s)
    st = lib().swiglu_train_forward(a, w1, w2, _dev_bf16(Y, "Y"), _dev_bf16(G, "G"), _dev_bf16(U, "U"), M, K, N,
                                    _ptr(ws), ws_bytes, s)
    _check("swiglu_train_forward", st)
    return Y, G, U


def _grads(needed: bool, given, shape, names, device, s: int, stream):
    """Gradient outputs: the caller's, new ones, or (not needed) None."""
    if not needed:
        if any(t is not None for t in given):
            raise ValueError("%s given but not requested" % ", ".join(names))
        return [None] * len(given)
    out = []
    for t, name in zip(given, names):
        _shape(t, shape, name)
        out.append(_new(shape, device, s, stream) if t is None else t)
    return out


def swiglu_train_backward(dY: torch.Tensor, A: torch.Tensor, W1: torch.Tensor, W2: torch.Tensor,
                          G: torch.Tensor | None = None, U: torch.Tensor | None = None,
                          dA: torch.Tensor | None = None, dW1: torch.Tensor | None = None,
                          dW2: torch.Tensor | None = None, need_dA: bool = True, need_dW: bool = True, workspace=None,
                          stream=None):
    """Gradients of Y = SiLU(A @ W1) * (A @ W2): returns (dA, dW1, dW2), None for
    those not requested.  G and U are those of swiglu_train_forward, or None:
    they are then computed again from A, W1, W2 and not kept."""
    M, K, N = _weights(A, W1, W2)
    for t, name in ((dY, "dY"), (G, "G"), (U, "U")):
        _shape(t, (M, N), name)
    if (G is None) != (U is None):
        raise ValueError("G and U go together")
    ins = [_dev_bf16(t, n) for t, n in ((dY, "dY"), (A, "A"), (W1, "W1"), (W2, "W2"))]
    kept = [0 if t is None else _dev_bf16(t, n) for t, n in ((G, "G"), (U, "U"))]
    s = _stream(stream)
    dA, = _grads(need_dA, (dA,), (M, K), ("dA",), A.device, s, stream)
    dW1, dW2 = _grads(need_dW, (dW1, dW2), (K, N), ("dW1", "dW2"), A.device, s, stream)
    ws, ws_bytes = _scratch(workspace, _cached(swiglu_train_workspace_bytes, M, K, N, A.device), A.device, s)
    outs = [0 if t is None else _dev_bf16(t, n) for t, n in ((dA, "dA"), (dW1, "dW1"), (dW2, "dW2"))]
    st = lib().swiglu_train_backward(*ins, *kept, *outs, M, K, N, _ptr(ws), ws_bytes, s)
    _check("swiglu_train_backward", st)
    return dA, dW1, dW2


def swiglu_mlp_train_backward(dZ: torch.Tensor, A: torch.Tensor, W1: torch.Tensor, W2: torch.Tensor,
                              W3: torch.Tensor, G: torch.Tensor, U: torch.Tensor, Y: torch.Tensor,
                              dA: torch.Tensor | None = None, dW1: torch.Tensor | None = None,
                              dW2: torch.Tensor | None = None, dW3: torch.Tensor | None = None,
                              need_dA: bool = True, need_dW: bool = True, workspace=None, stream=None):
    """Gradients of the block Z = (SiLU(G) * U) @ W3 from dZ [M,K]: returns
    (dA, dW1, dW2, dW3), None for those not requested (Y may be None without the
    weight gradients)."""
    M, K, N = _weights(A, W1, W2)
    _shape(dZ, (M, K), "dZ")
    _shape(W3, (N, K), "W3")
    for t, name in ((G, "G"), (U, "U"), (Y, "Y")):
        _shape(t, (M, N), name)
    if need_dW and Y is None:
        raise ValueError("Y is needed for the gradient of W3")
    ins = [_dev_bf16(t, n) for t, n in ((dZ, "dZ"), (A, "A"), (W1, "W1"), (W2, "W2"), (W3, "W3"), (G, "G"), (U, "U"))]
    y = _dev_bf16(Y, "Y") if Y is not None else 0
    s = _stream(stream)
    dA, = _grads(need_dA, (dA,), (M, K), ("dA",), A.device, s, stream)
    dW1, dW2 = _grads(need_dW, (dW1, dW2), (K, N), ("dW1", "dW2"), A.device, s, stream)
    dW3, = _grads(need_dW, (dW3,), (N, K), ("dW3",), A.device, s, stream)
    ws, ws_bytes = _scratch(workspace, _cached(swiglu_train_workspace_bytes, M, K, N, A.device), A.device, s)
    outs = [0 if t is None else _dev_bf16(t, n)
            for t, n in ((dA, "dA"), (dW1, "dW1"), (dW2, "dW2"), (dW3, "dW3"))]
    st = lib().swiglu_mlp_train_backward(*ins, y, *outs, M, K, N, _ptr(ws), ws_bytes, s)
    _check("swiglu_mlp_train_backward", st)
    return dA, dW1, dW2, dW3


# ---------------------------------------------------------------------------
# autograd
# ---------------------------------------------------------------------------
def _rows(t: torch.Tensor) -> torch.Tensor:
    return t.reshape(-1, t.shape[-1]).contiguous()


class _Swiglu(torch.autograd.Function):
    @staticmethod
    def forward(ctx, A, W1, W2, recompute):
        rows = _rows(A)
        if recompute:
            Y, kept = swiglu_fused(rows, W1, W2), ()
        else:
            Y, *kept = swiglu_train_forward(rows, W1, W2)
        ctx.shape = A.shape
        ctx.save_for_backward(rows, W1, W2, *kept)
        return Y.view(*A.shape[:-1], W1.shape[1])

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dY):
        rows, W1, W2, *kept = ctx.saved_tensors
        need_a, need_1, need_2 = ctx.needs_input_grad[:3]
        dA, dW1, dW2 = swiglu_train_backward(_rows(dY), rows, W1, W2, *kept, need_dA=need_a,
                                             need_dW=need_1 or need_2)
        return (dA.view(ctx.shape) if need_a else None, dW1 if need_1 else None, dW2 if need_2 else None, None)


class _SwigluMlp(torch.autograd.Function):
    @staticmethod
    def forward(ctx, A, W1, W2, W3):
        rows = _rows(A)
        Y, G, U = swiglu_train_forward(rows, W1, W2)
        Z = swiglu_gemm_bf16(Y, W3)
        ctx.shape = A.shape
        ctx.save_for_backward(rows, W1, W2, W3, G, U, Y)
        return Z.view(*A.shape[:-1], W3.shape[1])

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dZ):
        need = ctx.needs_input_grad
        grads = swiglu_mlp_train_backward(_rows(dZ), *ctx.saved_tensors, need_dA=need[0], need_dW=any(need[1:]))
        dA = grads[0].view(ctx.shape) if need[0] else None
        return (dA,) + tuple(g if n else None for g, n in zip(grads[1:], need[1:]))


def swiglu(A: torch.Tensor, W1: torch.Tensor, W2: torch.Tensor, recompute: bool = False) -> torch.Tensor:
    """Differentiable Y = SiLU(A @ W1) * (A @ W2), A [..., K].  Keeps Gate and Up
    (4 M N bytes) for the backward pass, or (recompute) computes them again in
    it for 4 M K N more operations.  Without recompute they are written in every
    call, also where no gradient is wanted (swiglu_fused writes Y alone)."""
    return _Swiglu.apply(A, W1, W2, recompute)


def swiglu_mlp(A: torch.Tensor, W1: torch.Tensor, W2: torch.Tensor, W3: torch.Tensor) -> torch.Tensor:
    """Differentiable gated MLP block Z = (SiLU(A @ W1) * (A @ W2)) @ W3, A [..., K],
    W3 [N,K] (any [N, ...] where no gradient is wanted)."""
    if torch.is_grad_enabled() and any(t.requires_grad for t in (A, W1, W2, W3)):
        _shape(W3, (W1.shape[1], A.shape[-1]), "W3")
    return _SwigluMlp.apply(A, W1, W2, W3)
