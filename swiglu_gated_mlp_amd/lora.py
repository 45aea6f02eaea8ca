"""Low-rank adapters of many requests beside the packed products: argument
marshalling for the C entry points of the same names (``include/swiglu.h``)."""
from __future__ import annotations

import torch

from . import (_check, _dev_bf16, _gemm_packed_at_least, _new, _packed_at_least, _ptr, _scratch, _shape, _stream, lib)

_need: dict = {}


def _cached(fn, *args, device=None) -> int:
    key = (fn, args, None if device is None else device.index)
    need = _need.get(key)
    if need is None:
        if len(_need) >= 4096:
            _need.clear()
        need = _need[key] = fn(*args)
    return need


def swiglu_lora_packed_bytes(K: int, N: int, adapters: int, rank: int) -> int:
    return int(lib().swiglu_lora_packed_bytes(K, N, adapters, rank))


def swiglu_gemm_lora_packed_bytes(K: int, N: int, adapters: int, rank: int) -> int:
    return int(lib().swiglu_gemm_lora_packed_bytes(K, N, adapters, rank))


def swiglu_lora_workspace_bytes(M: int, K: int, N: int, rank: int) -> int:
    return int(lib().swiglu_lora_workspace_bytes(M, K, N, rank))


def swiglu_gemm_lora_workspace_bytes(M: int, K: int, N: int, rank: int) -> int:
    return int(lib().swiglu_gemm_lora_workspace_bytes(M, K, N, rank))


def _factors(pairs):
    """Checked pointers of (La, Lb) pairs, and (adapters, K, rank, N)."""
    La, Lb = pairs[0][0], pairs[0][2]
    if La.dim() != 3 or Lb.dim() != 3:
        raise ValueError("adapters are La [adapters,K,rank] and Lb [adapters,rank,N]")
    L, K, r = La.shape
    N = Lb.shape[2]
    ptrs = []
    for a, an, b, bn in pairs:
        _shape(a, (L, K, r), an)
        _shape(b, (L, r, N), bn)
    for a, an, b, bn in pairs:
        ptrs += [_dev_bf16(a, an), _dev_bf16(b, bn)]
    return ptrs, (L, K, r, N)


def _pack(fn: str, sizer, pairs, Lp, stream):
    ptrs, (L, K, r, N) = _factors(pairs)
    nbytes = sizer(K, N, L, r)
    if nbytes == 0:
        raise ValueError("invalid adapters: %d of [%d,%d] x [%d,%d]" % (L, K, r, r, N))
    s = _stream(stream)
    if Lp is None:
        Lp = _new(nbytes // 2, pairs[0][0].device, s, stream)
    elif Lp.numel() * Lp.element_size() < nbytes:
        raise ValueError("Lp too small: need %d bytes" % nbytes)
    _check(fn, getattr(lib(), fn)(*ptrs, _dev_bf16(Lp, "Lp"), K, N, L, r, s))
    return Lp


def swiglu_lora_pack(La1: torch.Tensor, Lb1: torch.Tensor, La2: torch.Tensor, Lb2: torch.Tensor,
                     Lp: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Pack the Gate adapters La1 [adapters,K,rank], Lb1 [adapters,rank,N] and the
    Up adapters La2, Lb2 for swiglu_fused_packed_lora."""
    return _pack("swiglu_lora_pack", swiglu_lora_packed_bytes, [(La1, "La1", Lb1, "Lb1"), (La2, "La2", Lb2, "Lb2")],
                 Lp, stream)


def swiglu_gemm_lora_pack(La: torch.Tensor, Lb: torch.Tensor, Lp: torch.Tensor | None = None,
                          stream=None) -> torch.Tensor:
    """Pack one projection's adapters for swiglu_gemm_packed_lora."""
    return _pack("swiglu_gemm_lora_pack", swiglu_gemm_lora_packed_bytes, [(La, "La", Lb, "Lb")], Lp, stream)


def _dev_vec(t: torch.Tensor, dtype, n, name: str) -> int:
    if not isinstance(t, torch.Tensor) or t.dtype != dtype:
        raise TypeError("%s must be a %s tensor" % (name, dtype))
    if t.device.type != "cuda":
        raise ValueError("%s must be a GPU tensor (got %s)" % (name, t.device))
    if t.dim() != 1 or not t.is_contiguous() or (n is not None and t.shape[0] != n):
        raise ValueError("%s must be a contiguous vector%s (got %s)" % (name, "" if n is None else " of %d" % n,
                                                                      list(t.shape)))
    return t.data_ptr()


def _call(fn: str, need_fn, sizer, A, W, Lp, ids, scales, N, rank, out, name, workspace, stream):
    M, K = A.shape
    a, lp = _dev_bf16(A, "A"), _dev_bf16(Lp, "Lp")
    idp, scp = _dev_vec(ids, torch.int32, M, "ids"), _dev_vec(scales, torch.float32, None, "scales")
    L = scales.shape[0]
    need_lp = _cached(sizer, K, N, L, rank)
    if need_lp == 0:
        raise ValueError("invalid adapters: %d of rank %s beside a [%d,%d] weight" % (L, rank, K, N))
    if Lp.numel() * Lp.element_size() < need_lp:
        raise ValueError("Lp holds %d bytes; %d packed adapters of rank %d need %d"
                         % (Lp.numel() * Lp.element_size(), L, rank, need_lp))
    _shape(out, (M, N), name)
    s = _stream(stream)
    out = _new((M, N), A.device, s, stream) if out is None else out
    ws, ws_bytes = _scratch(workspace, _cached(need_fn, M, K, N, rank, device=A.device), A.device, s)
    st = getattr(lib(), fn)(a, _dev_bf16(W, "W"), lp, idp, scp, _dev_bf16(out, name), M, K, N, L, rank, _ptr(ws),
                            ws_bytes, s)
    _check(fn, st)
    return out


def swiglu_fused_packed_lora(A: torch.Tensor, Wp: torch.Tensor, Lp: torch.Tensor, ids: torch.Tensor,
                             scales: torch.Tensor, N: int, rank: int, Y: torch.Tensor | None = None, workspace=None,
                             stream=None) -> torch.Tensor:
    """Y = SiLU(G) * U where row m's G and U have adapter ids[m] (int32 [M], -1:
    none) of the packed adapters Lp (scales: fp32, one an adapter) added to
    A @ W1 and A @ W2; Wp as for swiglu_fused_packed."""
    _packed_at_least(Wp, A.shape[1], N)
    return _call("swiglu_fused_packed_lora", swiglu_lora_workspace_bytes, swiglu_lora_packed_bytes, A, Wp, Lp, ids,
                 scales, N, rank, Y, "Y", workspace, stream)


def swiglu_gemm_packed_lora(A: torch.Tensor, Wg: torch.Tensor, Lp: torch.Tensor, ids: torch.Tensor,
                            scales: torch.Tensor, N: int, rank: int, C: torch.Tensor | None = None, workspace=None,
                            stream=None) -> torch.Tensor:
    """C = A @ W with row m's adapter ids[m] added; Wg as for swiglu_gemm_packed."""
    _gemm_packed_at_least(Wg, A.shape[1], N)
    return _call("swiglu_gemm_packed_lora", swiglu_gemm_lora_workspace_bytes, swiglu_gemm_lora_packed_bytes, A, Wg,
                 Lp, ids, scales, N, rank, C, "C", workspace, stream)
