"""Argument checks of training with Gate and Up kept as int8 (no GPU: every check
comes before the first HIP call, and the addresses are never read)."""
import pytest
import torch

import swiglu_gated_mlp_amd as sw

OK, NULLP, SHAPE, UNSUP, MISAL, ALIAS, WS = 0, 1, 2, 3, 4, 5, 6
# 1 GiB apart, never dereferenced
A, W1, W2, W3, Y, Q, S, DY, DA, DW1, DW2, DW3, WK, G, U = (0x40000000 * (i + 1) for i in range(15))
BIG = 1 << 29


def forward(a=A, w1=W1, w2=W2, y=Y, q=Q, s=S, M=4, K=64, N=72, ws=WK, nb=BIG):
    return sw.lib().swiglu_train_forward_int8(a, w1, w2, y, q, s, M, K, N, ws, nb, None)


def backward(dy=DY, a=A, w1=W1, w2=W2, q=Q, s=S, da=DA, dw1=DW1, dw2=DW2, M=4, K=64, N=72, ws=WK, nb=BIG):
    return sw.lib().swiglu_train_backward_int8(dy, a, w1, w2, q, s, da, dw1, dw2, M, K, N, ws, nb, None)


def block(dz=DY, a=A, w1=W1, w2=W2, w3=W3, q=Q, s=S, da=DA, dw1=DW1, dw2=DW2, dw3=DW3, M=4, K=64, N=72, ws=WK, nb=BIG):
    return sw.lib().swiglu_mlp_train_backward_int8(dz, a, w1, w2, w3, q, s, da, dw1, dw2, dw3, M, K, N, ws, nb, None)


def values(q=Q, s=S, g=G, u=U, M=4, N=72):
    return sw.lib().swiglu_dequantize_kept_int8(q, s, g, u, M, N, None)


@pytest.mark.parametrize("call", [forward, backward, block])
@pytest.mark.parametrize("shape,want", [
    (dict(M=-1), SHAPE), (dict(K=0), SHAPE), (dict(N=0), SHAPE), (dict(N=-8), SHAPE), (dict(M=1 << 31), SHAPE),
    (dict(K=60), UNSUP), (dict(N=60), UNSUP), (dict(K=(1 << 20) + 8), UNSUP), (dict(N=(1 << 20) + 8), UNSUP),
])
def test_shapes(call, shape, want):
    assert call(**shape) == want
    if "K" not in shape:
        assert values(**shape) == want


@pytest.mark.parametrize("call,names", [
    (forward, "a w1 w2 y q s"), (backward, "dy a w1 w2 q s dw1 dw2"), (block, "dz a w1 w2 w3 q s dw1 dw2 dw3"),
    (values, "q s g u"),
])
def test_null_and_misaligned(call, names):
    for n in names.split():
        assert call(**{n: None}) == NULLP, n
        assert call(**{n: 0x7000000008}) == MISAL, n
    if call is not values:
        assert call(ws=WK + 8) == MISAL


def test_aliasing():
    for call, outs, ins in ((forward, "y q s", (A, W1, W2)), (backward, "da dw1 dw2", (DY, A, W1, W2, Q, S)),
                            (block, "da dw1 dw2 dw3", (DY, A, W1, W2, W3, Q, S)), (values, "g u", (Q, S))):
        for o in outs.split():
            for i in ins:
                assert call(**{o: i + 16}) == ALIAS, (call.__name__, o, hex(i))
            if call is not values:
                assert call(**{o: WK + 32}) == ALIAS
    # codes of 72 columns take three groups, 768 bytes for 4 rows; scales 48
    assert forward(y=Q + 752) == ALIAS and forward(y=S + 32) == ALIAS
    assert values(g=Q + 752) == ALIAS and values(u=S + 32) == ALIAS and values(g=U) == ALIAS
    assert backward(w1=W2, ws=None, nb=0) == WS


def test_workspace():
    L = sw.lib()
    for shape in ((4, 64, 72), (64, 896, 4864), (1, 3584, 18944)):
        need = L.swiglu_train_workspace_bytes_int8(*shape)
        # [dG | dU] and Y
        assert need >= 6 * shape[0] * shape[2] and need >= L.swiglu_train_workspace_bytes(*shape)
        assert need >= L.swiglu_train_forward_workspace_bytes(*shape)
    need = L.swiglu_train_workspace_bytes_int8(4, 64, 72)
    assert block(nb=need - 1) == WS and block(ws=None, nb=0) == WS and backward(ws=None, nb=0) == WS
    assert backward(nb=L.swiglu_train_workspace_bytes(4, 64, 72) - 1) == WS
    for bad in ((0, 64, 64), (4, 60, 64), (4, 64, (1 << 20) + 8), (-1, 64, 64)):
        assert L.swiglu_train_workspace_bytes_int8(*bad) == 0


def test_empty_batch():
    assert forward(M=0, a=None, y=None, q=None) == OK and values(M=0, q=None, g=None) == OK
    assert backward(M=0, dy=None, a=None, q=None, s=None, da=None, dw1=None, dw2=None, ws=None, nb=0) == OK
    assert backward(M=0, dw1=DW1 + 8) == MISAL and backward(M=0, dw2=DW1) == ALIAS
    assert block(M=0, dw3=DW1) == ALIAS and block(M=0, dw3=None) == NULLP and block(dw3=None) == NULLP


def test_binding_refusals():
    bf = dict(dtype=torch.bfloat16)
    a, w, y = torch.zeros(4, 64, **bf), torch.zeros(64, 72, **bf), torch.zeros(4, 72, **bf)
    codes, scales = torch.zeros(4, 3, 2, 32, dtype=torch.int8), torch.zeros(3, 4, 2, **bf)
    w3 = torch.zeros(72, 64, **bf)
    for call in (lambda: sw.swiglu_train_forward_int8(a, w, w),
                 lambda: sw.swiglu_train_backward_int8(y, a, w, w, codes, scales),
                 lambda: sw.swiglu_mlp_train_backward_int8(a, a, w, w, w3, codes, scales),
                 lambda: sw.swiglu_dequantize_kept_int8(codes, scales, 72)):
        with pytest.raises(ValueError, match="GPU tensor"):
            call()
    with pytest.raises(ValueError, match="codes must be"):
        sw.swiglu_train_backward_int8(y, a, w, w, codes[:, :2], scales)
    with pytest.raises(ValueError, match="scales must be"):
        sw.swiglu_mlp_train_backward_int8(a, a, w, w, w3, codes, scales.transpose(0, 1))
    with pytest.raises(ValueError, match="codes must be"):
        sw.swiglu_dequantize_kept_int8(codes, scales, 104)
    with pytest.raises(ValueError, match="keep must be"):
        sw.swiglu(a, w, w, keep="fp8")
    with pytest.raises(ValueError, match="keep must be"):
        sw.swiglu_mlp(a, w, w, w3, keep="")
    with pytest.raises(ValueError, match="recompute keeps nothing"):
        sw.swiglu(a, w, w, recompute=True, keep="int8")
