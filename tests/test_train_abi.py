"""Argument checks of the training entry points (no GPU: every check comes
before the first HIP call, and the addresses are never read)."""
import pytest
import torch

import swiglu_gated_mlp_amd as sw

OK, NULLP, SHAPE, UNSUP, MISAL, ALIAS, WS = 0, 1, 2, 3, 4, 5, 6
# 1 GiB apart, never dereferenced
A, W1, W2, W3, Y, G, U, DY, DA, DW1, DW2, DW3, WK = (0x40000000 * (i + 1) for i in range(13))
BIG = 1 << 29


def forward(a=A, w1=W1, w2=W2, y=Y, g=G, u=U, M=4, K=64, N=72, ws=WK, nb=BIG):
    return sw.lib().swiglu_train_forward(a, w1, w2, y, g, u, M, K, N, ws, nb, None)


def backward(dy=DY, a=A, w1=W1, w2=W2, g=G, u=U, da=DA, dw1=DW1, dw2=DW2, M=4, K=64, N=72, ws=WK, nb=BIG):
    return sw.lib().swiglu_train_backward(dy, a, w1, w2, g, u, da, dw1, dw2, M, K, N, ws, nb, None)


def block(dz=DY, a=A, w1=W1, w2=W2, w3=W3, g=G, u=U, y=Y, da=DA, dw1=DW1, dw2=DW2, dw3=DW3, M=4, K=64, N=72, ws=WK,
          nb=BIG):
    return sw.lib().swiglu_mlp_train_backward(dz, a, w1, w2, w3, g, u, y, da, dw1, dw2, dw3, M, K, N, ws, nb, None)


@pytest.mark.parametrize("call", [forward, backward, block])
@pytest.mark.parametrize("shape,want", [
    (dict(M=-1), SHAPE), (dict(K=0), SHAPE), (dict(N=0), SHAPE), (dict(N=-8), SHAPE), (dict(M=1 << 31), SHAPE),
    (dict(K=60), UNSUP), (dict(N=60), UNSUP), (dict(K=(1 << 20) + 8), UNSUP), (dict(N=(1 << 20) + 8), UNSUP),
])
def test_shapes(call, shape, want):
    assert call(**shape) == want


@pytest.mark.parametrize("call,names", [
    (forward, "a w1 w2 y g u"), (backward, "dy a w1 w2 dw1 dw2"), (block, "dz a w1 w2 w3 g u y dw1 dw2 dw3"),
])
def test_null_and_misaligned(call, names):
    for n in names.split():
        assert call(**{n: None}) == NULLP, n
        assert call(**{n: 0x7000000008}) == MISAL, n
    assert call(ws=WK + 8) == MISAL


def test_optional_pointers():
    # Gate and Up go together, and so do the weight gradients
    assert backward(g=None) == NULLP and backward(u=None) == NULLP
    # with none of the optional ones, the workspace is the last check
    assert backward(g=None, u=None, da=None, dw1=None, dw2=None, ws=None, nb=0) == WS
    assert block(y=None, da=None, dw1=None, dw2=None, dw3=None, ws=None, nb=0) == WS
    assert block(dw3=None) == NULLP


def test_aliasing():
    for call, outs, ins in ((forward, "y g u", (A, W1, W2)), (backward, "da dw1 dw2", (DY, A, W1, W2, G, U)),
                            (block, "da dw1 dw2 dw3", (DY, A, W1, W2, W3, G, U, Y))):
        for o in outs.split():
            for i in ins:
                assert call(**{o: i + 16}) == ALIAS, (call.__name__, o, hex(i))
            assert call(**{o: WK + 32}) == ALIAS
    assert forward(y=G) == ALIAS and backward(dw1=DW2) == ALIAS and block(dw3=DW1) == ALIAS
    # inputs may overlap: W1 == W2 passes on to the workspace check
    assert backward(w1=W2, ws=None, nb=0) == WS


def test_workspace():
    L = sw.lib()
    for shape in ((4, 64, 72), (64, 896, 4864), (1, 3584, 18944)):
        need = L.swiglu_train_workspace_bytes(*shape)
        assert need >= 4 * shape[0] * shape[2]
        assert need >= L.swiglu_train_forward_workspace_bytes(*shape)
    need = L.swiglu_train_workspace_bytes(4, 64, 72)
    assert backward(nb=need - 1) == WS and block(nb=need - 1) == WS
    assert L.swiglu_train_workspace_bytes(0, 64, 64) == 0
    assert L.swiglu_train_workspace_bytes(4, 60, 64) == 0
    assert L.swiglu_train_workspace_bytes(4, 64, (1 << 20) + 8) == 0
    assert L.swiglu_train_forward_workspace_bytes(-1, 64, 64) == 0


def test_empty_batch():
    assert forward(M=0, a=None, y=None) == OK
    assert backward(M=0, dy=None, a=None, g=None, u=None, da=None, dw1=None, dw2=None, ws=None, nb=0) == OK
    assert backward(M=0, dw1=DW1 + 8) == MISAL
    assert backward(M=0, dw2=DW1) == ALIAS
    assert block(M=0, dw3=DW1) == ALIAS
    assert block(M=0, dw3=None) == NULLP


def test_binding_refusals():
    bf = dict(dtype=torch.bfloat16)
    a, w = torch.zeros(4, 64, **bf), torch.zeros(64, 72, **bf)
    y = torch.zeros(4, 72, **bf)
    with pytest.raises(ValueError, match="GPU tensor"):
        sw.swiglu_train_forward(a, w, w)
    with pytest.raises(ValueError, match="W2 must be"):
        sw.swiglu_train_forward(a, w, w[:, :64])
    with pytest.raises(ValueError, match=r"A must be \[M,K\]"):
        sw.swiglu_train_forward(a[0], w, w)
    with pytest.raises(ValueError, match="G must be"):
        sw.swiglu_train_backward(y, a, w, w, y[:2], y)
    with pytest.raises(ValueError, match="go together"):
        sw.swiglu_train_backward(y, a, w, w, y, None)
    with pytest.raises(ValueError, match="dZ must be"):
        sw.swiglu_mlp_train_backward(y, a, w, w, w.t(), y, y, y)
    with pytest.raises(ValueError, match="Y is needed"):
        sw.swiglu_mlp_train_backward(a, a, w, w, torch.zeros(72, 64, **bf), y, y, None)


def test_plan_probe():
    assert len(sw.TRAIN_LAUNCHES) == 7
    for launch in sw.TRAIN_LAUNCHES:
        for shape in ((1, 8, 8), (333, 896, 4864), (4096, 3584, 18944)):
            plan = sw.swiglu_probe_train_plan(launch, *shape)
            assert len(plan) == (2 if launch in ("dy_dw3", "da_dw") else 1)
            for p in plan:
                assert p["whole"] + p["rest"] > 0 and p["splits"] >= 1 and p["blocks"] >= 1
                assert (p["rest"] == 0) == (p["splits"] == 1)
        with pytest.raises(ValueError, match="invalid shape"):
            sw.swiglu_probe_train_plan(launch, 0, 64, 72)
        with pytest.raises(ValueError, match="invalid shape"):
            sw.swiglu_probe_train_plan(launch, 4, 60, 72)
    L = sw.lib()
    assert L.swiglu_probe_train_plan(7, 4, 64, 72, None) == 0 and L.swiglu_probe_train_plan(0, 4, 64, 72, None) == 0
