"""Argument checks of the low-rank adapter entry points (no GPU: every check
comes before the first HIP call, and the addresses are never read)."""
import pytest
import torch

import swiglu_gated_mlp_amd as sw

OK, NULLP, SHAPE, UNSUP, MISAL, ALIAS, WS = 0, 1, 2, 3, 4, 5, 6
A, W, LP, IDS, SC, Y, WK, LA1, LB1, LA2, LB2 = (0x40000000 * (i + 1) for i in range(11))
BIG = 1 << 29


def gated(a=A, w=W, lp=LP, ids=IDS, sc=SC, y=Y, M=4, K=64, N=72, L=3, r=16, ws=WK, nb=BIG):
    return sw.lib().swiglu_fused_packed_lora(a, w, lp, ids, sc, y, M, K, N, L, r, ws, nb, None)


def plain(a=A, w=W, lp=LP, ids=IDS, sc=SC, y=Y, M=4, K=64, N=72, L=3, r=16, ws=WK, nb=BIG):
    return sw.lib().swiglu_gemm_packed_lora(a, w, lp, ids, sc, y, M, K, N, L, r, ws, nb, None)


BAD = [(dict(K=0), SHAPE), (dict(N=-8), SHAPE), (dict(K=60), UNSUP), (dict(N=60), UNSUP), (dict(L=0), SHAPE),
       (dict(L=-1), SHAPE), (dict(r=0), SHAPE), (dict(r=-4), SHAPE), (dict(r=257), UNSUP), (dict(L=1 << 26), SHAPE)]


@pytest.mark.parametrize("call", [gated, plain])
@pytest.mark.parametrize("shape,want", BAD + [(dict(M=-1), SHAPE), (dict(M=1 << 31), SHAPE)])
def test_shapes(call, shape, want):
    assert call(**shape) == want


@pytest.mark.parametrize("call", [gated, plain])
def test_pointers(call):
    for n in "a w lp ids sc y".split():
        assert call(**{n: None}) == NULLP, n
    for n in "a w lp y".split():
        assert call(**{n: 0x7000000008}) == MISAL, n
    for n in ("ids", "sc"):
        assert call(**{n: 0x7000000002}) == MISAL, n
    # int32 and fp32 vectors need their own alignment only
    assert call(ids=IDS + 4, sc=SC + 4, ws=None) == WS
    assert call(ws=WK + 8) == MISAL
    for src in (A, W, LP, IDS, SC):
        assert call(y=src) == ALIAS and call(ws=src) == ALIAS
    assert call(ws=Y) == ALIAS
    assert call(M=0, a=None, w=None, lp=None, ids=None, sc=None, y=None, ws=None) == OK


def test_workspace():
    L = sw.lib()
    for call, need_fn in ((gated, L.swiglu_lora_workspace_bytes), (plain, L.swiglu_gemm_lora_workspace_bytes)):
        need = need_fn(4, 64, 72, 16)
        assert need > 0
        assert call(nb=need - 1) == WS and call(ws=None) == WS
        assert need_fn(0, 64, 72, 16) == 0 and need_fn(4, 64, 72, 257) == 0 and need_fn(4, 60, 72, 16) == 0
        # the factors: 64 bytes a row, chunk of 16 and projection
        assert need_fn(1024, 512, 8192, 17) >= 1024 * 2 * 64


@pytest.mark.parametrize("shape,want", BAD)
def test_pack(shape, want):
    d = dict(K=64, N=72, L=3, r=16)
    d.update(shape)
    L = sw.lib()
    args = (d["K"], d["N"], d["L"], d["r"])
    assert L.swiglu_lora_pack(LA1, LB1, LA2, LB2, LP, *args, None) == want
    assert L.swiglu_gemm_lora_pack(LA1, LB1, LP, *args, None) == want
    assert L.swiglu_lora_packed_bytes(*args) == 0 and L.swiglu_gemm_lora_packed_bytes(*args) == 0


def test_pack_pointers_and_sizes():
    L = sw.lib()
    args = (64, 72, 3, 16)
    ok = [LA1, LB1, LA2, LB2, LP]
    for i in range(5):
        for bad, want in ((None, NULLP), (ok[i] + 8, MISAL)):
            p = list(ok)
            p[i] = bad
            assert L.swiglu_lora_pack(*p, *args, None) == want
    assert L.swiglu_lora_pack(LA1, LB1, LP, LB2, LP, *args, None) == ALIAS
    assert L.swiglu_gemm_lora_pack(LA1, LP + 32, LP, *args, None) == ALIAS
    # per adapter, projection and chunk: 64-deep k blocks of 2 KiB, 32-column tiles of 1 KiB;
    # a 4-byte flag an adapter, in whole 16 bytes
    assert L.swiglu_lora_packed_bytes(64, 72, 3, 16) == 3 * 2 * (1 * 2048 + 4 * 1024) + 16
    assert L.swiglu_lora_packed_bytes(72, 136, 1, 17) == 2 * 2 * (2 * 2048 + 8 * 1024) + 16
    assert L.swiglu_gemm_lora_packed_bytes(72, 264, 5, 1) == 5 * (2 * 2048 + 16 * 1024) + 32


def test_binding_refusals():
    bf = dict(dtype=torch.bfloat16)
    la, lb = torch.zeros(3, 64, 16, **bf), torch.zeros(3, 16, 72, **bf)
    with pytest.raises(ValueError, match="GPU tensor"):
        sw.swiglu_lora_pack(la, lb, la, lb)
    with pytest.raises(ValueError, match="La"):
        sw.swiglu_gemm_lora_pack(la[0], lb)
    with pytest.raises(ValueError, match="Lb2 must be"):
        sw.swiglu_lora_pack(la, lb, la, lb[:, :8])
    a = torch.zeros(4, 64, **bf)
    ids, sc = torch.zeros(4, dtype=torch.int32), torch.ones(3)
    wp = torch.zeros(sw.swiglu_packed_bytes(64, 72) // 2, **bf)
    with pytest.raises(ValueError, match="GPU tensor"):
        sw.swiglu_fused_packed_lora(a, wp, wp, ids, sc, 72, 16)
    with pytest.raises(ValueError, match="Wp holds"):
        sw.swiglu_fused_packed_lora(a, wp[:8], wp, ids, sc, 72, 16)
    with pytest.raises(ValueError, match="Wg holds"):
        sw.swiglu_gemm_packed_lora(a, wp[:8], wp, ids, sc, 72, 16)
