"""Argument checks of the int8 products' entry points (no GPU: every check comes
before the first HIP call, and the addresses are never read)."""
import pytest
import torch

import swiglu_gated_mlp_amd as sw

OK, NULLP, SHAPE, UNSUP, MISAL, ALIAS, WS = 0, 1, 2, 3, 4, 5, 6
# 1 GiB apart, never dereferenced
A, SA, W, S1, S2, Y, W3, S3, Z, WK, Q, SQ = (0x40000000 * (i + 1) for i in range(12))
BIG = 1 << 29


def fused(a=A, sa=SA, w=W, s1=S1, s2=S2, y=Y, M=4, K=64, N=72, ws=WK, nb=BIG):
    return sw.lib().swiglu_fused_packed_int8(a, sa, w, s1, s2, y, M, K, N, ws, nb, None)


def gemm(a=A, sa=SA, w=W, s1=S1, y=Y, M=4, K=64, N=72, ws=WK, nb=BIG):
    return sw.lib().swiglu_gemm_packed_int8(a, sa, w, s1, y, M, K, N, ws, nb, None)


def mlp(a=A, w=W, s1=S1, s2=S2, w3=W3, s3=S3, y=Y, z=Z, M=4, K=64, N=80, ws=WK, nb=BIG):
    return sw.lib().swiglu_mlp_packed_int8(a, w, s1, s2, w3, s3, y, z, M, K, N, ws, nb, None)


def rows(a=A, q=Q, s=SQ, M=4, K=64):
    return sw.lib().swiglu_quantize_rows_int8(a, q, s, M, K, None)


def cols(a=A, q=Q, s=SQ, K=64, N=72):
    return sw.lib().swiglu_quantize_columns_int8(a, q, s, K, N, None)


@pytest.mark.parametrize("call", [fused, gemm, mlp])
@pytest.mark.parametrize("shape,want", [
    (dict(M=-1), SHAPE), (dict(K=0), SHAPE), (dict(N=0), SHAPE), (dict(N=-8), SHAPE), (dict(M=1 << 31), SHAPE),
    (dict(K=60), UNSUP), (dict(K=72), UNSUP), (dict(N=60), UNSUP), (dict(K=131072), UNSUP),
])
def test_shapes(call, shape, want):
    assert call(**shape) == want


def test_block_contracts_over_both_widths():
    assert mlp(N=72) == UNSUP and mlp(N=131072) == UNSUP
    assert sw.swiglu_mlp_workspace_bytes_int8(4, 64, 72) == 0
    assert sw.swiglu_mlp_workspace_bytes_int8(4, 64, 80) > 0


@pytest.mark.parametrize("call,matrices,vectors", [
    (fused, "a w y", "sa s1 s2"), (gemm, "a w y", "sa s1"), (mlp, "a w w3 y z", "s1 s2 s3"), (rows, "a q", "s"),
    (cols, "a q", "s"),
])
def test_null_and_misaligned(call, matrices, vectors):
    for n in (matrices + " " + vectors).split():
        assert call(**{n: None}) == NULLP, n
        assert call(**{n: 0x7000000002}) == MISAL, n
    for n in matrices.split():
        assert call(**{n: 0x7000000008}) == MISAL, n


def test_vectors_need_their_own_alignment_only():
    # on to the last check
    assert mlp(s1=S1 + 4, s2=S2 + 8, s3=S3 + 12, ws=None, nb=0) == WS


def test_aliasing():
    for call, outs, ins in ((fused, "y", (A, SA, W, S1, S2)), (gemm, "y", (A, SA, W, S1)),
                            (mlp, "y z", (A, W, S1, S2, W3, S3)), (rows, "q s", (A,)), (cols, "q s", (A,))):
        for o in outs.split():
            for i in ins:
                assert call(**{o: i}) == ALIAS, (call.__name__, o, hex(i))
        if call not in (rows, cols):
            for i in ins:
                assert call(ws=i) == ALIAS
            assert call(ws=Y) == ALIAS
    assert mlp(y=Z) == ALIAS and rows(s=Q) == ALIAS
    # inputs may be the same: both scales, both weights' halves
    assert mlp(s2=S1, ws=None, nb=0) == WS


def test_workspace():
    L = sw.lib()
    for shape in ((1, 896, 4864), (64, 3584, 18944), (4096, 896, 4864)):
        need = L.swiglu_mlp_workspace_bytes_int8(*shape)
        M, K, N = shape
        # codes and scales of A and of Y, and the splits' sums of either product
        assert need >= M * (K + N) + 8 * M + max(L.swiglu_workspace_bytes_int8(M, K, N),
                                                 L.swiglu_gemm_workspace_bytes_int8(M, N, K))
        assert mlp(M=M, K=K, N=N, nb=need - 1) in (WS, ALIAS)
    need = L.swiglu_mlp_workspace_bytes_int8(4, 64, 80)
    assert mlp(nb=need - 1) == WS and mlp(ws=None) == WS
    # splits of K: few tiles and a long contraction
    need = L.swiglu_gemm_workspace_bytes_int8(100, 16000, 1000)
    assert need > 0 and gemm(M=100, K=16000, N=1000, nb=need - 1) == WS
    need = L.swiglu_workspace_bytes_int8(100, 16000, 520)
    assert need > 0 and fused(M=100, K=16000, N=520, nb=need - 1) == WS
    for fn in (L.swiglu_workspace_bytes_int8, L.swiglu_gemm_workspace_bytes_int8, L.swiglu_mlp_workspace_bytes_int8):
        assert fn(0, 64, 64) == 0 and fn(4, 72, 64) == 0 and fn(-1, 64, 64) == 0 and fn(4, 131072, 64) == 0


def test_packed_bytes():
    L = sw.lib()
    assert L.swiglu_packed_bytes_int8(896, 4864) == 2 * 896 * 4864          # exact when tiles divide
    assert L.swiglu_packed_bytes_int8(144, 136) == 2 * 2 * 32768            # padded tail tiles
    assert L.swiglu_gemm_packed_bytes_int8(144, 264) == 2 * 2 * 32768
    for fn in (L.swiglu_packed_bytes_int8, L.swiglu_gemm_packed_bytes_int8):
        assert fn(72, 64) == 0 and fn(64, 60) == 0 and fn(0, 8) == 0 and fn(131072, 8) == 0 and fn(131056, 8) > 0


def test_pack_errors():
    L = sw.lib()
    assert L.swiglu_pack_weights_int8(W, W, Q, 72, 64, None) == UNSUP
    assert L.swiglu_pack_weights_int8(W, None, Q, 64, 64, None) == NULLP
    assert L.swiglu_pack_weights_int8(W, W3 + 8, Q, 64, 64, None) == MISAL
    assert L.swiglu_pack_weights_int8(W, W3, W3 + 64, 64, 64, None) == ALIAS
    assert L.swiglu_gemm_pack_weight_int8(W, W + 64, 64, 64, None) == ALIAS
    assert L.swiglu_gemm_pack_weight_int8(W, None, 64, 64, None) == NULLP


def test_empty_batch():
    assert fused(M=0, a=None, y=None, ws=None) == OK and gemm(M=0, a=None, y=None) == OK
    assert mlp(M=0, a=None, y=None, z=None, ws=None) == OK and rows(M=0, a=None, q=None, s=None) == OK


def test_quantize_shapes():
    assert rows(K=60) == UNSUP and rows(K=131072) == UNSUP and rows(M=-1) == SHAPE and cols(N=60) == UNSUP
    assert cols(K=0) == SHAPE


def test_binding_refusals():
    a8, a = torch.zeros(4, 64, dtype=torch.int8), torch.zeros(4, 64, dtype=torch.bfloat16)
    w8, v, r = torch.zeros(64, 72, dtype=torch.int8), torch.zeros(72), torch.zeros(4)
    wp = torch.zeros(sw.swiglu_packed_bytes_int8(64, 72), dtype=torch.int8)
    for call in (lambda: sw.swiglu_quantize_rows_int8(a), lambda: sw.swiglu_quantize_columns_int8(a),
                 lambda: sw.swiglu_pack_weights_int8(w8, w8), lambda: sw.swiglu_gemm_pack_weight_int8(w8),
                 lambda: sw.swiglu_fused_packed_int8(a8, r, wp, v, v), lambda: sw.swiglu_gemm_packed_int8(a8, r, wp, v)):
        with pytest.raises(ValueError, match="GPU tensor"):
            call()
    with pytest.raises(ValueError, match="Wp holds"):
        sw.swiglu_fused_packed_int8(a8, r, wp[:64], v, v)
    with pytest.raises(ValueError, match="Y must be"):
        sw.swiglu_fused_packed_int8(a8, r, wp, v, v, Y=a)
    with pytest.raises(ValueError, match="W2 must be"):
        sw.swiglu_pack_weights_int8(w8, w8[:, :64])
    with pytest.raises(ValueError, match="invalid int8 weight shape"):
        sw.swiglu_pack_weights_int8(w8[:60], w8[:60])
    with pytest.raises(ValueError, match="must be a matrix"):
        sw.swiglu_quantize_rows_int8(a[0])
    with pytest.raises(ValueError, match="scales must be"):
        sw.swiglu_quantize_rows_int8(a, scales=v)
    with pytest.raises(ValueError, match="invalid int8 weight shape"):
        sw.swiglu_mlp_packed_int8(a, wp, v, v, wp, torch.zeros(64))


def test_plan_probe():
    for gemm in (False, True):
        for shape, kernel in (((1, 64, 72), "decode"), ((8, 3584, 18944), "decode"), ((33, 3584, 18944), None),
                              ((8192, 3584, 18944), "stream")):
            p = sw.swiglu_probe_int8_plan(gemm, *shape)
            assert kernel in (None, p["kernel"]) and p["rows"] > 0 and p["cols"] > 0 and p["splits"] >= 1
            need = (sw.swiglu_gemm_workspace_bytes_int8 if gemm else sw.swiglu_workspace_bytes_int8)(*shape)
            assert (need > 0) == (p["splits"] > 1)
        for bad in ((0, 64, 72), (4, 72, 64), (4, 64, 60)):
            with pytest.raises(ValueError, match="invalid shape"):
                sw.swiglu_probe_int8_plan(gemm, *bad)
    assert sw.lib().swiglu_probe_int8_plan(0, 4, 64, 72, None) == 0


class Elsewhere(torch.Tensor):
    """A tensor that says it is on the second GPU."""
    device = torch.device("cuda:1")

    def get_device(self):
        return 1


def test_tensors_of_another_device_are_refused(monkeypatch):
    from swiglu_gated_mlp_amd import int8, train
    monkeypatch.setattr(int8, "_here", lambda: 0)
    monkeypatch.setattr(train, "_here", lambda: 0)
    a8, a = torch.zeros(4, 64, dtype=torch.int8), torch.zeros(4, 64, dtype=torch.bfloat16)
    w, v, r = torch.zeros(64, 72, dtype=torch.bfloat16), torch.zeros(72), torch.zeros(4)
    wp = torch.zeros(sw.swiglu_packed_bytes_int8(64, 72), dtype=torch.int8)
    w8, codes = torch.zeros(64, 72, dtype=torch.int8), torch.zeros(4, 3, 2, 32, dtype=torch.int8)
    kept, dy = torch.zeros(3, 4, 2, dtype=torch.bfloat16), torch.zeros(4, 72, dtype=torch.bfloat16)
    w3 = torch.zeros(72, 64, dtype=torch.bfloat16)
    a8, a, w, w3, v, r, wp, w8, codes, kept, dy = (t.as_subclass(Elsewhere) for t in
                                                   (a8, a, w, w3, v, r, wp, w8, codes, kept, dy))
    for call in (lambda: sw.swiglu_quantize_rows_int8(a), lambda: sw.swiglu_quantize_columns_int8(w),
                 lambda: sw.swiglu_pack_weights_int8(w8, w8), lambda: sw.swiglu_gemm_pack_weight_int8(w8),
                 lambda: sw.swiglu_fused_packed_int8(a8, r, wp, v, v), lambda: sw.swiglu_gemm_packed_int8(a8, r, wp, v),
                 lambda: sw.swiglu_mlp_packed_int8(a, wp, v[:64], v[:64], wp, v[:64]),
                 lambda: sw.swiglu_train_forward_int8(a, w, w), lambda: sw.swiglu_dequantize_kept_int8(codes, kept, 72),
                 lambda: sw.swiglu_train_backward_int8(dy, a, w, w, codes, kept),
                 lambda: sw.swiglu_mlp_train_backward_int8(a, a, w, w, w3, codes, kept)):
        with pytest.raises(ValueError, match="the current device is 0"):
            call()


def test_a_workspace_of_another_device_is_refused():
    from swiglu_gated_mlp_amd import int8
    elsewhere, here = torch.zeros(64, dtype=torch.uint8).as_subclass(Elsewhere), torch.zeros(64, dtype=torch.uint8)
    with pytest.raises(ValueError, match="workspace is on cuda:1, the current device is 0"):
        int8._space(elsewhere, 64, torch.device("cuda:0"), 0, 0)
    with pytest.raises(ValueError, match="GPU tensor"):
        int8._space(here, 64, torch.device("cuda:0"), 0, 0)
