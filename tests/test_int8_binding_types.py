"""What the int8 calls of the binding say of an argument that is no tensor, or no vector."""
import numpy
import pytest
import torch

import swiglu_gated_mlp_amd as sw

M, K, N = 4, 64, 72


def calls():
    """name -> (call, its arguments by name, their optional outputs)"""
    i8, bf, f32 = torch.int8, torch.bfloat16, torch.float32
    z = lambda *s, t=bf: torch.zeros(*s, dtype=t)   # noqa: E731
    a8, w8, a, w, w3 = z(M, K, t=i8), z(K, N, t=i8), z(M, K), z(K, N), z(N, K)
    sa, s, s3 = z(M, t=f32), z(N, t=f32), z(K, t=f32)
    wp, wg = z(sw.swiglu_packed_bytes_int8(K, N), t=i8), z(sw.swiglu_gemm_packed_bytes_int8(K, N), t=i8)
    n80 = 80
    wp80, w3g = z(sw.swiglu_packed_bytes_int8(K, n80), t=i8), z(sw.swiglu_gemm_packed_bytes_int8(n80, K), t=i8)
    codes, kept, y = z(M, 3, 2, 32, t=i8), z(3, M, 2), z(M, N)
    return {
        "swiglu_quantize_rows_int8": (dict(A=a), dict(Q=a8, scales=sa)),
        "swiglu_quantize_columns_int8": (dict(W=w), dict(Q=w8, scales=s)),
        "swiglu_pack_weights_int8": (dict(W1=w8, W2=w8), dict(Wp=wp)),
        "swiglu_gemm_pack_weight_int8": (dict(W=w8), dict(Wg=wg)),
        "swiglu_fused_packed_int8": (dict(A=a8, sa=sa, Wp=wp, s1=s, s2=s), dict(Y=y)),
        "swiglu_gemm_packed_int8": (dict(A=a8, sa=sa, Wg=wg, sw=s), dict(C=y)),
        "swiglu_mlp_packed_int8": (dict(A=a, Wp=wp80, s1=z(n80, t=f32), s2=z(n80, t=f32), W3g=w3g, s3=s3),
                                   dict(Y=z(M, n80), Z=a)),
        "swiglu_train_forward_int8": (dict(A=a, W1=w, W2=w), dict(Y=y, codes=codes, scales=kept)),
        "swiglu_dequantize_kept_int8": (dict(codes=codes, scales=kept), dict(G=y, U=y)),
        "swiglu_train_backward_int8": (dict(dY=y, A=a, W1=w, W2=w, codes=codes, scales=kept), dict(dA=a, dW1=w, dW2=w)),
        "swiglu_mlp_train_backward_int8": (dict(dZ=a, A=a, W1=w, W2=w, W3=w3, codes=codes, scales=kept),
                                           dict(dA=a, dW1=w, dW2=w, dW3=w3)),
    }


@pytest.fixture(autouse=True)
def on_the_cpu(monkeypatch):
    """CPU tensors pass for the current GPU's, so that every argument is reached."""
    from swiglu_gated_mlp_amd import int8, train
    for m in (int8, train):
        monkeypatch.setattr(m, "_here", lambda: -1)
        monkeypatch.setattr(m, "_stream_at", lambda here, stream: 0)
        monkeypatch.setattr(m, "_space", lambda *rest: (0, 0))
    monkeypatch.setattr(int8, "_out", lambda t, *rest: torch.zeros(1) if t is None else t)
    monkeypatch.setattr(train, "_out", lambda t, *rest: torch.zeros(1) if t is None else t)
    monkeypatch.setattr(train, "_new", lambda *rest: torch.zeros(1))


@pytest.mark.parametrize("fn", list(calls()))
def test_no_tensor(fn):
    needed, outs = calls()[fn]
    extra = dict(N=N) if fn == "swiglu_dequantize_kept_int8" else {}
    for name, t in list(needed.items()) + list(outs.items()):
        for bad in ([0.0] * 4, numpy.zeros(tuple(t.shape), dtype=numpy.float32), 3, "x") + (
                (None,) if name in needed else ()):
            args = {**needed, **outs, **extra, name: bad}
            with pytest.raises(TypeError, match="^%s must be a torch tensor$" % name):
                getattr(sw, fn)(**args)


@pytest.mark.parametrize("fn,names", [("swiglu_fused_packed_int8", "sa s1 s2"), ("swiglu_gemm_packed_int8", "sa sw"),
                                      ("swiglu_mlp_packed_int8", "s1 s2 s3")])
def test_scales_are_vectors(fn, names):
    needed, _ = calls()[fn]
    for name in names.split():
        for bad in (needed[name].reshape(1, -1), needed[name][0]):
            with pytest.raises(ValueError, match=name):
                getattr(sw, fn)(**{**needed, name: bad})


@pytest.mark.parametrize("fn", ["swiglu_train_forward_int8", "swiglu_train_backward_int8",
                                "swiglu_mlp_train_backward_int8", "swiglu_dequantize_kept_int8"])
def test_kept_values_of_other_dimensions(fn):
    needed, outs = calls()[fn]
    extra = dict(N=N) if fn == "swiglu_dequantize_kept_int8" else {}
    for name in {"codes", "scales"} & {*needed, *outs}:
        for bad in ({**needed, **outs}[name][0], torch.zeros(())):
            with pytest.raises(ValueError, match="%s must be" % name):
                getattr(sw, fn)(**{**needed, **outs, **extra, name: bad})
