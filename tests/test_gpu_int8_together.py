"""The int8 operators as they are used one after another: a step trained with int8
checkpoints, its weights quantized, packed and served; and the example that does so."""
import importlib.util
import os

import pytest
import torch

import swiglu_gated_mlp_amd as sw

from test_gpu_int8 import check_fused, check_gemm, dev, quantized  # noqa: F401

pytestmark = pytest.mark.gpu


def example():
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples",
                        "train_and_serve_int8.py")
    spec = importlib.util.spec_from_file_location("train_and_serve_int8", path)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def randn(dev, seed, *shape):
    g = torch.Generator(device=dev).manual_seed(seed)
    return torch.randn(*shape, generator=g, device=dev)


def test_trained_quantized_served(dev):  # noqa: F811
    """Each step is its definition on what the step before it left."""
    M, K, N = 200, 208, 336
    A, W = randn(dev, 1, M, K).bfloat16(), [randn(dev, 2 + i, *s) / s[0] ** 0.5 for i, s in
                                            enumerate(((K, N), (K, N), (N, K)))]
    W = [w.bfloat16().requires_grad_() for w in W]
    dZ = (randn(dev, 5, M, K) / M).bfloat16()
    Z = sw.swiglu_mlp(A, *W, keep="int8")
    Y, kept, kept_scales = sw.swiglu_train_forward_int8(A, W[0].detach(), W[1].detach())
    grads = torch.autograd.grad(Z, W, dZ)
    want = sw.swiglu_mlp_train_backward_int8(dZ, A, *(w.detach() for w in W), kept, kept_scales, need_dA=False)[1:]
    for a, b in zip(grads, want):
        assert torch.equal(a, b)
    # one step, then what a server holds of it
    W = [(w.detach().float() - 0.01 * g.float() / g.float().square().mean().sqrt()).bfloat16()
         for w, g in zip(W, grads)]
    W8 = [sw.swiglu_quantize_columns_int8(w) for w in W]
    for w, (q, s) in zip(W, W8):
        q0, s0 = quantized(w, 0)
        assert torch.equal(q, q0) and torch.equal(s, s0)
    Wp, W3g = sw.swiglu_pack_weights_int8(W8[0][0], W8[1][0]), sw.swiglu_gemm_pack_weight_int8(W8[2][0])
    ws = sw.Workspace(dev)
    for m in (1, 40, 100, 200, 3):   # prompts and single tokens in turn, in one workspace
        Y, Z = sw.swiglu_mlp_packed_int8(A[:m], Wp, W8[0][1], W8[1][1], W3g, W8[2][1], workspace=ws)
        q, sa = quantized(A[:m], 1)
        check_fused(Y, q, sa, W8[0][0], W8[0][1], W8[1][0], W8[1][1], "Y")
        q, sy = quantized(Y, 1)
        check_gemm(Z, q, sy, W8[2][0], W8[2][1], "Z")


def test_two_streams_at_once(dev):  # noqa: F811
    """Calls that run side by side, each with a workspace of its own."""
    K, N = 14336, 528   # K long enough that the product of 100 rows is split
    W = [randn(dev, 7 + i, *s).bfloat16() for i, s in enumerate(((K, N), (K, N), (N, K)))]
    W8 = [sw.swiglu_quantize_columns_int8(w) for w in W]
    w = (sw.swiglu_pack_weights_int8(W8[0][0], W8[1][0]), W8[0][1], W8[1][1],
         sw.swiglu_gemm_pack_weight_int8(W8[2][0]), W8[2][1])
    assert sw.swiglu_workspace_bytes_int8(100, K, N) > 0
    A = [randn(dev, 20 + i, 100, K).bfloat16() for i in range(2)]
    want = [sw.swiglu_mlp_packed_int8(a, *w) for a in A]
    streams, spaces = [torch.cuda.Stream() for _ in A], [sw.Workspace(dev) for _ in A]
    torch.cuda.synchronize()
    got = []
    for _ in range(5):
        for a, s, space in zip(A, streams, spaces):
            with torch.cuda.stream(s):
                got.append(sw.swiglu_mlp_packed_int8(a, *w, workspace=space))
    torch.cuda.synchronize()
    for i, (Y, Z) in enumerate(got):
        assert torch.equal(Y, want[i % 2][0]) and torch.equal(Z, want[i % 2][1])


def test_the_example_runs(dev):  # noqa: F811
    W, worst = example().main(steps=3, K=144, N=272, rows=256, out=lambda s: None)
    assert all(torch.isfinite(w.float()).all() for w in W)
    # A code is off by half a step of 1/127 of the largest value of its row or column,
    # which is below 5 times the root mean square (Y's, of a product, below 8): errors
    # of 5 / 127 / 12^0.5 = 0.0114 each, 0.018 for Y's codes.  G and U have two (0.016);
    # SiLU and its slope have about the same root mean square, so Y has 0.016 * 2^0.5 =
    # 0.023; Z, with Y's codes and W3's, (0.023^2 + 0.018^2 + 0.0114^2)^0.5 = 0.031, of
    # which twice as much is allowed for a single row
    assert worst < 0.06


def test_the_examples_gradients(dev):  # noqa: F811
    """Against autograd's on the plain block in 64 bits, Gate and Up kept with errors of
    half a step of at most 1/127 (1 + 2^-7) of a group's largest value."""
    m, M, K, N = example(), 96, 144, 264
    W = [(randn(dev, 40 + i, *s) / s[0] ** 0.5).bfloat16() for i, s in enumerate(((K, N), (K, N), (N, K)))]
    A, target = randn(dev, 50, M, K).bfloat16(), randn(dev, 51, M, K)
    loss, grads = m.gradients(A, target, W)
    X = [w.double().requires_grad_() for w in W]
    h = torch.nn.functional.silu(A.double() @ X[0]) * (A.double() @ X[1])
    ref = (h @ X[2] - target.double()).square().mean()
    for got, want in zip(grads, torch.autograd.grad(ref, X)):
        # A kept value is off by 3 / 127 / 12^0.5 = 0.007 of the root mean square (the
        # largest of 32 is about 2.2 times that, 3 leaves room).  dU = dY SiLU(G) has one
        # of them, dG = dY U SiLU'(G) and Y two (0.0096); the roundings to bf16 of Z, dZ,
        # dY, D and the gradient 2^-8 / 3^0.5 = 0.0023 each: 0.011 together
        err = (got.double() - want).square().mean().sqrt() / want.square().mean().sqrt()
        assert err < 0.02
    assert abs(float(loss) - float(ref.detach())) < 2 * 2.0 ** -8 * float(ref.detach())
