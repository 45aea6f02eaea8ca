"""Training with Gate and Up kept as int8, on the GPU, against the definition in fp64.

Tolerances as in test_gpu_train.py for everything computed from codes and scales,
whose values (code times scale) are taken as exact.  What is kept of a sum x, known
to e in fp32:
  scale   max |x| / 127 rounded up to bf16: between (max |x| - e) / 127 and
          (max |x| + e) / 127 times 1 + 2^-7 (and two fp32 roundings), or 2^-126
  code    at most half a step from x / s: |code s - x| <= s (1/2 + 2^-15) + e, as the
          quotient of at most 127 is formed with an error of 2^-22 of itself
"""
import pytest
import torch

import swiglu_gated_mlp_amd as sw

from test_gpu_train import (F, H, LARGE, SIZES, case, check, check_products, d64, dev, fenced,  # noqa: F401
                            kept_grads, sig, sums)

pytestmark = pytest.mark.gpu


def values(codes, scales, N):
    """G and U, exactly, in fp64, and their scales [M,N]."""
    M, groups = codes.shape[:2]
    s = scales.double().permute(1, 0, 2)[..., None].expand(M, groups, 2, 32)
    v = codes.double() * s
    flat = lambda x, i: x[:, :, i].reshape(M, groups * 32)[:, :N]   # noqa: E731
    return flat(v, 0), flat(v, 1), flat(s, 0), flat(s, 1)


def keep(g, u):
    """Codes and scales of fp32 G and U by the definition."""
    M, N = g.shape
    groups = (N + 31) // 32
    x = torch.zeros(M, groups, 2, 32, device=g.device)
    for i, v in ((0, g), (1, u)):
        full = torch.zeros(M, groups * 32, device=g.device)
        full[:, :N] = v
        x[:, :, i] = full.view(M, groups, 32)
    t = x.abs().amax(3).double() / 127.0
    up = ((t.float().view(torch.int32) + 0xFFFF) >> 16 << 16).view(torch.float32).clamp_min(2.0 ** -126)
    codes = torch.round(x.double() / up.double()[..., None]).to(torch.int8)
    return codes.contiguous(), up.to(torch.bfloat16).permute(1, 0, 2).contiguous()


def check_kept(codes, scales, x, e, which, N):
    """Codes of [M,N] values x known to e."""
    M, groups = codes.shape[:2]
    s = scales[:, :, which].double().t()                       # [M, groups]
    pad = lambda v: torch.nn.functional.pad(v, (0, groups * 32 - N)).view(M, groups, 32)   # noqa: E731
    x, e = pad(x), pad(e)
    top, et = x.abs().amax(2), e.amax(2)
    lo, hi = (top - et).clamp_min(0) / 127, (top + et) / 127 * (1 + 2.0 ** -7) * (1 + 4 * F)
    assert (s >= lo * (1 - 4 * F)).all() and (s <= hi.clamp_min(2.0 ** -126)).all()
    c = codes[:, :, which].double()
    assert c.abs().max() <= 127
    assert ((c * s[..., None] - x).abs() <= s[..., None] * (0.5 + 2.0 ** -15) + e).all()
    if N % 32:
        assert not codes[:, -1, which, N % 32:].any()


def kept_case(dev, M, K, N, seed=0):
    t = case(dev, M, K, N, seed=seed)
    g = torch.Generator(device=dev).manual_seed(M + K + N)
    t["codes"], t["scales"] = keep(2 * torch.randn(M, N, generator=g, device=dev),
                                   torch.randn(M, N, generator=g, device=dev))
    return t


def fp64_of(t):
    x = d64({k: v for k, v in t.items() if k not in ("codes", "scales")})
    x["G"], x["U"], _, _ = values(t["codes"], t["scales"], t["W1"].shape[1])
    return x


@pytest.mark.parametrize("M,K,N", SIZES + LARGE)
def test_forward(dev, M, K, N):
    t = case(dev, M, K, N)
    Y, codes, scales = sw.swiglu_train_forward_int8(t["A"], t["W1"], t["W2"])
    assert torch.equal(Y, sw.swiglu_train_forward(t["A"], t["W1"], t["W2"])[0])
    g, u, eg, eu = sums(d64(t))
    check_kept(codes, scales, g, eg, 0, N)
    check_kept(codes, scales, u, eu, 1, N)


@pytest.mark.parametrize("M,N", [(1, 8), (3, 40), (4, 64), (7, 72), (130, 328), (1003, 584), (50, 18944)])
def test_dequantized(dev, M, N):
    t = kept_case(dev, M, 8, N)
    G, U = sw.swiglu_dequantize_kept_int8(t["codes"], t["scales"], N)
    g, u, _, _ = values(t["codes"], t["scales"], N)
    assert torch.equal(G, g.float().to(torch.bfloat16)) and torch.equal(U, u.float().to(torch.bfloat16))


def test_dequantized_largest(dev):
    """127 times the largest scale that bf16 holds it with: -128 times it is infinite."""
    codes = torch.full((3, 1, 2, 32), 127, dtype=torch.int8, device=dev)
    codes[1] = -127
    codes[2] = 0
    s = torch.full((1, 3, 2), 2.0 ** 121, dtype=torch.bfloat16, device=dev)
    for x in sw.swiglu_dequantize_kept_int8(codes, s, 32):
        assert torch.equal(x.double(), codes[:, 0, 0].double() * 2.0 ** 121)


@pytest.mark.parametrize("M,K,N", SIZES + LARGE)
def test_backward(dev, M, K, N):
    t = kept_case(dev, M, K, N)
    dA, dW1, dW2 = sw.swiglu_train_backward_int8(t["dY"], t["A"], t["W1"], t["W2"], t["codes"], t["scales"])
    x = fp64_of(t)
    check_products(x, *kept_grads(x, x["dY"], 0.0), dA, dW1, dW2, "%s" % ((M, K, N),))


@pytest.mark.parametrize("M,K,N", SIZES + LARGE)
def test_block_backward(dev, M, K, N):
    t = kept_case(dev, M, K, N, seed=2)
    dA, dW1, dW2, dW3 = sw.swiglu_mlp_train_backward_int8(t["dZ"], t["A"], t["W1"], t["W2"], t["W3"], t["codes"],
                                                          t["scales"])
    x = fp64_of(t)
    dY = x["dZ"] @ x["W3"].t()
    e = (K + 1) * F * (x["dZ"].abs() @ x["W3"].abs().t())
    check_products(x, *kept_grads(x, dY, e), dA, dW1, dW2, "%s" % ((M, K, N),))
    # Y, from the kernels' sigmoid and rounded to bf16
    y = x["G"] * sig(x["G"]) * x["U"]
    ey = y.abs() * (H + (x["G"].abs() + 12) * 2.0 ** -23)
    ref, S = y.t() @ x["dZ"], y.abs().t() @ x["dZ"].abs()
    sq = (y ** 2).t() @ (x["dZ"] ** 2) + ref ** 2
    check(dW3, ref, (ey.t() @ x["dZ"].abs() + (M + 1) * F * S) * (1 + H) + H * ref.abs(), sq.sqrt(),
          "%s dW3" % ((M, K, N),))


@pytest.mark.parametrize("M,K,N", [(40, 64, 136), (257, 520, 776)])
def test_a_step_against_unrounded_gradients(dev, M, K, N):
    """Forward, then backward: within what half a step moves Gate and Up from the
    gradients of the unrounded ones."""
    t = case(dev, M, K, N)
    _, codes, scales = sw.swiglu_train_forward_int8(t["A"], t["W1"], t["W2"])
    dA, dW1, dW2 = sw.swiglu_train_backward_int8(t["dY"], t["A"], t["W1"], t["W2"], codes, scales)
    x = d64(t)
    x["G"], x["U"], eg, eu = sums(x)
    _, _, sg, su = values(codes, scales, N)
    dG, dU, E_G, E_U = kept_grads(x, x["dY"], 0.0, eg + 0.501 * sg, eu + 0.501 * su)
    E_G = E_G + 0.5 * (0.51 * sg) * (0.51 * su) * x["dY"].abs()      # both errors at once
    for got, ref, e in ((dA, dG @ x["W1"].t() + dU @ x["W2"].t(), E_G @ x["W1"].abs().t() + E_U @ x["W2"].abs().t()),
                        (dW1, x["A"].t() @ dG, x["A"].abs().t() @ E_G), (dW2, x["A"].t() @ dU, x["A"].abs().t() @ E_U)):
        assert ((got.double() - ref).abs() <= 1.01 * e + 2 * H * ref.abs()).all()
        # and near them on the whole: each kept element is off by 0.003 of its group's
        # largest (a third of a step in 254), of about 2 root mean squares
        assert (got.double() - ref).norm() <= 0.02 * ref.norm()


def test_autograd_against_differences(dev):
    """Gates that codes hold exactly (whole numbers up to 127 in every group, times
    2^-5): the gradient is then the unrounded function's, and is held against central
    differences as in test_gpu_train.py."""
    M, K, N = 40, 64, 136
    t = case(dev, M, K, N)
    g = torch.Generator(device=dev).manual_seed(9)
    for n in ("W1", "W2"):
        w = torch.randint(-127, 128, (K, N), generator=g, device=dev).float()
        w[:, ::32] = 127
        t[n] = w.to(torch.bfloat16)
    A = torch.zeros(M, K, device=dev)
    A[torch.arange(M), torch.randint(0, K, (M,), generator=g, device=dev)] = 2.0 ** -5
    t["A"] = A.to(torch.bfloat16)
    _, codes, scales = sw.swiglu_train_forward_int8(t["A"], t["W1"], t["W2"])
    G, U, _, _ = values(codes, scales, N)
    assert torch.equal(G, t["A"].double() @ t["W1"].double()) and torch.equal(U, t["A"].double() @ t["W2"].double())

    def f64(A, W1, W2, W3=None):
        z = A @ W1
        y = z * sig(z) * (A @ W2)
        return y if W3 is None else y @ W3

    for names, fn, up in (("A W1 W2", lambda *a: sw.swiglu(*a, keep="int8"), "dY"),
                          ("A W1 W2 W3", lambda *a: sw.swiglu_mlp(*a, keep="int8"), "dZ")):
        names = names.split()
        leaves = [t[n].clone().requires_grad_() for n in names]
        fn(*leaves).backward(t[up])
        x = [t[n].double() for n in names]
        w = t[up].double()
        gen = torch.Generator(device=dev).manual_seed(5)
        for i, leaf in enumerate(leaves):
            v = torch.randn(x[i].shape, generator=gen, device=dev, dtype=torch.float64)
            # the gate moves by up to 127 h for A
            h = 1e-7 if names[i] == "A" else 1e-5
            hi = [y + h * v if j == i else y for j, y in enumerate(x)]
            lo = [y - h * v if j == i else y for j, y in enumerate(x)]
            num = float(((f64(*hi) - f64(*lo)) * w).sum()) / (2 * h)
            ana = float((leaf.grad.double() * v).sum())
            scale = float((leaf.grad.double() * v).pow(2).sum().sqrt())
            assert abs(num - ana) <= 6 * 2 * H * scale + 1e-6 * abs(num), (names[i], num, ana, scale)


def test_autograd_is_the_calls(dev):
    t = case(dev, 24, 64, 72)
    A = t["A"].view(2, 12, 64).clone().requires_grad_()
    W1 = t["W1"].clone().requires_grad_()
    sw.swiglu(A, W1, t["W2"], keep="int8").sum().backward()     # an expanded (stride 0) gradient
    ones = torch.ones(24, 72, dtype=torch.bfloat16, device=dev)
    _, *kept = sw.swiglu_train_forward_int8(t["A"], t["W1"], t["W2"])
    want = sw.swiglu_train_backward_int8(ones, t["A"], t["W1"], t["W2"], *kept)
    assert torch.equal(A.grad.view(24, 64), want[0]) and torch.equal(W1.grad, want[1])
    leaves = [t[n].clone().requires_grad_() for n in ("A", "W1", "W2", "W3")]
    Z = sw.swiglu_mlp(*leaves, keep="int8")
    assert torch.equal(Z, sw.swiglu_mlp(*leaves))
    Z.backward(t["dZ"])
    want = sw.swiglu_mlp_train_backward_int8(t["dZ"], *(t[n] for n in ("A", "W1", "W2", "W3")), *kept)
    assert all(torch.equal(x.grad, w) for x, w in zip(leaves, want))
    # a leaf alone
    W3 = t["W3"].clone().requires_grad_()
    sw.swiglu_mlp(t["A"], t["W1"], t["W2"], W3, keep="int8").backward(t["dZ"])
    assert torch.equal(W3.grad, want[3])


@pytest.mark.parametrize("M,K,N", [(5, 72, 136), (130, 200, 328)])
def test_partial_gradients_and_repeats(dev, M, K, N):
    t = kept_case(dev, M, K, N)
    kept = (t["codes"], t["scales"])
    args = [t[k] for k in ("dY", "A", "W1", "W2")]
    full = sw.swiglu_train_backward_int8(*args, *kept)
    only_a = sw.swiglu_train_backward_int8(*args, *kept, need_dW=False)
    only_w = sw.swiglu_train_backward_int8(*args, *kept, need_dA=False)
    assert only_a[1] is None and only_w[0] is None
    assert torch.equal(only_a[0], full[0]) and torch.equal(only_w[1], full[1]) and torch.equal(only_w[2], full[2])
    args = [t[k] for k in ("dZ", "A", "W1", "W2", "W3")]
    ws = sw.Workspace(dev)
    full = sw.swiglu_mlp_train_backward_int8(*args, *kept, workspace=ws)
    ws.buf.fill_(0xFF)
    again = sw.swiglu_mlp_train_backward_int8(*args, *kept, workspace=ws)
    assert all(torch.equal(a, b) for a, b in zip(full, again))
    assert torch.equal(sw.swiglu_mlp_train_backward_int8(*args, *kept, need_dW=False)[0], full[0])
    again = sw.swiglu_mlp_train_backward_int8(*args, *kept, need_dA=False)
    assert again[0] is None and all(torch.equal(a, b) for a, b in zip(again[1:], full[1:]))


def test_empty_batch(dev):
    t = case(dev, 0, 64, 72)
    Y, codes, scales = sw.swiglu_train_forward_int8(t["A"], t["W1"], t["W2"])
    assert Y.shape == (0, 72) and codes.shape == (0, 3, 2, 32) and scales.shape == (3, 0, 2)
    for out in (sw.swiglu_train_backward_int8(t["dY"], t["A"], t["W1"], t["W2"], codes, scales),
                sw.swiglu_mlp_train_backward_int8(t["dZ"], t["A"], t["W1"], t["W2"], t["W3"], codes, scales)):
        assert out[0].shape == (0, 64)
        for dW in out[1:]:
            assert not dW.any()
    leaf = t["W1"].clone().requires_grad_()
    sw.swiglu(t["A"], leaf, t["W2"], keep="int8").sum().backward()
    assert not leaf.grad.any()


@pytest.mark.parametrize("M,K,N", [(1, 8, 8), (65, 136, 264), (1003, 264, 584), (1500, 200, 8200)])
def test_nothing_outside_is_read_or_written(dev, M, K, N):
    """Inputs lie between NaNs (codes between the largest), outputs between marks."""
    t = kept_case(dev, M, K, N)
    calls = (lambda d, o: sw.swiglu_train_forward_int8(d["A"], d["W1"], d["W2"], *o),
             lambda d, o: sw.swiglu_train_backward_int8(d["dY"], d["A"], d["W1"], d["W2"], d["codes"], d["scales"], *o),
             lambda d, o: sw.swiglu_mlp_train_backward_int8(*(d[k] for k in ("dZ", "A", "W1", "W2", "W3", "codes",
                                                                            "scales")), *o),
             lambda d, o: sw.swiglu_dequantize_kept_int8(d["codes"], d["scales"], N, *o))
    f = {k: fenced(v, 127 if v.dtype == torch.int8 else float("nan"))[1] for k, v in t.items()}
    for i, call in enumerate(calls):
        want = call(t, ())
        bufs, outs = zip(*(fenced(torch.zeros_like(w), 7) for w in want))
        call(f, outs)
        for b, o, w in zip(bufs, outs, want):
            assert torch.equal(o, w), i
            assert (torch.cat((b[:4096], b[-4096:])) == 7).all(), i


def test_zeros_and_bad_values(dev):
    M, K, N = 70, 64, 136
    t = case(dev, M, K, N)
    t["A"][3] = 0
    t["A"][5] *= 2.0 ** -120
    clean = t["A"].clone()
    t["A"][40, 7] = float("nan")
    t["A"][41, 9] = float("inf")
    _, codes, scales = sw.swiglu_train_forward_int8(t["A"], t["W1"], t["W2"])
    bad = torch.tensor([40, 41], device=dev)
    assert scales[:, bad].isnan().all() and not codes[bad].any()
    assert not codes[3].any() and (scales[:, 3].double() == 2.0 ** -126).all()
    rest = [m for m in range(M) if m not in (40, 41)]
    _, c, s = sw.swiglu_train_forward_int8(clean, t["W1"], t["W2"])
    assert torch.equal(codes[rest], c[rest]) and torch.equal(scales[:, rest], s[:, rest])
    G, _ = sw.swiglu_dequantize_kept_int8(codes, scales, N)
    assert G[bad].isnan().all() and torch.isfinite(G[rest]).all()
    dA = sw.swiglu_train_backward_int8(t["dY"], t["A"], t["W1"], t["W2"], codes, scales, need_dW=False)[0]
    want = sw.swiglu_train_backward_int8(t["dY"], clean, t["W1"], t["W2"], c, s, need_dW=False)[0]
    assert dA[bad].isnan().all() and torch.equal(dA[rest], want[rest])
    dA = sw.swiglu_mlp_train_backward_int8(t["dZ"], t["A"], t["W1"], t["W2"], t["W3"], codes, scales, need_dW=False)[0]
    want = sw.swiglu_mlp_train_backward_int8(t["dZ"], clean, t["W1"], t["W2"], t["W3"], c, s, need_dW=False)[0]
    assert dA[bad].isnan().all() and torch.equal(dA[rest], want[rest])


def test_other_stream(dev):
    t = kept_case(dev, 130, 200, 328)
    args = [t[k] for k in ("dZ", "A", "W1", "W2", "W3", "codes", "scales")]
    want = sw.swiglu_mlp_train_backward_int8(*args)
    fwd = sw.swiglu_train_forward_int8(t["A"], t["W1"], t["W2"])
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = sw.swiglu_mlp_train_backward_int8(*args, stream=side)
    gf = sw.swiglu_train_forward_int8(t["A"], t["W1"], t["W2"], stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got + gf, want + fwd))


def test_graph_replays(dev):
    M, K, N = 65, 896, 520
    t = kept_case(dev, M, K, N)
    live = {k: v.clone() for k, v in t.items()}

    def run(d):
        Y, codes, scales = sw.swiglu_train_forward_int8(d["A"], d["W1"], d["W2"])
        return ((Y, codes, scales) + sw.swiglu_train_backward_int8(d["dY"], d["A"], d["W1"], d["W2"], codes, scales) +
                sw.swiglu_mlp_train_backward_int8(*(d[k] for k in ("dZ", "A", "W1", "W2", "W3", "codes", "scales"))))

    run(live)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = run(live)
    for seed in (3, 4, 5):
        fresh = kept_case(dev, M, K, N, seed=seed)
        for k in live:
            live[k].copy_(fresh[k])
        want = run(fresh)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, want)), seed


def test_codes_past_2gib(dev):
    """60000 rows of 18944 columns: codes end past 2^31 bytes, scales past 2^27."""
    M, K, N = 60000, 8, 18944
    t = {k: v for k, v in case(dev, M, K, N).items() if k in ("A", "W1", "W2", "W3", "dY", "dZ")}
    Y, codes, scales = sw.swiglu_train_forward_int8(t["A"], t["W1"], t["W2"])
    dA = sw.swiglu_train_backward_int8(t["dY"], t["A"], t["W1"], t["W2"], codes, scales, need_dW=False)[0]
    dB = sw.swiglu_mlp_train_backward_int8(t["dZ"], t["A"], t["W1"], t["W2"], t["W3"], codes, scales,
                                           need_dW=False)[0]
    for r in (slice(0, 100), slice(29950, 30050), slice(M - 100, M)):
        x = {k: (v[r] if k in ("A", "dY", "dZ") else v).double() for k, v in t.items()}
        g, u, eg, eu = sums(x)
        check_kept(codes[r], scales[:, r], g, eg, 0, N)
        check_kept(codes[r], scales[:, r], u, eu, 1, N)
        x["G"], x["U"], _, _ = values(codes[r], scales[:, r], N)
        check_products(x, *kept_grads(x, x["dY"], 0.0), dA[r], None, None, "product")
        dY = x["dZ"] @ x["W3"].t()
        e = (K + 1) * F * (x["dZ"].abs() @ x["W3"].abs().t())
        check_products(x, *kept_grads(x, dY, e), dB[r], None, None, "block")
