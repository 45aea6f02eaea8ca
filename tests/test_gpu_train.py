"""Training entry points on the GPU against their definition in fp64.

Tolerances.  A rounding to bf16 is off by at most 2^-8 of the value, one to fp32
by 2^-24.  With S a sum's terms in absolute value:
  sums            K 2^-24 S for a sum of K terms in any order
  exp, rcp        the kernels' sigmoid: relative error (|g| + 8) 2^-23 (the
                  rounding of g log2 e scales with |g|; a few ulp for the rest)
  dG, dU          one bf16 rounding each, and what the sums' errors in G, U or dY
                  move them by (|SiLU'| <= 1.1, |SiLU''| <= 0.5)
  dA, dW          the errors of dG and dU through the product, in absolute value,
                  plus the sum's own, plus one bf16 rounding
The worst case over N or M terms is far above what independent roundings give, so
the root mean square is held to 2^-8 of the terms' root sum of squares too: two
roundings in a row have a root mean square of at most sqrt(2/3) 2^-8.
"""
import pytest
import torch

import swiglu_gated_mlp_amd as sw

pytestmark = pytest.mark.gpu

H = torch.finfo(torch.bfloat16).eps / 2   # 2^-8
F = 2.0 ** -24


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    return torch.device("cuda:0")


def case(dev, M, K, N, seed=0, kept=True, std_dy=1.0):
    g = torch.Generator(device=dev).manual_seed(1000 * seed + M + 3 * K + 7 * N)

    def rnd(*shape, std=1.0):
        return (torch.randn(*shape, generator=g, device=dev) * std).to(torch.bfloat16)

    t = dict(A=rnd(M, K), W1=rnd(K, N, std=K ** -0.5), W2=rnd(K, N, std=K ** -0.5), W3=rnd(N, K, std=N ** -0.5),
             dY=rnd(M, N, std=std_dy), dZ=rnd(M, K, std=std_dy))
    t["G"], t["U"] = rnd(M, N, std=2.0), rnd(M, N)
    gf = t["G"].float()
    t["Y"] = (gf * torch.sigmoid(gf) * t["U"].float()).to(torch.bfloat16)
    return t


def d64(t):
    return {k: v.double() for k, v in t.items()}


def sig(g):
    return 1.0 / (1.0 + torch.exp(-g))


def check(got, ref, bound, scale, what):
    """|got - ref| <= bound everywhere; rms error <= 2^-8 rms(scale)."""
    assert torch.isfinite(got).all(), what
    err = (got.double() - ref).abs()
    bad = err > bound + 1e-30
    assert not bad.any(), "%s: %d of %d outside the bound, worst %g times it" % (
        what, int(bad.sum()), bad.numel(), float((err / (bound + 1e-30)).max()))
    if err.numel() >= 64:
        rms, lim = err.pow(2).mean().sqrt(), H * scale.pow(2).mean().sqrt()
        assert rms <= lim, "%s: rms error %g, limit %g" % (what, float(rms), float(lim))


def kept_grads(x, dY, E_dy, E_g=0.0, E_u=0.0):
    """(dG, dU, bound of their error) for dY, G, U in fp64 known to E_dy, E_g, E_u."""
    g, u = x["G"], x["U"]
    s = sig(g)
    h, d1 = g * s, s * (1 + g * (1 - s))
    ap = (g.abs() + 8) * 2.0 ** -23
    dU, dG = dY * h, dY * u * d1
    E_U = E_dy * h.abs() + dY.abs() * (1.1 * E_g + h.abs() * ap)
    E_G = E_dy * (u * d1).abs() + dY.abs() * (E_u * 1.1 + u.abs() * (0.5 * E_g + s * (1 + g.abs()) * 2 * ap))
    return dG, dU, E_G * (1 + H) + H * dG.abs(), E_U * (1 + H) + H * dU.abs()


def check_products(x, dG, dU, E_G, E_U, dA, dW1, dW2, tag):
    M, K = x["A"].shape
    N = x["W1"].shape[1]
    if dA is not None:
        ref = dG @ x["W1"].t() + dU @ x["W2"].t()
        S = dG.abs() @ x["W1"].abs().t() + dU.abs() @ x["W2"].abs().t()
        E = E_G @ x["W1"].abs().t() + E_U @ x["W2"].abs().t() + 2 * (N + 1) * F * (1 + H) * S
        sq = (dG ** 2) @ (x["W1"] ** 2).t() + (dU ** 2) @ (x["W2"] ** 2).t() + ref ** 2
        check(dA, ref, E * (1 + H) + H * ref.abs(), sq.sqrt(), tag + " dA")
    for dW, d, e, name in ((dW1, dG, E_G, "dW1"), (dW2, dU, E_U, "dW2")):
        if dW is not None:
            At = x["A"].t()
            ref = At @ d
            E = At.abs() @ e + (M + 1) * F * (1 + H) * (At.abs() @ d.abs())
            check(dW, ref, E * (1 + H) + H * ref.abs(), ((At ** 2) @ (d ** 2) + ref ** 2).sqrt(), tag + " " + name)


def sums(x):
    """G, U of A, W1, W2 and the bounds of their fp32 sums."""
    K = x["A"].shape[1]
    c = (K + 1) * F
    return (x["A"] @ x["W1"], x["A"] @ x["W2"], c * (x["A"].abs() @ x["W1"].abs()), c * (x["A"].abs() @ x["W2"].abs()))


# every tile edge: one token, ragged rows, columns and depths, each tile size
SIZES = [(1, 8, 8), (1, 64, 128), (2, 72, 136), (16, 896, 520), (63, 128, 200), (64, 256, 64), (65, 136, 264),
         (128, 192, 384), (129, 320, 328), (257, 520, 776), (300, 256, 1032), (1003, 264, 584)]
# products large enough for 256-row tiles: forward and dY; dA; dW; dW3
LARGE = [(1500, 200, 8200), (4100, 3592, 72), (70, 3592, 2000), (100, 6200, 2056)]


@pytest.mark.parametrize("M,K,N", SIZES + LARGE)
def test_forward(dev, M, K, N):
    t = case(dev, M, K, N)
    Y, G, U = sw.swiglu_train_forward(t["A"], t["W1"], t["W2"])
    x = d64(t)
    g, u, eg, eu = sums(x)
    for got, ref, e, name in ((G, g, eg, "G"), (U, u, eu, "U")):
        check(got, ref, e * (1 + H) + H * ref.abs(), ref + e, "%s %s" % ((M, K, N), name))
    h = g * sig(g)
    e = u.abs() * (1.1 * eg + h.abs() * (g.abs() + 8) * 2.0 ** -23) + (h.abs() + 1.1 * eg) * eu
    check(Y, h * u, e * (1 + H) + H * (h * u).abs(), h * u + e, "%s Y" % ((M, K, N),))


@pytest.mark.parametrize("M,K,N", SIZES + LARGE)
def test_backward_kept(dev, M, K, N):
    t = case(dev, M, K, N)
    dA, dW1, dW2 = sw.swiglu_train_backward(t["dY"], t["A"], t["W1"], t["W2"], t["G"], t["U"])
    x = d64(t)
    check_products(x, *kept_grads(x, x["dY"], 0.0), dA, dW1, dW2, "%s" % ((M, K, N),))


@pytest.mark.parametrize("M,K,N", SIZES + LARGE)
def test_backward_recomputed(dev, M, K, N):
    t = case(dev, M, K, N, seed=1)
    dA, dW1, dW2 = sw.swiglu_train_backward(t["dY"], t["A"], t["W1"], t["W2"])
    x = d64(t)
    x["G"], x["U"], eg, eu = sums(x)
    check_products(x, *kept_grads(x, x["dY"], 0.0, eg, eu), dA, dW1, dW2, "%s" % ((M, K, N),))


@pytest.mark.parametrize("M,K,N", SIZES + LARGE)
def test_block_backward(dev, M, K, N):
    t = case(dev, M, K, N, seed=2)
    dA, dW1, dW2, dW3 = sw.swiglu_mlp_train_backward(t["dZ"], t["A"], t["W1"], t["W2"], t["W3"], t["G"], t["U"],
                                                     t["Y"])
    x = d64(t)
    dY = x["dZ"] @ x["W3"].t()
    e = (K + 1) * F * (x["dZ"].abs() @ x["W3"].abs().t())
    check_products(x, *kept_grads(x, dY, e), dA, dW1, dW2, "%s" % ((M, K, N),))
    ref, S = x["Y"].t() @ x["dZ"], x["Y"].abs().t() @ x["dZ"].abs()
    check(dW3, ref, (M + 1) * F * (1 + H) * S + H * ref.abs(), ref, "%s dW3" % ((M, K, N),))


@pytest.mark.parametrize("M,K,N", [(5, 72, 136), (130, 200, 328)])
def test_partial_gradients_and_repeats(dev, M, K, N):
    """What is not asked for is not needed for the rest, and repeats are bitwise equal."""
    t = case(dev, M, K, N)
    args = [t[k] for k in ("dY", "A", "W1", "W2", "G", "U")]
    dA, dW1, dW2 = sw.swiglu_train_backward(*args)
    only_a = sw.swiglu_train_backward(*args, need_dW=False)
    only_w = sw.swiglu_train_backward(*args, need_dA=False)
    assert only_a[1] is None and only_a[2] is None and only_w[0] is None
    assert torch.equal(only_a[0], dA) and torch.equal(only_w[1], dW1) and torch.equal(only_w[2], dW2)
    bargs = [t[k] for k in ("dZ", "A", "W1", "W2", "W3", "G", "U")]
    full = sw.swiglu_mlp_train_backward(*bargs, t["Y"])
    assert torch.equal(sw.swiglu_mlp_train_backward(*bargs, None, need_dW=False)[0], full[0])
    again = sw.swiglu_mlp_train_backward(*bargs, t["Y"], need_dA=False)
    assert again[0] is None and all(torch.equal(p, q) for p, q in zip(again[1:], full[1:]))


def test_empty_batch(dev):
    t = case(dev, 0, 64, 72)
    Y, G, U = sw.swiglu_train_forward(t["A"], t["W1"], t["W2"])
    assert Y.shape == G.shape == U.shape == (0, 72)
    for out in (sw.swiglu_train_backward(t["dY"], t["A"], t["W1"], t["W2"], G, U),
                sw.swiglu_train_backward(t["dY"], t["A"], t["W1"], t["W2"]),
                sw.swiglu_mlp_train_backward(t["dZ"], t["A"], t["W1"], t["W2"], t["W3"], G, U, Y)):
        assert out[0].shape == (0, 64)
        for dW in out[1:]:
            assert not dW.any()


def fenced(t, fill):
    """A copy of t in the middle of a buffer of `fill` (whole 16-byte pieces)."""
    n, pad = t.numel(), 4096
    buf = torch.full((n + 2 * pad,), fill, dtype=t.dtype, device=t.device)
    v = buf[pad:pad + n].view(t.shape)
    v.copy_(t)
    return buf, v


@pytest.mark.parametrize("M,K,N", [(1, 8, 8), (65, 136, 264), (1003, 264, 584), (1500, 200, 8200)])
def test_nothing_outside_is_read_or_written(dev, M, K, N):
    """Inputs lie between NaNs, which must not reach a result; outputs lie between
    marks, which must stay."""
    t = case(dev, M, K, N)
    want = (sw.swiglu_train_forward(t["A"], t["W1"], t["W2"]) +
            sw.swiglu_train_backward(t["dY"], t["A"], t["W1"], t["W2"]) +
            sw.swiglu_mlp_train_backward(*(t[k] for k in ("dZ", "A", "W1", "W2", "W3", "G", "U", "Y"))))
    f = {k: fenced(v, float("nan"))[1] for k, v in t.items()}
    bufs, outs = zip(*(fenced(torch.zeros_like(w), 7.0) for w in want))
    sw.swiglu_train_forward(f["A"], f["W1"], f["W2"], *outs[:3])
    sw.swiglu_train_backward(f["dY"], f["A"], f["W1"], f["W2"], None, None, *outs[3:6])
    sw.swiglu_mlp_train_backward(*(f[k] for k in ("dZ", "A", "W1", "W2", "W3", "G", "U", "Y")), *outs[6:])
    for i, (b, o, w) in enumerate(zip(bufs, outs, want)):
        assert torch.equal(o, w), i
        edge = torch.cat((b[:4096], b[-4096:]))
        assert (edge == 7.0).all(), i


def test_extreme_gates(dev):
    """SiLU' at gates from -300 to 300: 0 and 1 in the limits, never NaN."""
    M, K, N = 4, 64, 64
    t = case(dev, M, K, N)
    vals = torch.tensor([-1e30, -300.0, -90.0, -88.0, -20.0, -1.2785, 0.0, 1e-30, 20.0, 88.0, 300.0, 1e30],
                        device=dev).to(torch.bfloat16)
    t["G"] = vals.repeat(22)[:M * N].view(M, N).contiguous()
    x = d64(t)
    dA, dW1, dW2 = sw.swiglu_train_backward(t["dY"], t["A"], t["W1"], t["W2"], t["G"], t["U"])
    # finite U and dY against gates of 1e30: dU up to 1e30, in range of bf16
    check_products(x, *kept_grads(x, x["dY"], 0.0), dA, dW1, dW2, "extreme")


def test_autograd_against_differences(dev):
    """The differentiable forms' gradients against central differences of the
    fp64 function along random directions.  The gradient's relative error from
    its bf16 roundings is below 2 x 2^-8 along a direction of random signs, and
    the difference quotient's below 1e-6."""
    M, K, N = 40, 64, 136
    t = case(dev, M, K, N)

    def f64(A, W1, W2, W3=None):
        g = A @ W1
        y = g * sig(g) * (A @ W2)
        return y if W3 is None else y @ W3

    for names, fn, up in (("A W1 W2", lambda *a: sw.swiglu(*a), "dY"),
                          ("A W1 W2", lambda *a: sw.swiglu(*a, recompute=True), "dY"),
                          ("A W1 W2 W3", lambda *a: sw.swiglu_mlp(*a), "dZ")):
        names = names.split()
        leaves = [t[n].clone().requires_grad_() for n in names]
        out = fn(*leaves)
        out.backward(t[up])
        x = [t[n].double() for n in names]
        w = t[up].double()
        gen = torch.Generator(device=dev).manual_seed(5)
        for i, leaf in enumerate(leaves):
            v = torch.randn(x[i].shape, generator=gen, device=dev, dtype=torch.float64)
            h = 1e-5
            hi = [y + h * v if j == i else y for j, y in enumerate(x)]
            lo = [y - h * v if j == i else y for j, y in enumerate(x)]
            num = float(((f64(*hi) - f64(*lo)) * w).sum()) / (2 * h)
            ana = float((leaf.grad.double() * v).sum())
            # the scale of the sum, as random signs add up
            scale = float((leaf.grad.double() * v).pow(2).sum().sqrt())
            assert abs(num - ana) <= 6 * 2 * H * scale + 1e-6 * abs(num), (names[i], num, ana, scale)


def test_autograd_needs_and_shapes(dev):
    t = case(dev, 24, 64, 72)
    A = t["A"].view(2, 12, 64).clone().requires_grad_()
    Y = sw.swiglu(A, t["W1"], t["W2"])
    assert Y.shape == (2, 12, 72)
    Y.sum().backward()          # an expanded (stride 0) gradient
    ones = torch.ones(24, 72, dtype=torch.bfloat16, device=dev)
    _, G, U = sw.swiglu_train_forward(t["A"], t["W1"], t["W2"])
    want = sw.swiglu_train_backward(ones, t["A"], t["W1"], t["W2"], G, U)
    assert torch.equal(A.grad.view(24, 64), want[0])
    W1 = t["W1"].clone().requires_grad_()
    sw.swiglu(t["A"], W1, t["W2"]).sum().backward()
    assert torch.equal(W1.grad, want[1])
    # a non-contiguous activation
    At = t["A"].t().contiguous().t().requires_grad_()
    sw.swiglu(At, t["W1"], t["W2"]).sum().backward()
    assert torch.equal(At.grad, want[0])


def test_other_stream(dev):
    t = case(dev, 130, 200, 328)
    args = [t[k] for k in ("dY", "A", "W1", "W2", "G", "U")]
    want = sw.swiglu_train_backward(*args)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = sw.swiglu_train_backward(*args, stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_graph_replays(dev):
    """A captured forward and backward, replayed with new inputs, with eager work
    and synchronisations between the replays."""
    M, K, N = 65, 896, 520
    t = case(dev, M, K, N)
    live = {k: v.clone() for k, v in t.items()}
    run = lambda d: (sw.swiglu_train_forward(d["A"], d["W1"], d["W2"]) +   # noqa: E731
                     sw.swiglu_train_backward(d["dY"], d["A"], d["W1"], d["W2"], d["G"], d["U"]) +
                     sw.swiglu_mlp_train_backward(*(d[k] for k in ("dZ", "A", "W1", "W2", "W3", "G", "U", "Y"))))
    run(live)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = run(live)
    for seed in (3, 4, 5):
        fresh = case(dev, M, K, N, seed=seed)
        for k in live:
            live[k].copy_(fresh[k])
        want = run(fresh)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, want)), seed
