"""Training calls on the plans that their large products use -- whole tiles, and the last
round's split over the contraction -- in every product that has one, and recomputation and
the block on matrices of more than 2^31 elements.  Bounds as for the small cases."""
import pytest
import torch

import swiglu_gated_mlp_amd as sw
import test_gpu_train as train
from test_gpu_operators_large import spread

pytestmark = pytest.mark.gpu

H, F = train.H, train.F


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    yield torch.device("cuda:0")
    torch.cuda.empty_cache()


def splits_the_rest(launch, product, M, K, N):
    p = sw.swiglu_probe_train_plan(launch, M, K, N)[product]
    assert p["whole"] > 0 and p["rest"] > 0 and p["splits"] > 1, (launch, product, p)


@pytest.mark.parametrize("M,K,N", [(3157, 536, 2456), (1363, 544, 5384)])
def test_forward(dev, M, K, N):
    splits_the_rest("forward", 0, M, K, N)
    t = train.case(dev, M, K, N, seed=6)
    Y, G, U = sw.swiglu_train_forward(t["A"], t["W1"], t["W2"])
    x = train.d64({k: t[k] for k in ("A", "W1", "W2")})
    g, u, eg, eu = train.sums(x)
    for got, ref, e, name in ((G, g, eg, "G"), (U, u, eu, "U")):
        train.check(got, ref, e * (1 + H) + H * ref.abs(), ref + e, name)
    h = g * train.sig(g)
    e = u.abs() * (1.1 * eg + h.abs() * (g.abs() + 8) * 2.0 ** -23) + (h.abs() + 1.1 * eg) * eu
    train.check(Y, h * u, e * (1 + H) + H * (h * u).abs(), h * u + e, "Y")


@pytest.mark.parametrize("M,K,N", [(3157, 536, 2456), (1363, 544, 5384)])
def test_recomputed(dev, M, K, N):
    splits_the_rest("recomputed", 0, M, K, N)
    t = train.case(dev, M, K, N, seed=7)
    out = sw.swiglu_train_backward(t["dY"], t["A"], t["W1"], t["W2"])
    x = train.d64(t)
    x["G"], x["U"], eg, eu = train.sums(x)
    train.check_products(x, *train.kept_grads(x, x["dY"], 0.0, eg, eu), *out, "recomputed")


@pytest.mark.parametrize("launch,product,M,K,N", [
    ("da", 0, 6412, 2384, 264), ("da", 0, 2371, 6424, 272), ("dw", 0, 522, 3136, 2472), ("dw", 0, 541, 1064, 6616),
    ("da_dw", 0, 4112, 3872, 464), ("da_dw", 0, 2051, 7816, 464), ("da_dw", 1, 1003, 4048, 2112),
    ("da_dw", 1, 1400, 1712, 4832)])
def test_gradients(dev, launch, product, M, K, N):
    splits_the_rest(launch, product, M, K, N)
    t = train.case(dev, M, K, N, seed=8)
    out = sw.swiglu_train_backward(*(t[k] for k in ("dY", "A", "W1", "W2", "G", "U")), need_dA=launch != "dw",
                                   need_dW=launch != "da")
    x = train.d64(t)
    train.check_products(x, *train.kept_grads(x, x["dY"], 0.0), *out, launch)


@pytest.mark.parametrize("launch,product,M,K,N", [
    ("dy", 0, 3093, 528, 4928), ("dy", 0, 7305, 544, 2056), ("dy_dw3", 0, 2125, 1024, 7728),
    ("dy_dw3", 0, 2814, 1048, 6160), ("dy_dw3", 1, 984, 2064, 7856), ("dy_dw3", 1, 951, 2128, 7936)])
def test_block(dev, launch, product, M, K, N):
    splits_the_rest(launch, product, M, K, N)
    t = train.case(dev, M, K, N, seed=9)
    dA, dW1, dW2, dW3 = sw.swiglu_mlp_train_backward(*(t[k] for k in ("dZ", "A", "W1", "W2", "W3", "G", "U", "Y")),
                                                     need_dW=launch != "dy")
    x = train.d64(t)
    dY = x["dZ"] @ x["W3"].t()
    e = (K + 1) * F * (x["dZ"].abs() @ x["W3"].abs().t())
    train.check_products(x, *train.kept_grads(x, dY, e), dA, dW1, dW2, launch)
    if dW3 is not None:
        ref, S = x["Y"].t() @ x["dZ"], x["Y"].abs().t() @ x["dZ"].abs()
        train.check(dW3, ref, (M + 1) * F * (1 + H) * S + H * ref.abs(), ref, launch + " dW3")


# M N = 2^31 + 3e7 elements; rows at byte offsets 2^31 and 2^32
LARGE, NEAR = (66001, 72, 33000), (32541, 65081)


def test_recomputed_past_two_to_31(dev):
    M, K, N = LARGE
    t = train.case(dev, M, K, N, seed=10)
    del t["G"], t["U"], t["Y"]
    dA, dW1, dW2 = sw.swiglu_train_backward(t["dY"], t["A"], t["W1"], t["W2"])
    rows, cols = spread(M, 40, *NEAR).to(dev), spread(N, 8, 16500).to(dev)
    for take in ("rows", "columns"):
        if take == "rows":
            x = {k: (v[rows] if k in ("A", "dY") else v).double() for k, v in t.items()}
            outs = dA[rows], None, None
        else:
            x = {k: t[k][:, cols].double() for k in ("dY", "W1", "W2")}
            x["A"] = t["A"].double()
            outs = None, dW1[:, cols], dW2[:, cols]
        x["G"], x["U"], eg, eu = train.sums(x)
        train.check_products(x, *train.kept_grads(x, x["dY"], 0.0, eg, eu), *outs, take)


def test_block_past_two_to_31(dev):
    M, K, N = LARGE
    t = train.case(dev, M, K, N, seed=11)
    dA, dW1, dW2, dW3 = sw.swiglu_mlp_train_backward(*(t[k] for k in ("dZ", "A", "W1", "W2", "W3", "G", "U", "Y")))
    rows, cols = spread(M, 40, *NEAR).to(dev), spread(N, 8, 16500).to(dev)
    for take in ("rows", "columns"):
        if take == "rows":
            x = {k: (t[k][rows] if k in ("A", "dZ", "G", "U") else t[k]).double()
                 for k in ("A", "dZ", "G", "U", "W1", "W2", "W3")}
            outs = dA[rows], None, None
        else:
            x = {k: t[k][:, cols].double() for k in ("G", "U", "Y", "W1", "W2")}
            x.update({k: t[k].double() for k in ("A", "dZ")}, W3=t["W3"][cols].double())
            outs = None, dW1[:, cols], dW2[:, cols]
        dY = x["dZ"] @ x["W3"].t()
        e = (K + 1) * F * (x["dZ"].abs() @ x["W3"].abs().t())
        train.check_products(x, *train.kept_grads(x, dY, e), *outs, take)
    ref, S = x["Y"].t() @ x["dZ"], x["Y"].abs().t() @ x["dZ"].abs()
    train.check(dW3[cols], ref, (M + 1) * F * (1 + H) * S + H * ref.abs(), ref, "dW3")
