"""Training and adapter operators on matrices of more than 2^31 elements or bytes:
rows and columns across their whole range against the definition in fp64, with the
bounds of the small cases."""
import pytest
import torch

import swiglu_gated_mlp_amd as sw
import test_gpu_lora as lora
import test_gpu_train as train

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    yield torch.device("cuda:0")
    torch.cuda.empty_cache()


def spread(n, count, *more):
    """`count` indexes at each end of n, and some around the given ones."""
    near = [i for m in more for i in range(max(0, m - 3), min(n, m + 3))]
    return torch.tensor(sorted(set(range(count)) | set(near) | set(range(n - count, n))))


def test_training(dev):
    M, K, N = 66001, 72, 33000   # M N = 2^31 + 3e7 elements
    t = train.case(dev, M, K, N)
    Y, G, U = sw.swiglu_train_forward(t["A"], t["W1"], t["W2"])
    rows, cols = spread(M, 40, 32541, 65081).to(dev), spread(N, 8, 16500).to(dev)   # byte offsets 2^31, 2^32
    x = {k: (v[rows] if k in ("A", "dY", "G", "U", "Y") else v).double() for k, v in t.items()}
    g, u, eg, eu = train.sums(x)
    H = train.H
    train.check(G[rows], g, eg * (1 + H) + H * g.abs(), g + eg, "G")
    train.check(U[rows], u, eu * (1 + H) + H * u.abs(), u + eu, "U")
    h = g * train.sig(g)
    e = u.abs() * (1.1 * eg + h.abs() * (g.abs() + 8) * 2.0 ** -23) + (h.abs() + 1.1 * eg) * eu
    train.check(Y[rows], h * u, e * (1 + H) + H * (h * u).abs(), h * u + e, "Y")
    del Y, G, U
    dA, dW1, dW2 = sw.swiglu_train_backward(t["dY"], t["A"], t["W1"], t["W2"], t["G"], t["U"])
    train.check_products(x, *train.kept_grads(x, x["dY"], 0.0), dA[rows], None, None, "rows")
    c = {k: t[k][:, cols].double() for k in ("dY", "G", "U", "W1", "W2")}
    c["A"] = t["A"].double()
    train.check_products(c, *train.kept_grads(c, c["dY"], 0.0), None, dW1[:, cols], dW2[:, cols], "columns")


@pytest.mark.parametrize("M,K,N", [(60001, 18944, 72), (60001, 72, 36000)])
def test_adapters(dev, M, K, N):
    L, r = 3, 20
    t = lora.case(dev, M, K, N, L, r, ("1", "2", ""), "runs")
    Y, C = lora.gated(t, r), lora.plain(t, r)
    # 30208: where a batch of more than 2^31 bytes is cut; the others: offsets of Y
    rows = spread(M, 40, 30208, 29826, 59652).to(dev)
    x = dict(t, A=t["A"][rows], ids=t["ids"][rows])
    lora.check_gated(Y[rows], x, "%s" % ((M, K, N),))
    lora.check_plain(C[rows], x, "%s" % ((M, K, N),))
