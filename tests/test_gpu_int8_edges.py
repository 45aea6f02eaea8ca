"""Int8 calls at sizes and in uses that their documentation allows: weights and blocks
past 4 GiB, empty batches, the same tensor twice, graphs and threads side by side."""
import threading

import pytest
import torch

import swiglu_gated_mlp_amd as sw

from test_gpu_int8 import activations, block, check_fused, check_gemm, codes, dev, scales   # noqa: F401
from test_gpu_train_int8 import kept_case

pytestmark = pytest.mark.gpu


def test_weights_past_4gib(dev):   # noqa: F811
    """The packed weights' offsets pass 32 bits, in every kernel."""
    K, N = 65536, 40008
    unit = 2.0 ** -10
    W1, W2 = codes(dev, K, N, 1), codes(dev, K, N, 2)
    s1, s2 = scales(dev, N, 3, unit), scales(dev, N, 4, unit)
    Wp, Wg = sw.swiglu_pack_weights_int8(W1, W2), sw.swiglu_gemm_pack_weight_int8(W1)
    assert Wp.numel() > 1 << 32
    cols = [slice(0, 256), slice(N // 2, N // 2 + 256), slice(N - 264, N)]
    W1, W2 = [W1[:, c].clone() for c in cols], [W2[:, c].clone() for c in cols]
    for M in (1, 20, 40, 200, 600, 1500):
        A, sa = codes(dev, M, K, M), scales(dev, M, M + 1, unit)
        Y = sw.swiglu_fused_packed_int8(A, sa, Wp, s1, s2)
        C = sw.swiglu_gemm_packed_int8(A, sa, Wg, s1)
        for i, c in enumerate(cols):
            check_fused(Y[:, c], A, sa, W1[i], s1[c], W2[i], s2[c], "fused %d" % M)
            check_gemm(C[:, c], A, sa, W1[i], s1[c], "gemm %d" % M)


@pytest.mark.parametrize("K,N", [(131056, 64), (64, 131056)])
def test_a_block_in_row_chunks(dev, K, N):   # noqa: F811
    """Codes of A, or of Y, past 2 GiB: the block is its steps, bit for bit."""
    M = (1 << 31) // 131056 + 300
    _, w, _ = block(dev, 1, K, N, 3)
    A = torch.empty(M, K, dtype=torch.bfloat16, device=dev)
    g = torch.Generator(device=dev).manual_seed(5)
    for r in range(0, M, 4096):
        A[r:r + 4096] = torch.randn(min(4096, M - r), K, generator=g, device=dev).to(torch.bfloat16)
    Y, Z = sw.swiglu_mlp_packed_int8(A, *w)
    Q, sa = sw.swiglu_quantize_rows_int8(A)
    del A
    assert torch.equal(Y, sw.swiglu_fused_packed_int8(Q, sa, w[0], w[1], w[2]))
    Q, sy = sw.swiglu_quantize_rows_int8(Y)
    assert torch.equal(Z, sw.swiglu_gemm_packed_int8(Q, sy, w[3], w[4]))
    # rows by themselves take another kernel, and the sums are whole numbers
    for r in (slice(0, 40), slice(M // 2, M // 2 + 40), slice(M - 40, M)):
        assert torch.equal(Z[r], sw.swiglu_gemm_packed_int8(Q[r].contiguous(), sy[r].contiguous(), w[3], w[4]))


def test_empty_batches(dev):   # noqa: F811
    N = 72
    kept = torch.empty(0, 3, 2, 32, dtype=torch.int8, device=dev), torch.empty(3, 0, 2, dtype=torch.bfloat16, device=dev)
    for x in sw.swiglu_dequantize_kept_int8(*kept, N):
        assert x.shape == (0, N)
    A = torch.empty(2, 0, 64, dtype=torch.bfloat16, device=dev, requires_grad=True)
    W = [activations(dev, *s, 1).requires_grad_() for s in ((64, N), (64, N), (N, 64))]
    Z = sw.swiglu_mlp(A, *W, keep="int8")
    assert Z.shape == (2, 0, 64)
    Z.sum().backward()
    assert A.grad.shape == A.shape and not any(w.grad.any() for w in W)


def test_no_gradient_asked_for(dev):   # noqa: F811
    t = kept_case(dev, 40, 64, 136)
    none = sw.swiglu_train_backward_int8(t["dY"], t["A"], t["W1"], t["W2"], t["codes"], t["scales"], need_dA=False,
                                         need_dW=False)
    assert none == (None, None, None)
    none = sw.swiglu_mlp_train_backward_int8(*(t[k] for k in ("dZ", "A", "W1", "W2", "W3", "codes", "scales")),
                                             need_dA=False, need_dW=False)
    assert none == (None, None, None, None)


def test_the_same_tensor_twice(dev):   # noqa: F811
    """Both weights, both scales, gradient and activations may be one tensor."""
    M, K = 70, 144
    W, s = codes(dev, K, K, 1), scales(dev, K, 2, 2.0 ** -9)
    A, sa = codes(dev, M, K, 3), scales(dev, M, 4, 2.0 ** -9)
    Wp = sw.swiglu_pack_weights_int8(W, W)
    check_fused(sw.swiglu_fused_packed_int8(A, sa, Wp, s, s), A, sa, W, s, W, s, "one weight twice")
    assert torch.equal(Wp, sw.swiglu_pack_weights_int8(W, W.clone()))
    t = kept_case(dev, M, K, K)
    same = sw.swiglu_mlp_train_backward_int8(t["A"], t["A"], t["W1"], t["W1"], t["W1"], t["codes"], t["scales"])
    own = sw.swiglu_mlp_train_backward_int8(t["A"].clone(), t["A"], t["W1"], t["W1"].clone(), t["W1"].clone(),
                                            t["codes"], t["scales"])
    assert all(torch.equal(a, b) for a, b in zip(same, own))
    w = t["W1"].clone().requires_grad_()
    sw.swiglu_mlp(t["A"], w, w, w, keep="int8").backward(t["A"])
    leaves = [t["W1"].clone().requires_grad_() for _ in range(3)]
    sw.swiglu_mlp(t["A"], *leaves, keep="int8").backward(t["A"])
    total = sum(x.grad.double() for x in leaves)
    # two additions of gradients, each rounded to bf16
    bound = 2 * 2.0 ** -8 * (1 + 2.0 ** -8) * sum(x.grad.double().abs() for x in leaves)
    assert ((w.grad.double() - total).abs() <= bound).all()


def test_backward_twice(dev):   # noqa: F811
    t = kept_case(dev, 130, 200, 328)
    leaves = [t[k].clone().requires_grad_() for k in ("A", "W1", "W2", "W3")]
    Z = sw.swiglu_mlp(*leaves, keep="int8")
    first = torch.autograd.grad(Z, leaves, t["dZ"], retain_graph=True)
    again = torch.autograd.grad(Z, leaves, t["dZ"])
    assert all(torch.equal(a, b) for a, b in zip(first, again))


def test_a_captured_step_of_autograd(dev):   # noqa: F811
    """Forward and backward of both forms in a graph, replayed on new inputs."""
    M, K, N = 70, 200, 328
    t = kept_case(dev, M, K, N)
    live = {k: t[k].clone().requires_grad_(k in ("A", "W1", "W2", "W3")) for k in ("A", "W1", "W2", "W3", "dY", "dZ")}

    def step(d):
        a = [d["A"], d["W1"], d["W2"]]
        Y = sw.swiglu(*a, keep="int8")
        Z = sw.swiglu_mlp(*a, d["W3"], keep="int8")
        return (Y.detach(), Z.detach(), *torch.autograd.grad(Y, a, d["dY"]),
                *torch.autograd.grad(Z, a + [d["W3"]], d["dZ"]))

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(live)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        outs = step(live)
    for seed in (3, 4, 5):
        fresh = kept_case(dev, M, K, N, seed=seed)
        with torch.no_grad():
            for k in live:
                live[k].copy_(fresh[k])
        want = step({k: fresh[k].requires_grad_(k in ("A", "W1", "W2", "W3")) for k in live})
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, want)), seed


def test_two_graphs_side_by_side(dev):   # noqa: F811
    """Graphs of the block without a workspace have buffers of their own: replayed on
    two streams at once, with eager calls between."""
    K, N = 14336, 528
    _, w, _ = block(dev, 1, K, N, 9)
    xs = [activations(dev, 100, K, 30 + i) for i in range(2)]
    want = [sw.swiglu_mlp_packed_int8(x, *w) for x in xs]
    torch.cuda.synchronize()
    graphs, outs, streams = [], [], [torch.cuda.Stream() for _ in xs]
    for x, s in zip(xs, streams):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            outs.append(sw.swiglu_mlp_packed_int8(x, *w))
        graphs.append(g)
    for _ in range(4):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        eager = sw.swiglu_mlp_packed_int8(xs[0], *w)
        torch.cuda.synchronize()
        for (Y, Z), (y, z) in zip(outs + [eager], want + [want[0]]):
            assert torch.equal(Y, y) and torch.equal(Z, z)
            if Y is not eager[0]:
                Y.zero_(), Z.zero_()
        torch.cuda.synchronize()


def test_two_threads_at_once(dev):   # noqa: F811
    """Each on a stream of its own, without a workspace."""
    _, w, _ = block(dev, 1, 896, 1040, 5)
    xs = [activations(dev, m, 896, m) for m in (1, 40, 100, 333)]
    want = [sw.swiglu_mlp_packed_int8(x, *w) for x in xs]
    torch.cuda.synchronize()
    wrong = []

    def work(i):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(20):
                    for x, (y, z) in zip(xs[i:] + xs[:i], want[i:] + want[:i]):
                        Y, Z = sw.swiglu_mlp_packed_int8(x, *w)
                        if not (torch.equal(Y, y) and torch.equal(Z, z)):
                            wrong.append((i, len(x)))
        except Exception as e:   # noqa: BLE001
            wrong.append((i, repr(e)))

    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    for x in threads:
        x.start()
    for x in threads:
        x.join()
    assert not wrong, wrong[:4]
