"""The training and adapter operators as a program issues them: empty batches, other
streams, captures and several threads."""
import threading

import pytest
import torch

import swiglu_gated_mlp_amd as sw

pytestmark = pytest.mark.gpu

BF = dict(dtype=torch.bfloat16)


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    return torch.device("cuda:0")


@pytest.mark.parametrize("lead", [(0,), (2, 0)])
@pytest.mark.parametrize("fn", ["kept", "recomputed", "block"])
def test_backward_of_an_empty_batch(dev, fn, lead):
    """No rows: an empty gradient of A in A's own shape, zeros for the weights."""
    K, N = 64, 72
    A = torch.zeros(*lead, K, device=dev, **BF).requires_grad_()
    W = [torch.ones(*s, device=dev, **BF).requires_grad_() for s in ((K, N), (K, N), (N, K))]
    if fn == "block":
        out = sw.swiglu_mlp(A, *W)
    else:
        W.pop()
        out = sw.swiglu(A, *W, recompute=fn == "recomputed")
    assert out.shape == (*lead, W[-1].shape[1])
    out.float().sum().backward()
    assert A.grad.shape == A.shape
    for w in W:
        assert w.grad.shape == w.shape and not w.grad.any()


def stream_of(t):
    """Handle of the stream that t's memory belongs to in the allocator."""
    for seg in torch.cuda.memory_snapshot():
        if seg["address"] <= t.data_ptr() < seg["address"] + seg["total_size"]:
            return seg["stream"]


def test_default_stream_given_beside_another(dev):
    """stream=0 and the default stream's object, with a side stream current: outputs and
    workspaces belong to the default stream, on which they are used."""
    M, K, N = 130, 200, 328
    g = torch.Generator(device=dev).manual_seed(1)
    A, W1, W2 = (torch.randn(*s, generator=g, device=dev).to(torch.bfloat16) for s in ((M, K), (K, N), (K, N)))
    want = sw.swiglu_train_forward(A, W1, W2)
    torch.cuda.synchronize()
    with torch.cuda.stream(torch.cuda.Stream()):
        for stream in (0, torch.cuda.default_stream()):
            ws = sw.Workspace(dev)
            got = sw.swiglu_train_forward(A, W1, W2, workspace=ws, stream=stream)
            assert [stream_of(t) for t in got] == [0, 0, 0]
            assert stream_of(sw.Workspace(dev).get(1 << 20, 0)) == 0
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(got, want))


def operators(dev, M, K, N, seed):
    """A batch, and its training and adapter calls as fn(stream) -> outputs."""
    L, r = 5, 16
    g = torch.Generator(device=dev).manual_seed(seed)

    def rnd(*shape):
        return (torch.randn(*shape, generator=g, device=dev) * shape[-2] ** -0.5).to(torch.bfloat16)

    dZ, dY, A, G, U, Y = rnd(M, K), rnd(M, N), rnd(M, K), rnd(M, N), rnd(M, N), rnd(M, N)
    W1, W2, W3 = rnd(K, N), rnd(K, N), rnd(N, K)
    ids = (torch.arange(M, device=dev) * 7 // 3 % (L + 1) - 1).int()
    scales = torch.rand(L, generator=g, device=dev) + 0.5
    Wp, Wg = sw.swiglu_pack_weights(W1, W2), sw.swiglu_gemm_pack_weight(W1)
    Lp = sw.swiglu_lora_pack(rnd(L, K, r), rnd(L, r, N), rnd(L, K, r), rnd(L, r, N))
    Lg = sw.swiglu_gemm_lora_pack(rnd(L, K, r), rnd(L, r, N))
    return (lambda s=None: sw.swiglu_train_forward(A, W1, W2, stream=s) +
            sw.swiglu_train_backward(dY, A, W1, W2, stream=s) +
            sw.swiglu_mlp_train_backward(dZ, A, W1, W2, W3, G, U, Y, stream=s) +
            (sw.swiglu_fused_packed_lora(A, Wp, Lp, ids, scales, N, r, stream=s),
             sw.swiglu_gemm_packed_lora(A, Wg, Lg, ids, scales, N, r, stream=s)))


# adapters' factors read in the lanes, from memory, and on the matrix units; split and whole products
BATCHES = [(16, 200, 264), (130, 1096, 776), (600, 2048, 520)]


def test_capture_forked_to_another_stream(dev):
    """Calls given a side stream of a capture, with the capturing stream's own allocations
    and writes beside them: every replay gives the eager results."""
    runs = [operators(dev, *b, seed) for seed, b in enumerate(BATCHES)]
    want = [run() for run in runs]
    torch.cuda.synchronize()
    side, graph, outs = torch.cuda.Stream(), torch.cuda.CUDAGraph(), []
    with torch.cuda.graph(graph):
        main = torch.cuda.current_stream()
        side.wait_stream(main)
        for run in runs:
            outs.append(run(side))
            for log in range(9, 25):   # blocks of every size the calls could have left behind
                torch.empty(1 << log, dtype=torch.uint8, device=dev).fill_(0xFF)
        main.wait_stream(side)
    for _ in range(4):
        for out in outs:
            for t in out:
                t.fill_(7.0)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.isfinite(torch.randn(1 << 16, device=dev).sum())
        for out, ref in zip(outs, want):
            assert all(torch.equal(a, b) for a, b in zip(out, ref))


def test_threads_on_one_stream(dev):
    """Calls of different sizes from several threads, all on the default stream, give what
    one thread's calls give; and no call keeps memory after it."""
    runs = [operators(dev, *b, seed) for seed, b in enumerate(BATCHES)]
    want = [run() for run in runs]
    torch.cuda.synchronize()
    before = torch.cuda.memory_allocated(dev)
    for run in runs:
        run()
    torch.cuda.synchronize()
    assert torch.cuda.memory_allocated(dev) == before
    wrong, gate = [], threading.Barrier(len(runs), timeout=60)

    def thread(run, ref):
        try:
            gate.wait()
            for i in range(30):
                wrong.extend((i, j) for j, (a, b) in enumerate(zip(run(), ref)) if not torch.equal(a, b))
        except Exception as e:   # noqa: BLE001
            wrong.append(e)
            gate.abort()

    threads = [threading.Thread(target=thread, args=a) for a in zip(runs, want)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong


def test_block_gradients_from_threads(dev):
    """Forward and backward passes of the differentiable block in two threads: the backward
    passes run on autograd's thread beside the other's calls."""
    def weights(M, K, N):
        g = torch.Generator(device=dev).manual_seed(M)
        return [(torch.randn(*s, generator=g, device=dev) * s[0] ** -0.5).to(torch.bfloat16).requires_grad_()
                for s in ((M, K), (K, N), (K, N), (N, K))]

    def step(leaves):
        Z = sw.swiglu_mlp(*leaves)
        return (Z.detach(),) + torch.autograd.grad(Z, leaves, torch.ones_like(Z))

    sets = [weights(333, 896, 1160), weights(70, 264, 2056)]
    want = [step(s) for s in sets]
    torch.cuda.synchronize()
    wrong = []

    def thread(leaves, ref):
        try:
            for i in range(30):
                wrong.extend((i, j) for j, (a, b) in enumerate(zip(step(leaves), ref)) if not torch.equal(a, b))
        except Exception as e:   # noqa: BLE001
            wrong.append(e)

    threads = [threading.Thread(target=thread, args=a) for a in zip(sets, want)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong
