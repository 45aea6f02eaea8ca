"""The training and adapter operators as a program issues them: empty batches, other
streams, captures and several threads."""
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
