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
