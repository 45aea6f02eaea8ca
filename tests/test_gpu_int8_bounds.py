"""The bounds that include/swiglu.h states for int8 results, at their edges."""
import pytest
import torch

import swiglu_gated_mlp_amd as sw

from test_gpu_int8 import dev   # noqa: F401

pytestmark = pytest.mark.gpu


def test_a_kept_element_halfway_between_codes(dev):   # noqa: F811
    """A group whose scale is rounded up by nearly 2^-7 of it, and elements half a step
    from the next code.  G is exact: a row's only inputs are 1 and 2^-10."""
    M, K, N = 3, 8, 64
    A = torch.zeros(M, K, dtype=torch.bfloat16, device=dev)
    A[:, 0], A[:, 1] = 1.0, 2.0 ** -10
    W = torch.zeros(K, N, dtype=torch.bfloat16, device=dev)
    W[:2, ::32] = 127.0                                   # 127 (1 + 2^-10)
    step = 1.0 + 2.0 ** -7
    W[0, 1:32], W[0, 33:] = 0.5 * step, -0.5 * step       # 129 / 256: a bf16 number
    codes, scales = sw.swiglu_train_forward_int8(A, W, W)[1:]
    x = A.double() @ W.double()
    assert (scales.double() == step).all()
    kept = (codes.double() * scales.double().permute(1, 0, 2)[..., None])
    top = 127.0 * (1.0 + 2.0 ** -10)
    for which in (0, 1):
        err = (kept[:, :, which].reshape(M, N) - x).abs()
        assert (err <= top / 252).all() and float(err.max()) == 0.5 * step > top / 253
