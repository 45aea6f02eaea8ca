"""The bounds that include/swiglu.h states for int8 results, at their edges."""
import pytest
import torch

import swiglu_gated_mlp_amd as sw

from test_gpu_int8 import check_gemm, codes, dev, same, sums   # noqa: F401

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


@pytest.mark.parametrize("M", [1, 16, 40, 100, 400, 4100])
def test_large_column_scales_with_small_row_scales(dev, M):   # noqa: F811
    """C is (sum * sw) * sa in fp32 steps: finite up to a column scale below 2^97, beyond
    it infinite where the first step overflows, although the row's scale is small."""
    K, N = 256, 4872
    A, W = codes(dev, M, K, M), codes(dev, K, N, M + 1)
    sw_ = torch.full((N,), 2.0 ** 96, device=dev)
    sa = torch.full((M,), 2.0 ** -100, device=dev)
    Wg = sw.swiglu_gemm_pack_weight_int8(W)
    check_gemm(sw.swiglu_gemm_packed_int8(A, sa, Wg, sw_), A, sa, W, sw_, "gemm")
    sw_[::3] = 2.0 ** 111            # |sums| of 2^17 and more overflow
    C = sw.swiglu_gemm_packed_int8(A, sa, Wg, sw_)
    S = sums(A, W)
    want = ((S.float() * sw_) * sa[:, None]).to(torch.bfloat16)
    assert same(C, want) and torch.equal(C.isinf(), want.isinf())
    over = S.abs()[:, ::3] >= 2.0 ** 17
    assert over.any() and not over.all() and torch.equal(C[:, ::3].isinf(), over)
    # SiLU(G) U of G infinite and U > 0
    ones = torch.full((N,), 2.0 ** 96, device=dev)
    Y = sw.swiglu_fused_packed_int8(A, sa, sw.swiglu_pack_weights_int8(W, W), sw_, ones)
    assert torch.isfinite(Y[:, 1::3]).all() and not torch.isfinite(Y[:, ::3][over & (S[:, ::3] > 0)]).any()
