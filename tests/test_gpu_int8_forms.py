"""Int8 products in every form of the kernels for many rows (256-row tiles, with
128-row tiles behind them, panels) and of the decode kernel, with K a multiple of 128
(as model widths are) and not, against the definition in fp64; bounds as in
test_gpu_int8.py."""
import pytest

import swiglu_gated_mlp_amd as sw

from test_gpu_int8 import check_fused, check_gemm, dev, pair  # noqa: F401

pytestmark = pytest.mark.gpu

# K of 3 n, 3 n + 1 and 3 n + 2 blocks of 128; rows and columns that end inside a tile
MANY = [(2048, 896, 4864), (8192, 896, 4864), (8192, 912, 4864), (4096, 3584, 18944), (4096, 18944, 3584),
        (4096, 18960, 3584), (3000, 1024, 12000), (2560, 1152, 8448), (5000, 2560, 4104), (1300, 3600, 18952),
        (8190, 3600, 4872), (200, 8192, 29568), (200, 8208, 29568), (130, 8320, 30008), (1800, 3600, 18952)]
FEW = [(1, 1024, 25000), (1, 1040, 25000), (4, 896, 4864), (4, 1040, 520), (8, 3584, 1024), (8, 16384, 1024),
       (7, 144, 136), (12, 2048, 65544), (12, 2064, 65544), (16, 896, 520), (16, 912, 520), (30, 8192, 24584),
       (17, 1024, 1040), (32, 9440, 4096), (31, 2064, 65544), (20, 256, 17144), (31, 416, 12664), (33, 896, 4864),
       (64, 4880, 904), (1, 16384, 5120)]


def run(dev, M, K, N):   # noqa: F811
    A, sa, W1, s1, W2, s2 = pair(dev, M, K, N, M + K + N)
    check_fused(sw.swiglu_fused_packed_int8(A, sa, sw.swiglu_pack_weights_int8(W1, W2), s1, s2), A, sa, W1, s1, W2, s2,
                "fused")
    check_gemm(sw.swiglu_gemm_packed_int8(A, sa, sw.swiglu_gemm_pack_weight_int8(W1), s1), A, sa, W1, s1, "gemm")


@pytest.mark.parametrize("M,K,N", MANY)
def test_many_rows(dev, M, K, N):   # noqa: F811
    run(dev, M, K, N)


@pytest.mark.parametrize("M,K,N", FEW)
def test_few_rows(dev, M, K, N):   # noqa: F811
    run(dev, M, K, N)


def test_the_forms_are_met(dev):   # noqa: F811
    """As the shapes above are planned on this device."""
    met = set()
    for gemm in (False, True):
        for shape in MANY + FEW:
            kernel, f = sw.swiglu_probe_int8_plan(gemm, *shape)["kernel"], sw.swiglu_probe_int8_form(gemm, *shape)
            if kernel == "stream":
                met.add((gemm, "panels" if f["panels"] else "tail" if f["tail"] else "tiles", f["ragged"]))
            elif kernel == "decode":
                met.add((gemm, f["wide"], *(shape[0] <= m for m in (4, 8, 16, 32)), f["ragged"]))
    for ragged in (False, True):
        for gemm in (False, True):
            assert (gemm, "tiles", ragged) in met and (gemm, "tail", ragged) in met, (gemm, ragged)
        assert (False, "panels", ragged) in met
        # workgroups of one or two groups of columns: up to 4, 8, 16, 32 rows and above; of many: up to 8, 16, 32
        upto = {m: tuple(m <= x for x in (4, 8, 16, 32)) for m in (4, 8, 16, 32, 64)}
        for m in (4, 8, 16, 32):
            assert (False, False, *upto[m], ragged) in met and (True, False, *upto[m], ragged) in met, (m, ragged)
        assert (True, False, *upto[64], ragged) in met
        assert any((False, True, *upto[m], ragged) in met for m in (4, 8, 16, 32))
        for m in (16, 32):
            assert (True, True, *upto[m], ragged) in met, (m, ragged)
