"""The probe of the int8 kernels' forms: its refusals, and what it says of plain shapes."""
import pytest

import swiglu_gated_mlp_amd as sw


def test_form_probe():
    for gemm in (False, True):
        assert sw.swiglu_probe_int8_form(gemm, 8, 3584, 18944)["panels"] == 0
        for K, ragged in ((3584, False), (3600, True)):
            assert sw.swiglu_probe_int8_form(gemm, 8192, K, 4864)["ragged"] is ragged
        for bad in ((0, 64, 72), (4, 72, 64), (4, 64, 60), (4, 131072, 64)):
            with pytest.raises(ValueError, match="invalid shape"):
                sw.swiglu_probe_int8_form(gemm, *bad)
        # activations past 2 GiB run in chunks
        f = sw.swiglu_probe_int8_form(gemm, 20000, 131056, 24)
        assert f["ragged"] and f["tail"] == f["panels"] == 0 and not f["wide"]
    assert sw.lib().swiglu_probe_int8_form(0, 4, 64, 72, None) == 0
