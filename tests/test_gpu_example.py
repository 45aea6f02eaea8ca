"""The example that trains a block, fine-tunes it and serves the variants together."""
import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu


def test_finetune_and_serve():
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples",
                        "finetune_and_serve.py")
    spec = importlib.util.spec_from_file_location("finetune_and_serve", path)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    losses, worst = m.main(steps=30, K=136, N=264, rank=4, tasks=2, rows=256, out=lambda s: None)
    assert losses[-1] < 0.8 * losses[0]
    # Y is rounded once (2^-8 at most, so below that in the mean), Z once more, and the
    # merged weights are not
    assert worst < 2 * 2.0 ** -8
