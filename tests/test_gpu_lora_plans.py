"""Adapters on the launches that only wide or very deep products reach: 256- and 128-row
tiles in one launch, and chunks of rows with a short last one."""
import pytest
import torch

import swiglu_gated_mlp_amd as sw
import test_gpu_lora as lora

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    yield torch.device("cuda:0")
    torch.cuda.empty_cache()


# tiles of 256 x 128 (of the pack's columns) past one round of 256 CUs, the last round
# less than six tenths full: it runs as 128-row tiles, which share the lists of 256 rows
@pytest.mark.parametrize("kind", ["runs", "mixed"])
@pytest.mark.parametrize("K", [128, 200])
@pytest.mark.parametrize("M,N,pairs", [(1100, 8200, ("1", "2")), (1100, 16648, ("",)), (1351, 11800, ("",))])
def test_two_tile_heights_in_one_launch(dev, M, N, pairs, K, kind):
    t = lora.case(dev, M, K, N, 12, 24, pairs, kind, seed=3)
    if pairs == ("",):
        lora.check_plain(lora.plain(t, 24), t, kind)
    else:
        lora.check_gated(lora.gated(t, 24), t, kind)


def test_short_last_chunk(dev):
    """K = 2^22: rows go in chunks of at most 256, and the last one's take the schedule and
    the adapter form of a short batch.  A is zero but in 300 columns, so that a sum has 300
    terms and the bound of one of 300."""
    M, K, N, L, r, kept = 261, 1 << 22, 72, 2, 8, 300
    g = torch.Generator(device=dev).manual_seed(4)
    cols = torch.randperm(K, generator=torch.Generator().manual_seed(5))[:kept].sort().values.to(dev)
    cols[0], cols[-1] = 0, K - 1
    s = lora.case(dev, M, kept, N, L, r, ("1", "2", ""), "mixed", seed=4)
    t = dict(s, A=torch.zeros(M, K, dtype=torch.bfloat16, device=dev))
    t["A"][:, cols] = s["A"]
    for x in ("1", "2", ""):
        t["W" + x] = (torch.randn(K, N, generator=g, device=dev) * 0.1).to(torch.bfloat16)
        t["La" + x] = (torch.randn(L, K, r, generator=g, device=dev) * 0.1).to(torch.bfloat16)
        t["W" + x][cols], t["La" + x][:, cols] = s["W" + x], s["La" + x]
    lora.check_gated(lora.gated(t, r), s, "chunks")
    lora.check_plain(lora.plain(t, r), s, "chunks")
