"""What include/swiglu.h promises of a kept element's error, held against the definition
of its scale (max |x| / 127 rounded up to bf16, at least 2^-126) in fp64, on the CPU."""
import os
import re

import torch

HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "swiglu.h")


def stated():
    """n of the header's bound max |x| / n."""
    with open(HEADER) as f:
        text = re.sub(r"\s*\n \*\s*", " ", f.read())
    return int(re.search(r"max \|x\| of its group / (\d+)", text).group(1))


def kept_scale(top):
    t = torch.as_tensor(top, dtype=torch.float32) / torch.full((), 127.0)
    up = (t.view(torch.int32) + 0xFFFF) >> 16 << 16
    return up.view(torch.float32).clamp_min(2.0 ** -126).double()


def test_half_a_step_is_within_the_stated_bound():
    """Largest magnitudes of every mantissa and of exponents all over the range: half a
    step, and the 2^-16 of one by which a code may be beside the nearest."""
    mantissa = torch.arange(1 << 23, dtype=torch.int32)
    worst = 0.0
    for exponent in (-119, -20, -1, 0, 1, 7, 100, 127):
        top = (mantissa + ((exponent + 127) << 23)).view(torch.float32)
        worst = max(worst, float((kept_scale(top) * (0.5 + 2.0 ** -16) / top.double()).max()))
    # nothing to spare: the next whole number would not hold
    assert worst <= 1.0 / stated() and worst > 1.0 / (stated() + 1)


def test_tiny_groups_have_steps_of_their_own():
    """Below 127 * 2^-126 the scale stays and half a step is 2^-127."""
    top = torch.tensor([0.0, 2.0 ** -126, 100 * 2.0 ** -126, 127 * 2.0 ** -126])
    assert (kept_scale(top) == 2.0 ** -126).all()
    with open(HEADER) as f:
        assert "2^-127" in f.read()
