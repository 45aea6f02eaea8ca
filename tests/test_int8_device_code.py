"""Checks of the int8 kernels' compiled code that no run shows: waits that count loads
rely on the loads' order, and a kernel that nothing launches is never run."""
import os
import re
import subprocess

import pytest

from swiglu_gated_mlp_amd import build


@pytest.fixture(scope="module")
def kernels(tmp_path_factory):
    """The instructions of the int8 unit's kernels, by their demangled names."""
    out = str(tmp_path_factory.mktemp("code") / "int8.s")
    cmd = [build.hipcc(), *build.compile_flags(), "-x", "hip", "-S", "--offload-device-only",
           os.path.join(build.CSRC, "int8_api.hip"), "-o", out]
    subprocess.run(cmd, check=True, stdout=subprocess.DEVNULL, stderr=subprocess.DEVNULL)
    with open(out) as f:
        text = f.read()
    symbols = re.findall(r"^\s*\.amdhsa_kernel (\S+)$", text, re.M)
    names = subprocess.run(["c++filt", *symbols], check=True, capture_output=True, text=True).stdout.splitlines()
    found = {}
    for symbol, name in zip(symbols, names):
        body = text[text.index("\n%s:" % symbol):]
        body = body[:body.index(".amdhsa_kernel")]
        found[name] = [x.split(";")[0].strip() for x in body.splitlines()]
    return found


def first_loads(code):
    """The loads before the first barrier: w weights (16 bytes a lane to registers), L to LDS, s the scales'
    rows (4 bytes); and the count of loads that the last wait before it leaves in flight."""
    loads, left = "", None
    for x in code:
        if x.startswith("s_barrier"):
            return loads, left
        if re.match(r"(global|buffer|flat)_load", x):
            loads += "L" if "lds" in x else "w" if "dwordx4" in x else "s"
        wait = re.search(r"vmcnt\((\d+)\)", x)
        left = int(wait.group(1)) if wait else left
    raise AssertionError("no barrier")


def test_narrow_kernels_issue_a_stage_after_the_other(kernels):
    """The wait for stage 0 leaves the loads of two stages in flight, which have to be
    stages 1 and 2: with a load of theirs before stage 0's, it would pass too early."""
    found = 0
    for name, code in kernels.items():
        tile = re.search(r"narrow_kernel<swq::Narrow<(\d+), (\d+), (\d+), (\d+), (\w+), (\w+)> >", name)
        if not tile:
            continue
        rows, waves, blocks, stages = (int(tile.group(i)) for i in range(1, 5))
        found += 1
        activations = -(-rows // 8 // waves)
        stage = "w" * 4 * blocks + "L" * activations
        loads, left = first_loads(code)
        # before them the scales: 4 a block of columns, 1 of 32 rows
        scales = "w" * 4 * blocks + "s" * (rows // 32)
        assert len(loads) == len(scales) + len(stage) * (stages - 1), (name, loads)
        for i in range(stages - 1):
            at = len(scales) + i * len(stage)
            assert sorted(loads[at:at + len(stage)]) == sorted(stage), (name, loads, i)
        assert left == len(stage) * (stages - 2), (name, left)
    assert found >= 20


def test_every_kernel_is_launched(kernels):
    """The unit holds no kernel that its host code does not launch."""
    host = ""
    for name in ("int8_api.hip", "launch.hpp"):
        with open(os.path.join(build.CSRC, name)) as f:
            host += f.read()
    launched = set(re.findall(r"&sw[kq]::(\w+)", host))
    for name in kernels:
        assert re.search(r"sw[kq]::(\w+)", name).group(1) in launched, name
