"""Checks of the device code that no run shows: special registers that inline assembly
overwrites, in the sources and in the code the compiler makes of them."""
import os
import re
import subprocess

from swiglu_gated_mlp_amd import build

ASM = re.compile(r"asm volatile\((.*?)\);", re.S)
M0 = re.compile(r"\bm0\b")


def test_assembly_that_writes_m0_says_so():
    found = 0
    for name in sorted(os.listdir(build.CSRC)):
        with open(os.path.join(build.CSRC, name)) as f:
            for body in ASM.findall(f.read()):
                if "s_mov_b32 m0" in body:
                    found += 1
                    assert re.search(r':\s*"m0"', body), "%s: %s" % (name, body)
    assert found > 0


def test_nothing_else_uses_m0_beside_the_untracked_loads(tmp_path):
    """The loads' own two lines are the only ones of the training kernels with m0."""
    out = str(tmp_path / "train.s")
    cmd = [build.hipcc(), *build.compile_flags(), "-x", "hip", "-S", "--offload-device-only",
           os.path.join(build.CSRC, "train_api.hip"), "-o", out]
    subprocess.run(cmd, check=True, stdout=subprocess.DEVNULL, stderr=subprocess.DEVNULL)
    loads = 0
    with open(out) as f:
        lines = [x.strip() for x in f]
    for i, x in enumerate(lines):
        x = x.split(";")[0]
        if M0.search(x):
            assert re.fullmatch(r"s_mov_b32 m0, s\d+\s*", x), x
            assert lines[i - 1] == ";;#ASMSTART" and lines[i + 1] == "s_nop 0", lines[i - 2:i + 3]
            assert lines[i + 2].startswith("buffer_load_dwordx4 ") and lines[i + 2].endswith(" offen lds")
            loads += 1
        elif x.startswith("buffer_load") and x.endswith(" lds"):
            assert lines[i - 2].startswith("s_mov_b32 m0")
    assert loads > 0
