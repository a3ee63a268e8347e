"""The INT8 product's kernel hands its launch registers out again by role; the
shares must fit what a launch has (a larger sum would wait forever), so every
instantiation has to be compiled to the count the split was worked out for."""
import os
import re
import shutil

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PKG = os.path.join(ROOT, "combine_moe_dispatch_layout_gb300")


def _constant(text, name):
    return int(re.search(r"\b%s = (\d+)" % name, text).group(1))


def test_linear_i8_registers_cover_the_split():
    if shutil.which("nvcc") is None and not os.path.exists("/usr/local/cuda/bin/nvcc"):
        pytest.skip("nvcc not available")
    import __graft_entry__
    __graft_entry__._load_builder().build()
    src = open(os.path.join(PKG, "csrc", "linear_i8.cu")).read()
    warps = [(_constant(src, "kEpiWarps"), _constant(src, "kEpiRegs")),
             (_constant(src, "kConvWarps"), _constant(src, "kConvRegs")),
             (4, _constant(src, "kCtrlRegs"))]
    threads = 32 * sum(w for w, _ in warps)
    split = 32 * sum(w * r for w, r in warps)
    report = open(os.path.join(PKG, "_build", "linear_i8.ptxas.txt")).read()
    used = [int(m) for m in re.findall(r"linear_i8_tile_kernel.*?Used (\d+) registers", report,
                                       re.S)]
    assert len(used) == 16                  # two widths, four outputs, split or not
    for regs in used:
        assert regs % 8 == 0 and split <= threads * regs <= 65536, (regs, split, threads)
