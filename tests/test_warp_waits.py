"""A whole warp's wait for a barrier's phase passes once every lane has seen it: whichever
lane then issues copies or products, or reads, has acquired what the phase stands for."""
import os
import re

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "combine_moe_dispatch_layout_gb300", "csrc")


@pytest.mark.parametrize("unit,waits", [
    ("tcgen05.cuh", ["warp_bar_wait", "warp_bar_wait4"]),
    ("linear_f8_polls.cu", ["warp_role_wait"])])
def test_every_lane_sees_the_phase(unit, waits):
    text = re.sub(r"//[^\n]*", "", open(os.path.join(CSRC, unit)).read())
    for name in waits:
        body = text[text.index("bool %s(" % name):]
        body = body[:body.index("\n}\n")]
        assert len(re.findall(r"if \(__all_sync\(0xffffffffu, [^;]*\)\) return true;",
                              body)) == 1, name
        assert "__any_sync" not in body and "__ballot" not in body, name
