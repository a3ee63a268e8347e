"""The INT8 product of few rows reads the bytes of a's rows up to K and none behind
them (the last row may end its buffer there)."""
import os
import re

import numpy as np
import pytest
import torch

import plain_ops as P

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SOURCE = os.path.join(ROOT, "combine_moe_dispatch_layout_gb300", "csrc", "linear_i8_few.cu")


def test_a_piece_that_reaches_past_k_is_read_by_its_bytes():
    """Every 16-byte load of a token's codes stands under j + 16 <= K."""
    text = re.sub(r"//[^\n]*", "", open(SOURCE).read())
    loads = [m.start() for m in re.finditer(r"const uint4\*>\(at\)", text)]
    assert loads
    for at in loads:
        assert re.search(r"j \+ 16 <= K \?\s*\*reinterpret_cast<$", text[:at]), text[at - 80:at]


@pytest.mark.gpu
@pytest.mark.parametrize("rows,N", [(1, 40), (3, 700), (8, 130)])
def test_rows_that_end_their_buffer(rows, N):
    import combine_moe_dispatch_layout_gb300 as ep
    rng = np.random.default_rng(rows)
    for K in list(range(1, 36)) + [511, 513, 1000, 1992, 2047]:
        wide = (K + 15) // 16 * 16
        a = rng.integers(-128, 128, (rows, K)).astype(np.int8)
        w = rng.integers(-128, 128, (1, N, wide)).astype(np.int8)       # garbage past K
        buf = torch.full(((rows - 1) * wide + K,), 77, dtype=torch.int8, device="cuda")
        view = torch.as_strided(buf, (rows, K), (wide, 1))
        view.copy_(torch.from_numpy(a))
        c = torch.zeros((rows, N), dtype=torch.int32, device="cuda")
        st = torch.zeros(1, dtype=torch.int32, device="cuda")
        ep.moe_linear_i8(view, torch.from_numpy(w).cuda(), K, None, None, None, None, c, st)
        assert int(st.item()) == 0
        assert np.array_equal(c.cpu().numpy(), P.linear_i8(a, w[:, :, :K], [rows]))
