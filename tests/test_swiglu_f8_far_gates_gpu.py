"""SwiGLU to e4m3 row images where the gate is far below 0: h within its bound as long as
1 + exp(-gate) is at most 2^126 (gate above -126 ln 2 = -87.3365), and 0 where it is more."""
import numpy as np
import pytest
import torch

import plain_f8 as P

pytestmark = pytest.mark.gpu
LAST = -126 * float(np.log(2.0))
# the exponential is within 2^-17 of itself there, which moves the border by as much
NEAR = 2.0 ** -16


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("I", [128, 384, 1024])
def test_gates_about_the_last_one(dtype, I):
    """With `up` so large that none of the results is lost in the codes."""
    import combine_moe_dispatch_layout_gb300 as ep
    gate = torch.linspace(-86.0, -89.0, I, device="cuda").flip(0)
    gate[:8] = torch.tensor([-87.0, -87.25, -87.3, -87.33, -87.34, -87.35, -87.5, -88.0])
    gate[8:16] = -86.0                     # (one of each block sets its scale)
    gate[15::64] = -86.5
    up = torch.full((I,), 1e38, device="cuda")
    h = torch.stack([torch.cat([gate, up]), torch.cat([gate, -up])]).to(dtype)
    image = torch.empty((2, ep.f8_row_bytes(I)), dtype=torch.uint8, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    ep.moe_swiglu_f8(h, None, image, st)
    assert int(st.item()) == 0
    gates = h[0, :I].double().cpu()
    assert bool(((gates - LAST).abs() > NEAR).all())
    live = (gates > LAST)
    assert 16 < int(live.sum()) < I - 16
    want = P.swiglu(h).cpu() * live
    P.check_image(image, want.numpy(), 2.0 ** -16)
    codes, _, _ = P.split_image(image, I)
    assert not codes[:, ~live.numpy()].any()
    assert codes[:, live.numpy()].all()
