"""The e4m3 product by the type of its results: which form 16-bit results take (the plan
weighs the store, which their type changes), results of each against float64, and what the
order of the sums depends on: a call with 16-bit results gives the fp32 call's rounded where
both take K in the same parts, and is one of its own where they do not."""
import ctypes

import pytest
import torch

from test_linear_f8_gpu import Problem
from test_linear_f8_plans import SMS, _built, _ids

BF16, FP16, FP32 = 0, 1, 2
FORMS = {  # channels per tile, CTAs that work on it: sizes, N, K
    (256, 2): [((3000,), 800, 1000), ((8192,), 1000, 1000), ((700, 0, 1157, 900, 1), 2000, 500)],
    (128, 2): [((256,), 1024, 1792), ((60,), 4096, 700), ((60, 2, 90), 1032, 1100),
               ((130, 126, 0, 256), 2000, 2600)],
    (64, 2): [((129,), 1500, 700), ((129,), 1501, 700), ((100, 140), 700, 600)],
    (128, 4): [((64,), 4096, 4096), ((512,), 2304, 7168), ((130,), 2328, 2591)],
    (64, 4): [((300,), 1000, 2000), ((197,), 1001, 1992), ((500,), 264, 2008)],
    (256, 1): [((130, 126, 0, 256) * 4, 1032, 1100), ((5, 0, 1, 40) * 15, 1500, 700),
               ((1,) * 200, 700, 2000)],
    (0, 0): [((1,), 4096, 7168), ((16,), 7168, 512), ((6,) * 40, 512, 512)],
}
CASES = [s for some in FORMS.values() for s in some]
# 16-bit and fp32 results whose K is taken in different parts
DIFFER = [((256,), 1024, 1792)]


def _plan(lib, sizes, N, K, dtype):
    i32 = ctypes.c_int32
    fn = lib.moe_test_linear_f8_plan_of
    fn.argtypes = [ctypes.c_int64, i32, i32, i32, i32, i32, ctypes.c_void_p]
    fn.restype = None
    plan = (i32 * 3)()
    fn(sum(sizes), len(sizes), N, K, dtype, SMS, plan)
    assert plan[1] * plan[2] <= SMS
    return plan[0], plan[2]


def test_forms_of_16_bit_results():
    lib = ctypes.CDLL(_built())
    for form, shapes in FORMS.items():
        for shape in shapes:
            for dtype in (BF16, FP16):
                assert _plan(lib, *shape, dtype) == form, shape
            parts = form[1] == 4
            differs = (_plan(lib, *shape, FP32)[1] == 4) != parts
            assert differs == (shape in DIFFER), shape


@pytest.fixture(scope="module")
def ep():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a CUDA device")
    import combine_moe_dispatch_layout_gb300 as ep
    return ep


@pytest.mark.gpu
@pytest.mark.parametrize("sizes,N,K", CASES, ids=_ids)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_results_of_16_bits(ep, sizes, N, K, dtype):
    p, wide = (Problem(ep, list(sizes), N, K, d, bias=True, images=N % 3 != 1)
               for d in (dtype, torch.float32))
    for q in (p, wide):
        q.run()
        q.check()
    if (sizes, N, K) not in DIFFER:
        assert torch.equal(p.c, wide.c.to(dtype))
