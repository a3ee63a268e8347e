"""The INT8 product's tile kernel in every form it takes: both tile widths, K whole and
split over clusters of two, three and four pairs, one group and several.  On the CPU:
that the shapes below take those forms.  On the GPU: exact sums, and calls whose
waits run out at once or here and there, which must end, report MOE_ERR_TIMEOUT, write
nothing outside c (and, where K is whole, no value inside that is not the exact one),
and leave the GPU as a normal call right behind them needs it.  Short waits come from
the test entry point moe_test_linear_i8_polls; the closing waits keep their bound.
The roles' barriers, step by step, are modelled in tests/test_linear_i8_pair_model.py."""
import ctypes
import os
import shutil

import numpy as np
import pytest
import torch

SMS = 152
PLANS = {  # (tokens per tile, pairs per K): sizes, N, K
    (256, 1): [((24576,), 40, 4096), ((3000,), 1000, 200),
               ((100, 900, 0, 1200, 300, 1, 400, 99), 520, 1100)],
    (256, 2): [((512,), 3300, 2048), ((400, 500, 600), 1000, 2000)],
    (256, 3): [((600,), 1500, 3000), ((0, 600, 250, 50), 700, 4000)],
    (256, 4): [((600,), 1000, 4096), ((200, 300, 0, 400), 300, 4000)],
    (128, 1): [((100,), 10000, 600), ((15,) * 20, 1000, 600)],
    (128, 2): [((64,), 7168, 2048)],
    (128, 3): [((100,), 4096, 3000), ((150, 0, 100, 50), 700, 4000)],
    (128, 4): [((100,), 1001, 2000), ((30,), 3000, 4096)],
}
SHAPES = [s for some in PLANS.values() for s in some]


def _ids(v):
    return str(v).replace(" ", "")[:32]


def test_the_shapes_take_every_form():
    if shutil.which("nvcc") is None and not os.path.exists("/usr/local/cuda/bin/nvcc"):
        pytest.skip("nvcc not available")
    import __graft_entry__
    fn = ctypes.CDLL(__graft_entry__._load_builder().build()).moe_test_linear_i8_plan
    i32 = ctypes.c_int32
    fn.argtypes = [ctypes.c_int64, i32, i32, i32, i32, ctypes.c_void_p]
    fn.restype = None
    for form, shapes in PLANS.items():
        for sizes, N, K in shapes:
            plan = (i32 * 3)()
            fn(sum(sizes), len(sizes), N, K, SMS, plan)
            assert tuple(plan[:2]) == form, (sizes, N, K, tuple(plan))
            assert 2 * plan[1] * plan[2] <= SMS


@pytest.fixture(scope="module")
def ep():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a CUDA device")
    import combine_moe_dispatch_layout_gb300 as ep
    vp, i32, i64 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64
    fn = ep.lib().moe_test_linear_i8_polls
    fn.argtypes = [vp, i64, i64, vp, i64, i32, i32, i32, vp, vp, ctypes.c_uint32, vp, vp]
    fn.restype = ctypes.c_int
    return ep


class Case:
    def __init__(self, sizes, N, K, seed):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        wide = (K + 15) // 16 * 16
        self.rows, self.N, self.K = sum(sizes), N, K
        self.a = torch.randint(-128, 128, (self.rows, wide), generator=g, dtype=torch.int8,
                               device="cuda")
        self.w = torch.randint(-128, 128, (len(sizes), N, wide), generator=g, dtype=torch.int8,
                               device="cuda")
        self.sizes = torch.tensor(sizes, dtype=torch.int32, device="cuda")
        self.raw = torch.zeros(self.rows * N + 128, dtype=torch.int32, device="cuda")
        self.c = self.raw[64:64 + self.rows * N].view(self.rows, N)
        self.st = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.want = torch.empty((self.rows, N), dtype=torch.int32, device="cuda")
        at = 0
        for e, n in enumerate(sizes):          # exact in float64
            self.want[at:at + n] = torch.round(
                self.a[at:at + n, :K].double() @ self.w[e, :, :K].double().t()).int()
            at += n

    SENTINEL = -0x5A5A5A5B

    def reset(self):
        self.raw.fill_(self.SENTINEL)
        self.st.zero_()

    def check_margins(self):
        assert (self.raw[:64] == self.SENTINEL).all() and (self.raw[-64:] == self.SENTINEL).all()

    def call(self, ep):
        ep.moe_linear_i8(self.a, self.w, self.K, self.sizes, None, None, None, self.c, self.st)

    def polls(self, ep, n):
        rc = ep.lib().moe_test_linear_i8_polls(
            self.a.data_ptr(), self.rows, self.a.shape[1], self.w.data_ptr(), self.w.shape[2],
            self.w.shape[0], self.N, self.K, self.sizes.data_ptr(), self.c.data_ptr(), n,
            self.st.data_ptr(), torch.cuda.current_stream().cuda_stream)
        assert rc == 0, ep.status_string(rc)


@pytest.mark.gpu
@pytest.mark.parametrize("sizes,N,K", SHAPES, ids=_ids)
def test_exact_sums(ep, sizes, N, K):
    c = Case(sizes, N, K, seed=N + K)
    for _ in range(5):
        c.reset()
        c.call(ep)
        assert torch.equal(c.c, c.want)
    assert int(c.st.item()) == 0
    c.check_margins()


@pytest.mark.gpu
@pytest.mark.parametrize("form", PLANS, ids=str)
def test_waits_that_run_out_then_a_normal_call(ep, form):
    sizes, N, K = PLANS[form][0]
    c = Case(sizes, N, K, seed=sum(form))
    gave_up = 0
    for polls in (1, 8, 40, 200, 1000, 1 << 20):
        c.reset()
        c.polls(ep, polls)
        torch.cuda.synchronize()
        status = int(c.st.item())
        assert status in (0, ep.MOE_ERR_TIMEOUT)
        c.check_margins()
        if status == 0:
            assert torch.equal(c.c, c.want)
        else:
            gave_up += 1
            if form[1] == 1:
                written = c.c != c.SENTINEL
                assert torch.equal(c.c[written], c.want[written])
        if polls == 1:
            assert status == ep.MOE_ERR_TIMEOUT     # operands take longer than one look
        if polls == 1 << 20:
            assert status == 0
        c.reset()
        c.call(ep)
        assert torch.equal(c.c, c.want) and int(c.st.item()) == 0
        c.check_margins()
    assert gave_up > 0
