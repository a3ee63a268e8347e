"""The e4m3 product's tile kernel in every form it takes.  On the CPU: that the shapes below
take those forms, and that the registers its roles ask for are the launch's.  On the GPU:
results of each form, and calls whose waits run out at once or here and there, which must
end, report MOE_ERR_TIMEOUT, write nothing outside c and no value inside that is not the
normal call's, and leave the GPU as a normal call right behind them needs it.  Short
waits come from the test entry point moe_test_linear_f8_polls; the closing waits keep their
bound."""
import ctypes
import os
import re
import shutil

import pytest
import torch

import plain_f8 as P

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PKG = os.path.join(ROOT, "combine_moe_dispatch_layout_gb300")
SMS = 152
PLANS = {  # channels per tile, CTAs that work on it: sizes, N, K
    (256, 2): [((3000,), 800, 1000), ((8192,), 1000, 1000), ((700, 0, 1157, 900, 1), 2000, 500),
               ((100, 900, 0, 1200, 300, 1, 900, 999), 1275, 1100)],
    (128, 2): [((24576,), 72, 700), ((5000,), 1000, 1300), ((12,), 8200, 4100),
               ((130, 126, 0, 256), 2000, 2600), ((60, 2, 900), 4000, 3000)],
    (64, 2): [((300,), 1000, 1025), ((129,), 1501, 700), ((60, 2, 90), 1032, 1100)],
    (128, 4): [((40,), 4096, 3500), ((700,), 1001, 3073), ((256,), 4601, 7168)],
    (64, 4): [((300,), 1000, 2000), ((197,), 1001, 1992), ((256,), 72, 16384)],
    (256, 1): [((130, 126, 0, 256) * 4, 1032, 1100), ((5, 0, 1, 40) * 15, 1500, 700),
               ((100, 900, 0, 1200, 300, 1, 400, 99) * 4, 1275, 1100), ((1,) * 200, 700, 2000)],
    (0, 0): [((1,), 4096, 7168), ((8,), 8200, 4100), ((16,), 7168, 512), ((6,) * 40, 512, 512),
             ((256,), 512, 1024), ((3,) * 8, 4000, 4000)],
}
TILES = [s for form, some in PLANS.items() if form[0] for s in some]


def _ids(v):
    return str(v).replace(" ", "")[:32]


def _built():
    if shutil.which("nvcc") is None and not os.path.exists("/usr/local/cuda/bin/nvcc"):
        pytest.skip("nvcc not available")
    import __graft_entry__
    return __graft_entry__._load_builder().build()


def test_the_shapes_take_every_form():
    fn = ctypes.CDLL(_built()).moe_test_linear_f8_plan
    i32 = ctypes.c_int32
    fn.argtypes = [ctypes.c_int64, i32, i32, i32, i32, ctypes.c_void_p]
    fn.restype = None
    for form, shapes in PLANS.items():
        for sizes, N, K in shapes:
            plan = (i32 * 3)()
            fn(sum(sizes), len(sizes), N, K, SMS, plan)
            assert (plan[0], plan[2]) == form, (sizes, N, K, tuple(plan))
            assert plan[1] * plan[2] <= SMS


def test_registers_cover_the_split():
    """A role's larger share of registers waits forever where the shares' sum is above the
    launch's."""
    _built()
    src = open(os.path.join(PKG, "csrc", "linear_f8.cu")).read()

    def constant(name):
        return int(re.search(r"\b%s = (\d+)" % name, src).group(1))

    epi, ctrl = constant("kEpiWarps"), constant("kCtrlWarps")
    threads = 32 * (epi + ctrl)
    split = 32 * (epi * constant("kEpiRegs") + ctrl * constant("kCtrlRegs"))
    for unit, kernels in (("linear_f8", 18), ("linear_f8_polls", 6)):
        report = open(os.path.join(PKG, "_build", unit + ".ptxas.txt")).read()
        used = [int(m) for m in re.findall(r"linear_f8_tile_kernel.*?Used (\d+) registers", report,
                                           re.S)]
        assert len(used) == kernels
        for regs in used:
            assert regs % 8 == 0 and split <= threads * regs <= 65536, (regs, split, threads)


@pytest.fixture(scope="module")
def ep():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a CUDA device")
    import combine_moe_dispatch_layout_gb300 as ep
    vp, i32, i64 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64
    fn = ep.lib().moe_test_linear_f8_polls
    fn.argtypes = [vp, i64, i64, vp, i64, i32, i32, i32, vp, vp, vp, i64, vp,
                   ctypes.c_uint32, vp, vp]
    fn.restype = ctypes.c_int
    return ep


class Problem:
    def __init__(self, ep, sizes, N, K):
        g = torch.Generator(device="cuda")
        g.manual_seed(sum(sizes) + N)
        self.ep, self.sizes, self.N, self.K = ep, sizes, N, K
        rows, G, wide = sum(sizes), len(sizes), (K + 15) // 16 * 16
        kb = P.blocks(K)

        def codes(*shape):
            v = torch.randn(shape, generator=g, device="cuda") * 90
            return v.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)

        self.a, self.w = codes(rows, wide), codes(G, N, wide)
        self.scale = torch.exp2(torch.randn((rows, kb), generator=g, device="cuda"))
        self.w_scale = torch.exp2(torch.randn((G, P.blocks(N), kb), generator=g,
                                              device="cuda")) * 1e-5
        self.counts = torch.tensor(sizes, dtype=torch.int32, device="cuda")
        self.raw = torch.full((rows * N + 128,), -7.0, device="cuda")
        self.c = self.raw[64:64 + rows * N].view(rows, N)
        self.st = torch.zeros(1, dtype=torch.int32, device="cuda")

    def run(self):
        self.st.zero_()
        grouped = self.counts if len(self.sizes) > 1 else None
        self.ep.moe_linear_f8(self.a, self.w, self.K, grouped, self.w_scale,
                              (self.scale, 0, 4 * self.scale.shape[1]), None, self.c, self.st)
        torch.cuda.synchronize()
        assert int(self.st.item()) == 0
        return self.c.clone()

    def check(self):
        got = self.run().double().cpu()
        want, mag = P.linear(self.a, self.scale, self.w, self.w_scale, self.K, self.sizes)
        assert bool(((got - want).abs() <= P.linear_bound(want, mag, self.K,
                                                          torch.float32)).all())

    def hook(self, polls):
        a, w, s = self.a, self.w, self.scale
        return self.ep.lib().moe_test_linear_f8_polls(
            a.data_ptr(), a.shape[0], a.shape[1], w.data_ptr(), w.shape[2], len(self.sizes),
            self.N, self.K, self.counts.data_ptr(), self.w_scale.data_ptr(), s.data_ptr(),
            4 * s.shape[1], self.c.data_ptr(), polls, self.st.data_ptr(),
            torch.cuda.current_stream().cuda_stream)


@pytest.mark.gpu
@pytest.mark.parametrize("sizes,N,K", TILES, ids=_ids)
def test_every_form(ep, sizes, N, K):
    Problem(ep, sizes, N, K).check()


@pytest.mark.gpu
@pytest.mark.parametrize("sizes,N,K", TILES, ids=_ids)
@pytest.mark.parametrize("polls", [1, 3, 30, 300, 3000])
def test_waits_that_run_out(ep, sizes, N, K, polls):
    p = Problem(ep, sizes, N, K)
    want = p.run()
    ended = 0
    for _ in range(3):
        p.raw.fill_(-7.0)
        p.st.zero_()
        assert p.hook(polls) == 0
        torch.cuda.synchronize()
        status = int(p.st.item())
        assert status in (0, ep.MOE_ERR_TIMEOUT)
        ended += status != 0
        assert bool((p.raw[:64] == -7).all()) and bool((p.raw[-64:] == -7).all())
        left = p.c == -7.0
        assert torch.equal(p.c[~left], want[~left])
        if status == 0:
            assert torch.equal(p.c, want)
        assert torch.equal(p.run(), want)       # the next call finds nothing in its way
    if polls == 1:
        assert ended == 3
