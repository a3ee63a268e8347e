"""The norm with the residual's addition and its 8-bit row images, and its gradient,
against float64.  Bounds: a row's sum of squares is a chain of at most 64 fused additions a
thread and 37 more over the threads, so rstd is within 51 roundings of 2^-24 and y within
54; what is asked of y is 64, of a gradient's sums 128."""
import numpy as np
import pytest
import torch

import plain_f8 as P

pytestmark = pytest.mark.gpu
EPS = 1e-6
REL = 64 * P.U32


@pytest.fixture(scope="module")
def ep():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a CUDA device")
    import combine_moe_dispatch_layout_gb300 as ep
    return ep


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _rows(T, H, dtype, g, scale=1.0):
    return (torch.randn((T, H), generator=g, device="cuda") * scale).to(dtype)


def _status():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


class Guarded:
    """[T, H] rows inside a wider, taller buffer of 0xA5 bytes, `gap` elements apart."""

    def __init__(self, T, H, dtype, gap=0):
        pitch = H + gap
        self.raw = torch.empty((T + 2, pitch), dtype=dtype, device="cuda")
        self.raw.view(torch.uint8).fill_(0xA5)
        self.t = self.raw[1:T + 1, :H]

    def check(self):
        H = self.t.shape[1]
        edge = [self.raw[0], self.raw[-1], self.raw[:, H:].contiguous()]
        for e in edge:
            assert bool((e.contiguous().view(torch.uint8) == 0xA5).all())


# every row width that a kernel is chosen by, its neighbours, odd last blocks
WIDTHS = [8, 16, 128, 136, 504, 512, 520, 1000, 1024, 1032, 2048, 2056, 4096, 4104, 7168, 8192,
          8200, 16384, 16392, 20000]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("H", WIDTHS)
@pytest.mark.parametrize("T", [1, 3, 300])
def test_forward(ep, T, H, dtype):
    g = _gen(T + H)
    gap = 8 * (H % 3)
    x, res = Guarded(T, H, dtype, gap), Guarded(T, H, dtype, 16)
    x.t.copy_(_rows(T, H, dtype, g, 3.0))
    res.t.copy_(_rows(T, H, dtype, g))
    gamma = 1 + 0.3 * torch.randn(H, generator=g, device="cuda")
    for residual, code in ((res, "f8"), (None, "f8"), (res, "i8"), (None, None)):
        s_out, out = Guarded(T, H, dtype, 8), Guarded(T, H, dtype, gap)
        rstd = torch.full((T,), -1.0, device="cuda")
        size = ep.f8_row_bytes(H) if code == "f8" else P.align32(H) + 32
        image = Guarded(T, size, torch.uint8) if code else None
        st = _status()
        ep.moe_rms_norm(x.t, residual.t if residual else None, gamma, EPS,
                        s_out.t if residual else None, out.t, image.t if image else None, rstd,
                        st, code=code or "f8")
        torch.cuda.synchronize()
        assert int(st.item()) == 0
        s, r, y = P.norm(x.t, residual.t if residual else None, gamma, EPS)
        for b in (x, res, s_out, out) + ((image,) if image else ()):
            b.check()
        if residual:
            assert torch.equal(s_out.t.double(), s)
        np.testing.assert_allclose(rstd.double().cpu(), r[:, 0].cpu(), rtol=REL)
        tol = (P.HALF[dtype] + REL) * y.abs() + torch.finfo(dtype).tiny * 2.0 ** -10
        assert bool(((out.t.double() - y).abs() <= tol).all())
        if code == "f8":
            P.check_image(image.t, y.cpu().numpy(), REL)
        if code == "i8":
            raw = image.t.cpu().numpy()
            codes = raw[:, :H].view(np.int8).astype(np.float64)
            at = P.align32(H)
            inv = raw[:, at:at + 4].copy().view(np.float32).astype(np.float64)[:, 0]
            assert not raw[:, H:at].any() and not raw[:, at + 4:].any()
            yy = y.cpu().numpy()
            q = 127.0 / (np.abs(yy).max(axis=1) + 1e-12)
            np.testing.assert_allclose(inv, 1 / q, rtol=REL + 4 * P.U32)
            assert (np.abs(codes - yy * q[:, None]) <= 0.5 + 127 * (2 * REL + 8 * P.U32)).all()


def test_in_place(ep):
    """The sum over the residual, the norm over the input."""
    g = _gen(5)
    for T, H in ((5, 1000), (300, 7168), (3, 20000)):
        x, res = _rows(T, H, torch.bfloat16, g), _rows(T, H, torch.bfloat16, g)
        gamma = torch.rand(H, generator=g, device="cuda")
        want = [torch.empty_like(x) for _ in range(2)]
        ep.moe_rms_norm(x, res, gamma, EPS, want[0], want[1], None, None, _status())
        a, b = x.clone(), res.clone()
        ep.moe_rms_norm(a, b, gamma, EPS, b, a, None, None, _status())
        assert torch.equal(b, want[0]) and torch.equal(a, want[1])
        a, b = x.clone(), res.clone()
        ep.moe_rms_norm(a, b, gamma, EPS, a, b, None, None, _status())
        assert torch.equal(a, want[0]) and torch.equal(b, want[1])


@pytest.mark.parametrize("H", [128, 1000, 7168, 16392])
def test_rows_that_say_nothing(ep, H):
    """Zeros, one value alone, subnormal rows, and rows with an infinity or a NaN, which
    stay in their row."""
    T = 8
    g = _gen(H)
    x = _rows(T, H, torch.float16, g)
    x[0] = 0
    x[1] = 0
    x[1, H // 2] = 2.0
    x[2] = 2.0 ** -24
    x[4, 3] = float("inf")
    x[6, H - 1] = float("nan")
    gamma = torch.ones(H, device="cuda")
    out = torch.empty_like(x)
    image = torch.empty((T, ep.f8_row_bytes(H)), dtype=torch.uint8, device="cuda")
    ep.moe_rms_norm(x, None, gamma, EPS, None, out, image, None, _status())
    _, _, y = P.norm(x, None, gamma, EPS)
    fine = [0, 1, 2, 3, 5, 7]
    tol = (P.HALF[torch.float16] + REL) * y[fine].abs() + 2.0 ** -25
    assert bool(((out[fine].double() - y[fine]).abs() <= tol).all())
    P.check_image(image[fine], y[fine].cpu().numpy(), REL)
    assert bool((image[0, :H] == 0).all())
    assert bool(out[6].isnan().all()) and bool(out[4, 3].isnan()) and bool((out[4, 4:] == 0).all())
    codes, scales, _ = P.split_image(image[6:7], H)
    assert np.isnan(codes).all() and np.isnan(scales).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("H", WIDTHS)
@pytest.mark.parametrize("T", [1, 2, 37, 1300])
def test_backward(ep, T, H, dtype):
    if T * H > 1 << 23:
        T = (1 << 23) // H
    g = _gen(T * 7 + H)
    x, dy, ds = (Guarded(T, H, dtype, gap) for gap in (8, 0, 24))
    x.t.copy_(_rows(T, H, dtype, g, 2.0))
    dy.t.copy_(_rows(T, H, dtype, g))
    ds.t.copy_(_rows(T, H, dtype, g))
    gamma = 1 + 0.3 * torch.randn(H, generator=g, device="cuda")
    _, r, _ = P.norm(x.t, None, gamma, EPS)
    rstd = r[:, 0].float()
    size = ep.rms_norm_backward_workspace_bytes(T, H)
    for d_sum in (ds, None):
        dx = Guarded(T, H, dtype, 16)
        raw = torch.full((H + 128,), -7.0, device="cuda")
        ws = torch.full((size + 512,), 0xA5, dtype=torch.uint8, device="cuda")
        ws[:size].fill_(0xFF)                       # NaN: nothing of it may count
        st = _status()
        ep.moe_rms_norm_backward(dy.t, x.t, gamma, rstd, d_sum.t if d_sum else None, dx.t,
                                 raw[64:64 + H], ws[:size], st)
        torch.cuda.synchronize()
        assert int(st.item()) == 0 and bool((ws[size:] == 0xA5).all())
        assert bool((raw[:64] == -7).all()) and bool((raw[64 + H:] == -7).all())
        for b in (x, dy, ds, dx):
            b.check()
        want, want_gamma = P.norm_backward(dy.t, x.t, gamma, EPS, d_sum.t if d_sum else None)
        xh, a = (x.t.double() * r), (dy.t.double() * gamma.double())
        mag = r * (a.abs() + xh.abs() * (a * xh).abs().mean(1, keepdim=True))
        tol = (P.HALF[dtype] * (1 + 2.0 ** -6) * want.abs() + 128 * P.U32 * mag
               + torch.finfo(dtype).tiny * 2.0 ** -10)
        assert bool(((dx.t.double() - want).abs() <= tol).all())
        gm = (dy.t.double() * xh).abs().sum(0)
        assert bool(((raw[64:64 + H].double() - want_gamma).abs() <= 128 * P.U32 * gm).all())


def test_backward_is_the_difference_quotient(ep):
    """Of <c, norm(x)> by float64 differences of the definition."""
    T, H = 3, 64
    g = _gen(1)
    x, c = _rows(T, H, torch.float16, g), _rows(T, H, torch.float16, g)
    gamma = torch.rand(H, generator=g, device="cuda") + 0.5
    _, r, _ = P.norm(x, None, gamma, EPS)
    dx, dg = torch.empty_like(x), torch.empty(H, device="cuda")
    ws = torch.empty(ep.rms_norm_backward_workspace_bytes(T, H), dtype=torch.uint8, device="cuda")
    ep.moe_rms_norm_backward(c, x, gamma, r[:, 0].float(), None, dx, dg, ws, _status())

    def loss(xs, gs):
        rr = (xs.pow(2).mean(1, keepdim=True) + EPS) ** -0.5
        return (c.double() * xs * rr * gs).sum(1)

    h = 1e-5
    for j in range(H):
        e = torch.zeros(H, dtype=torch.float64, device="cuda")
        e[j] = h
        d = (loss(x.double() + e, gamma.double()) - loss(x.double() - e, gamma.double())) / (2 * h)
        # a difference of step h is off by h^2 times third derivatives of order 10
        assert bool(((dx[:, j].double() - d).abs() <= 2.0 ** -10 * d.abs() + 1e-6).all())
        d = (loss(x.double(), gamma.double() + e) - loss(x.double(), gamma.double() - e)) / (2 * h)
        assert abs(float(dg[j]) - float(d.sum())) <= 1e-5


def test_backward_in_place_and_repeatable(ep):
    """d_x over any of its inputs; the same bits on every call."""
    g = _gen(9)
    for T, H in ((2000, 1000), (700, 7168), (40, 20000)):
        x, dy, ds = (_rows(T, H, torch.bfloat16, g) for _ in range(3))
        gamma = torch.rand(H, generator=g, device="cuda")
        _, r, _ = P.norm(x, None, gamma, EPS)
        rstd = r[:, 0].float()
        ws = torch.empty(ep.rms_norm_backward_workspace_bytes(T, H), dtype=torch.uint8,
                         device="cuda")

        def run(which):
            t = [dy.clone(), x.clone(), ds.clone(), torch.empty_like(x)]
            dg = torch.empty(H, device="cuda")
            ep.moe_rms_norm_backward(t[0], t[1], gamma, rstd, t[2], t[which], dg, ws, _status())
            return t[which], dg

        want = run(3)
        for which in (3, 0, 1, 2):
            got = run(which)
            assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]), which


def test_no_rows(ep):
    H = 64
    x = torch.empty((0, H), dtype=torch.bfloat16, device="cuda")
    gamma = torch.ones(H, device="cuda")
    assert ep.moe_rms_norm(x, None, gamma, EPS, None, x, None, None, _status()) == 0
    dg = torch.full((H,), 3.0, device="cuda")
    ws = torch.empty(ep.rms_norm_backward_workspace_bytes(0, H), dtype=torch.uint8, device="cuda")
    ep.moe_rms_norm_backward(x, x, gamma, torch.empty(0, device="cuda"), None, x, dg, ws,
                             _status())
    assert bool((dg == 0).all())


def test_far_rows(ep):
    """Rows whose offsets pass 2^32 bytes and 2^31 elements."""
    T, H, pitch = 3, 64, (1 << 30) + 64
    raw = torch.zeros((2 * pitch + H,), dtype=torch.float16, device="cuda")
    x = raw.as_strided((T, H), (pitch, 1))
    x.copy_(_rows(T, H, torch.float16, _gen(2)))
    gamma = torch.ones(H, device="cuda")
    out = torch.empty((T, H), dtype=torch.float16, device="cuda")
    ep.moe_rms_norm(x, None, gamma, EPS, None, out, None, None, _status())
    _, _, y = P.norm(x, None, gamma, EPS)
    assert bool(((out.double() - y).abs() <= (2.0 ** -11 + REL) * y.abs() + 1e-7).all())
