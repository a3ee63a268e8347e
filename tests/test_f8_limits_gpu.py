"""The norm, its gradient, SwiGLU to e4m3 rows and the e4m3 product at the largest sizes that
are documented: rows of 65,536 values, 65,536 channels, 4096 groups, and rows and results
past 32-bit offsets."""
import pytest
import torch

import plain_f8 as P
from test_linear_f8_gpu import Problem

pytestmark = pytest.mark.gpu
EPS = 1e-6
# a thread of the widest rows adds 8 chunks of 8 squares, 37 more follow: as the other widths
REL = 64 * P.U32


@pytest.fixture(scope="module")
def ep():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a CUDA device")
    import combine_moe_dispatch_layout_gb300 as ep
    return ep


def _status():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("T", [1, 9])
def test_the_widest_rows(ep, T):
    H = 65536
    g = torch.Generator(device="cuda")
    g.manual_seed(T)
    x, res, dy = (torch.randn((T, H), generator=g, device="cuda").bfloat16() for _ in range(3))
    gamma = 1 + 0.3 * torch.randn(H, generator=g, device="cuda")
    s, out, dx = (torch.empty_like(x) for _ in range(3))
    image = torch.empty((T, ep.f8_row_bytes(H)), dtype=torch.uint8, device="cuda")
    rstd, dg, st = torch.empty(T, device="cuda"), torch.empty(H, device="cuda"), _status()
    ep.moe_rms_norm(x, res, gamma, EPS, s, out, image, rstd, st)
    ws = torch.empty(ep.rms_norm_backward_workspace_bytes(T, H), dtype=torch.uint8, device="cuda")
    ep.moe_rms_norm_backward(dy, s, gamma, rstd, res, dx, dg, ws, st)
    assert int(st.item()) == 0
    want, r, y = P.norm(x, res, gamma, EPS)
    half = P.HALF[torch.bfloat16]
    assert torch.equal(s.double(), want)
    assert bool(((rstd.double() - r[:, 0]).abs() <= REL * r[:, 0]).all())
    assert bool(((out.double() - y).abs() <= (half + REL) * y.abs()).all())
    P.check_image(image, y.cpu().numpy(), REL)
    want, want_g = P.norm_backward(dy, s, gamma, EPS, res)
    xh, a = s.double() * r, dy.double() * gamma.double()
    mag = r * (a.abs() + xh.abs() * (a * xh).abs().mean(1, keepdim=True))
    assert bool(((dx.double() - want).abs()
                 <= half * (1 + 2.0 ** -6) * want.abs() + 128 * P.U32 * mag).all())
    gm = (dy.double() * xh).abs().sum(0)
    assert bool(((dg.double() - want_g).abs() <= 128 * P.U32 * gm).all())


def test_the_widest_swiglu(ep):
    I = 32768
    h = torch.randn((3, 2 * I), generator=torch.Generator(device="cuda").manual_seed(1),
                    device="cuda").half()
    image = torch.empty((3, ep.f8_row_bytes(I)), dtype=torch.uint8, device="cuda")
    st = _status()
    ep.moe_swiglu_f8(h, None, image, st)
    assert int(st.item()) == 0
    P.check_image(image, P.swiglu(h).cpu().numpy(), 2.0 ** -16)


# by the kernel for few rows, by pairs with K whole and in two parts, by SMs by themselves
@pytest.mark.parametrize("sizes,N,K,dtype", [
    ([5], 64, 65536, torch.float32), ([300], 72, 65536, torch.float32),
    ([40, 0, 150, 900], 40, 65536, torch.bfloat16),
    ([1], 65536, 256, torch.float32), ([2], 65536, 1000, torch.float16),
    ([260], 65536, 256, torch.float32), ([130], 65535, 128, torch.bfloat16),
    ([0, 1, 0, 0, 2, 0, 0, 0] * 512, 24, 136, torch.float32),
    ([0, 3, 0, 1, 2, 0, 5, 0] * 512, 72, 128, torch.float32),
    ([4096] + [0] * 4094 + [1000], 264, 128, torch.bfloat16)],
    ids=lambda v: str(v).replace(" ", "")[:24])
def test_the_largest_products(ep, sizes, N, K, dtype):
    p = Problem(ep, sizes, N, K, dtype, bias=True, extra=3)
    p.run()
    p.check()


@pytest.mark.parametrize("rows,N,K,dtype", [
    (300_000, 8192, 128, torch.float32),            # results past 2^31 values
    (700_000, 64, 7168, torch.bfloat16)])           # rows past 2^32 bytes
def test_far_rows_and_results(ep, rows, N, K, dtype):
    g = torch.Generator(device="cuda")
    g.manual_seed(rows)

    def codes(*shape):
        v = torch.randn(shape, generator=g, device="cuda") * 90
        return v.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)

    size, at, kb = ep.f8_row_bytes(K), P.align32(K), P.blocks(K)
    few = 300                                       # more than a tile from either end
    a = torch.zeros((rows, size), dtype=torch.uint8, device="cuda")
    a[:few, :K], a[-few:, :K] = codes(few, K), codes(few, K)
    a.view(torch.float32)[:, at // 4:at // 4 + kb] = 1.0
    w = codes(1, N, K)
    w_scale = torch.exp2(torch.randn((1, P.blocks(N), kb), generator=g, device="cuda")) * 1e-5
    c = torch.full((rows, N), 7.0, dtype=dtype, device="cuda")
    st = _status()
    ep.moe_linear_f8(a, w, K, None, w_scale, (a, at, size), None, c, st)
    assert int(st.item()) == 0
    assert bool((c[few:-few] == 0).all())
    ones = torch.ones((few, kb))
    for part in (slice(0, few), slice(rows - few, rows)):
        want, mag = P.linear(a[part], ones, w, w_scale, K, [few])
        err = (c[part].double().cpu() - want).abs()
        assert bool((err <= P.linear_bound(want, mag, K, dtype)).all())
