"""SwiGLU to e4m3 row images against float64.  h is asked within 2^-16 of itself, the
documented bound."""
import numpy as np
import pytest
import torch

import plain_f8 as P

pytestmark = pytest.mark.gpu
REL = 2.0 ** -16


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


def _guarded(rows, size):
    raw = torch.full((rows + 2, size), 0xA5, dtype=torch.uint8, device="cuda")
    return raw, raw[1:rows + 1]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("I", [8, 40, 128, 136, 256, 264, 384, 512, 520, 1000, 1032, 2048, 4608])
@pytest.mark.parametrize("M", [1, 5, 333])
def test_rows(ep, M, I, dtype):
    g = _gen(M + I)
    gap = 8 * (I % 5)
    wide = (torch.randn((M, 2 * I + gap), generator=g, device="cuda") * 3).to(dtype)
    h = wide[:, :2 * I]
    raw, image = _guarded(M, ep.f8_row_bytes(I))
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    ep.moe_swiglu_f8(h, None, image, st)
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    assert bool((raw[0] == 0xA5).all()) and bool((raw[-1] == 0xA5).all())
    P.check_image(image, P.swiglu(h).cpu().numpy(), REL)


@pytest.mark.parametrize("total", [0, 1, 7, 20])
def test_rows_past_the_groups_are_left(ep, total):
    M, I = 20, 384
    h = torch.randn((M, 2 * I), generator=_gen(total), device="cuda").bfloat16()
    off = torch.tensor([0, total // 2, total // 2, total], device="cuda")
    image = torch.full((M, ep.f8_row_bytes(I)), 0xA5, dtype=torch.uint8, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    ep.moe_swiglu_f8(h, off, image, st)
    torch.cuda.synchronize()
    assert int(st.item()) == 0 and bool((image[total:] == 0xA5).all())
    if total:
        P.check_image(image[:total], P.swiglu(h[:total]).cpu().numpy(), REL)


def test_offsets_past_the_rows(ep):
    M, I = 6, 128
    h = torch.randn((M, 2 * I), generator=_gen(1), device="cuda")
    image = torch.empty((M, ep.f8_row_bytes(I)), dtype=torch.uint8, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    ep.moe_swiglu_f8(h, torch.tensor([0, 9], device="cuda"), image, st)
    assert int(st.item()) == ep.MOE_ERR_CAPACITY
    P.check_image(image, P.swiglu(h).cpu().numpy(), REL)


def test_extreme_values(ep):
    """Gates far on both sides, zeros, the largest numbers, an infinity and a NaN: each in
    blocks of their own, the others untouched by them."""
    I = 1024
    h = torch.randn((1, 2 * I), generator=_gen(3), device="cuda")
    gate, up = h[:, :I], h[:, I:]
    gate[0, 0:128] = torch.linspace(-80, 80, 128, device="cuda")
    gate[0, 128:256] = 0
    up[0, 256:384] = 0
    gate[0, 384:512], up[0, 384:512] = 3e38, 1.0
    gate[0, 512:640] = -1e30                        # sigmoid 0: exactly nothing
    gate[0, 640] = float("nan")
    up[0, 768] = float("inf")
    image = torch.empty((1, ep.f8_row_bytes(I)), dtype=torch.uint8, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    ep.moe_swiglu_f8(h, None, image, st)
    codes, scales, _ = P.split_image(image, I)
    y = P.swiglu(h).cpu().numpy()
    assert np.isnan(codes[0, 640:768]).all() and np.isnan(scales[0, 5])
    assert np.isinf(scales[0, 6]) and np.isnan(codes[0, 768])
    assert not codes[0, 128:384].any() and not codes[0, 512:640].any()
    assert np.isfinite(codes[0, 384:512]).all()
    for b in (0, 1, 2, 3, 7):
        part = slice(128 * b, 128 * b + 128)
        ref = y[:, part]
        top = max(np.abs(ref).max(), P.TINY)
        np.testing.assert_allclose(scales[0, b], top / 448, rtol=REL + 4 * P.U32)
        tol = np.maximum(2.0 ** -4 * np.abs(ref), 2.0 ** -10 * scales[0, b]) * 1.001
        assert (np.abs(codes[:, part] * scales[0, b] - ref) <= tol + REL * np.abs(ref)).all()


def test_many_rows(ep):
    """More 128-value blocks than 32-bit bytes of input: 1,100,000 rows of 2 x 1024."""
    M, I = 1_100_000, 1024
    h = torch.zeros((M, 2 * I), dtype=torch.bfloat16, device="cuda")
    rows = [0, M // 2 + 1, M - 1]
    h[rows] = torch.randn((3, 2 * I), generator=_gen(4), device="cuda").bfloat16()
    image = torch.full((M, ep.f8_row_bytes(I)), 0xA5, dtype=torch.uint8, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    ep.moe_swiglu_f8(h, None, image, st)
    P.check_image(image[rows], P.swiglu(h[rows]).cpu().numpy(), REL)
    assert bool((image[1, :I] == 0).all()) and bool((image[M - 2, :I] == 0).all())
