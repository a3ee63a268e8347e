"""Host-side refusals of the norm, its gradient, SwiGLU to e4m3 and the e4m3 product, through
the C ABI (no GPU: pointers are never dereferenced), and the plain float64 forms against
hand-worked cases and difference quotients."""
import ctypes
import os
import shutil

import numpy as np
import pytest
import torch

import plain_f8 as P

OK = ctypes.c_void_p(0x10000)
ODD = ctypes.c_void_p(0x10008)
OFF = ctypes.c_void_p(0x10002)


@pytest.fixture(scope="module")
def lib():
    if shutil.which("nvcc") is None and not os.path.exists("/usr/local/cuda/bin/nvcc"):
        pytest.skip("nvcc not available")
    import __graft_entry__
    __graft_entry__._load_builder().build()
    import combine_moe_dispatch_layout_gb300 as ep
    return ep.lib()


NORM = dict(x=OK, dtype=0, T=4, H=64, x_stride=64, res=OK, res_stride=64, gamma=OK, eps=1e-6,
            sum=OK, sum_stride=64, out=OK, out_stride=64, codes=OK, code=1, rstd=OK, st=OK,
            stream=None)


@pytest.mark.parametrize("bad", [
    dict(x=None), dict(x=ODD), dict(dtype=2), dict(dtype=-1), dict(T=-1), dict(T=1 << 31),
    dict(H=0), dict(H=4), dict(H=68), dict(H=65544), dict(x_stride=56), dict(x_stride=68),
    dict(x_stride=1 << 32), dict(res=None), dict(res=ODD), dict(res_stride=60),
    dict(gamma=None), dict(gamma=ODD), dict(eps=0.0), dict(eps=-1.0), dict(eps=float("inf")),
    dict(eps=float("nan")), dict(sum=None), dict(sum=ODD), dict(sum_stride=8),
    dict(out=ODD), dict(out_stride=4), dict(out=None, codes=None), dict(codes=ODD),
    dict(code=2), dict(code=-1), dict(rstd=OFF), dict(st=None), dict(st=OFF)], ids=str)
def test_norm(lib, bad):
    assert lib.moe_rms_norm(*dict(NORM, **bad).values()) == 1


def test_norm_empty_batch_touches_nothing(lib):
    a = dict(NORM, T=0, x=None, res=None, sum=None, gamma=None, out=None, codes=None)
    assert lib.moe_rms_norm(*a.values()) == 0


BACK = dict(dy=OK, dtype=1, T=4, H=64, dy_stride=64, x=OK, x_stride=64, gamma=OK, rstd=OK, ds=OK,
            ds_stride=64, dx=OK, dx_stride=64, dg=OK, ws=OK, st=OK, stream=None)


@pytest.mark.parametrize("bad", [
    dict(dy=None), dict(dy=ODD), dict(dtype=2), dict(T=-1), dict(T=1 << 31), dict(H=7),
    dict(H=65544), dict(dy_stride=63), dict(x=None), dict(x=ODD), dict(x_stride=32),
    dict(gamma=None), dict(gamma=ODD), dict(rstd=None), dict(rstd=OFF), dict(ds=ODD),
    dict(ds_stride=0), dict(dx=None), dict(dx=ODD), dict(dx_stride=72 + 4), dict(dg=None),
    dict(dg=OFF), dict(ws=None), dict(ws=ODD), dict(st=None)], ids=str)
def test_norm_backward(lib, bad):
    assert lib.moe_rms_norm_backward(*dict(BACK, **bad).values()) == 1


def test_workspace_sizes(lib):
    size = lib.moe_rms_norm_backward_workspace_bytes
    for T, H in ((-1, 64), (4, 0), (4, 60), (4, 65544), (1 << 31, 64)):
        assert size(T, H) == 0
    for T in (0, 1, 5, 1000, 1 << 30):
        for H in (8, 64, 1000, 7168, 16384, 16392, 65536):
            n = size(T, H)
            assert n > 0 and n % (4 * H) == 0 and n <= 304 * 4 * H


SWIGLU = dict(h=OK, dtype=0, M=4, I=64, stride=128, off=OK, G=2, codes=OK, st=OK, stream=None)


@pytest.mark.parametrize("bad", [
    dict(h=None), dict(h=ODD), dict(dtype=3), dict(dtype=-1), dict(M=-1), dict(M=1 << 31),
    dict(M=(1 << 31) - 1, I=32768, stride=65536),
    dict(I=0), dict(I=60), dict(I=32776), dict(stride=120), dict(stride=132), dict(off=OFF),
    dict(G=0), dict(G=4097), dict(codes=None), dict(codes=ODD), dict(st=None), dict(st=OFF)],
    ids=str)
def test_swiglu(lib, bad):
    assert lib.moe_swiglu_f8(*dict(SWIGLU, **bad).values()) == 1


def test_swiglu_no_rows(lib):
    assert lib.moe_swiglu_f8(*dict(SWIGLU, M=0, h=None, codes=None).values()) == 0


LINEAR = dict(a=OK, rows=4, a_stride=320, w=OK, w_stride=304, G=2, N=24, K=300, sizes=OK, ws=OK,
              s=OK, s_stride=12, bias=OK, c=OK, dtype=0, st=OK, stream=None)


@pytest.mark.parametrize("bad", [
    dict(a=None), dict(a=ODD), dict(rows=-1), dict(rows=(1 << 31) - 512),
    dict(rows=1 << 30, N=65536), dict(a_stride=288), dict(a_stride=328), dict(a_stride=1 << 32),
    dict(w=None), dict(w=ODD), dict(w_stride=288), dict(w_stride=312), dict(w_stride=1 << 32),
    dict(G=0), dict(G=4097), dict(N=0), dict(N=65537), dict(K=0), dict(K=65537),
    dict(sizes=None), dict(sizes=OFF), dict(ws=None), dict(ws=OFF), dict(s=None), dict(s=OFF),
    dict(s_stride=8), dict(s_stride=14), dict(s_stride=1 << 32), dict(s_stride=-4),
    dict(bias=OFF), dict(c=None), dict(c=ODD), dict(dtype=3), dict(dtype=-1), dict(st=None),
    dict(st=OFF)], ids=str)
def test_linear(lib, bad):
    assert lib.moe_linear_f8(*dict(LINEAR, **bad).values()) == 1


def test_linear_no_rows(lib):
    assert lib.moe_linear_f8(*dict(LINEAR, rows=0, a=None, c=None).values()) == 0


def test_row_bytes(lib):
    for H, want in ((1, 64), (32, 64), (33, 96), (128, 160), (129, 192), (1000, 1056),
                    (1024, 1056), (1025, 1120), (7168, 7392), (65536, 67584)):
        assert lib.moe_f8_row_bytes(H) == want == P.f8_row_bytes(H)
    assert lib.moe_f8_row_bytes(0) == lib.moe_f8_row_bytes(65537) == -1


def test_binding_refuses_what_is_no_cuda_tensor(lib):
    import combine_moe_dispatch_layout_gb300 as ep
    x = torch.zeros((4, 64), dtype=torch.bfloat16)
    st = torch.zeros(1, dtype=torch.int32)
    with pytest.raises(TypeError):
        ep.moe_rms_norm(x, None, torch.ones(64), 1e-6, None, x, None, None, st)
    with pytest.raises(TypeError):
        ep.moe_rms_norm_backward(x, x, torch.ones(64), torch.ones(4), None, x, torch.ones(64),
                                 st, st)
    with pytest.raises(TypeError):
        ep.moe_swiglu_f8(x, None, st, st)
    with pytest.raises(TypeError):
        ep.moe_linear_f8(x, x[None], 64, None, None, (x, 0, 4), None, x, st)


# ---- the plain forms the GPU tests compare with -----------------------------------------

def test_e4m3_values():
    assert P.TABLE[0x7E] == 448 and np.isnan(P.TABLE[0x7F]) and P.TABLE[0x38] == 1.0
    assert P.TABLE[1] == 2.0 ** -9 and P.TABLE[0x08] == 2.0 ** -6 and P.TABLE[0xB8] == -1.0


def test_plain_norm_by_hand():
    x = torch.tensor([[3.0, 4.0, 0.0, 0.0]], dtype=torch.float16)
    s, r, y = P.norm(x, torch.tensor([[0.0, 0.0, 0.0, 12.0]], dtype=torch.float16),
                     torch.tensor([1.0, 2.0, 1.0, 0.5]), 0.0)
    assert s.tolist() == [[3.0, 4.0, 0.0, 12.0]]
    np.testing.assert_allclose(r, [[2 / 13]], rtol=1e-15)           # sqrt(4 / 169)
    np.testing.assert_allclose(y, [[6 / 13, 16 / 13, 0, 12 / 13]], rtol=1e-15)


def test_plain_norm_gradient_is_the_difference_quotient():
    g = torch.Generator().manual_seed(3)
    x, c, ds = (torch.randn((3, 16), generator=g, dtype=torch.float64) for _ in range(3))
    gamma = torch.rand(16, generator=g, dtype=torch.float64)
    d, dg = P.norm_backward(c, x, gamma, 1e-3, ds)

    def loss(v, w):
        return (c * P.norm(v, None, w, 1e-3)[2]).sum() + (ds * v).sum()

    h = 1e-6
    for j in range(16):
        for i in range(3):
            e = torch.zeros_like(x)
            e[i, j] = h
            q = (loss(x + e, gamma) - loss(x - e, gamma)) / (2 * h)
            assert abs(float(q - d[i, j])) < 1e-8
        e = torch.zeros_like(gamma)
        e[j] = h
        q = (loss(x, gamma + e) - loss(x, gamma - e)) / (2 * h)
        assert abs(float(q - dg[j])) < 1e-8


def test_plain_swiglu_by_hand():
    h = torch.tensor([[0.0, np.log(3.0), -np.log(3.0), 2.0, 4.0, 8.0]], dtype=torch.float64)
    np.testing.assert_allclose(P.swiglu(h), [[0.0, np.log(3.0) * 0.75 * 4,
                                              -np.log(3.0) * 0.25 * 8]], rtol=1e-15)


def test_plain_product_by_hand():
    one, two = 0x38, 0x40                                   # 1.0, 2.0
    a = torch.tensor([[one] * 128 + [two] * 2], dtype=torch.uint8)
    w = torch.full((1, 1, 130), two, dtype=torch.uint8)
    c, mag = P.linear(a, torch.tensor([[0.5, 3.0]]), w, torch.tensor([[[2.0, 10.0]]]), 130, [1],
                      torch.tensor([[-1.0]]))
    assert c.tolist() == [[0.5 * 2 * 256 + 3 * 10 * 8 - 1]] and mag.tolist() == [[497.0]]


def test_plain_image_check_sees_a_wrong_code():
    y = np.linspace(-2, 2, 128)[None]
    scale = 2.0 / 448
    near = np.abs(P.TABLE[None, :] - (y / scale)[0][:, None])
    codes = np.nanargmin(near, axis=1).astype(np.uint8)
    image = np.zeros((1, 160), np.uint8)
    image[0, :128] = codes
    image[0, 128:132] = np.array([scale], np.float32).view(np.uint8)
    P.check_image(torch.from_numpy(image), y, 0.0)
    for at, to in ((3, image[0, 3] - 1), (131, image[0, 131] ^ 1), (140, 1)):
        wrong = image.copy()
        wrong[0, at] = to
        with pytest.raises(AssertionError):
            P.check_image(torch.from_numpy(wrong), y, 0.0)
