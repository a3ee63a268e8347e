"""Rows and elements past the reach of 32-bit offsets: routing and its gradient
over logits whose rows lie far apart, the INT8 product with far rows, far
weights and a result of more than 2^31 elements."""
import numpy as np
import pytest
import torch

import plain_ops as P

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ep():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a CUDA device")
    import combine_moe_dispatch_layout_gb300 as ep
    return ep


@pytest.mark.parametrize("E", [64, 1200])
def test_logits_far_apart(ep, E):
    T, k, stride = 4, 6, (1 << 30) + 24
    rng = np.random.default_rng(E)
    buf = torch.empty((T - 1) * stride + E, dtype=torch.bfloat16, device="cuda")
    far = torch.as_strided(buf, (T, E), (stride, 1))
    near = torch.from_numpy(rng.standard_normal((T, E)).astype(np.float32)).cuda().bfloat16()
    far.copy_(near)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = []
    for x in (near, far):
        ids = torch.empty((T, k), dtype=torch.int32, device="cuda")
        w = torch.empty((T, k), device="cuda")
        ep.moe_route(x, None, "softmax", k, ids, w, st, renormalise=False)
        for renorm in (True, False):
            d = torch.empty((T, E), dtype=torch.bfloat16, device="cuda")
            ep.moe_route_backward(x, ids, w, "softmax", d, st, renormalise=renorm)
            out.append(d.view(torch.int16).cpu())
        out += [ids.cpu(), w.view(torch.int32).cpu()]
    assert int(st.item()) == 0
    for a, b in zip(out[:4], out[4:]):
        assert torch.equal(a, b)
    ref, _ = P.route(near.double().cpu().numpy(), None, "softmax", k, renormalise=False)
    assert np.array_equal(out[2].numpy(), ref)


def _codes(rng, shape):
    return rng.integers(-128, 128, shape).astype(np.int8)


def _far(codes, stride):
    """The rows of a 2-D array of codes on the device, `stride` bytes apart."""
    rows, K = codes.shape
    buf = torch.empty((rows - 1) * stride + K + 16, dtype=torch.int8, device="cuda")
    view = torch.as_strided(buf, (rows, (K + 15) // 16 * 16), (stride, 1))
    view[:, :K] = torch.from_numpy(codes).cuda()
    return view


@pytest.mark.parametrize("rows,N,K,stride", [
    (3, 200, 304, (1 << 31) + 16), (20, 7000, 96, (1 << 28) + 48)])
def test_rows_far_apart(ep, rows, N, K, stride):
    rng = np.random.default_rng(rows)
    a, w = _codes(rng, (rows, K)), _codes(rng, (1, N, K))
    y = torch.empty((rows, N), dtype=torch.int32, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    ep.moe_linear_i8(_far(a, stride), torch.from_numpy(w).cuda(), K, None, None, None, None, y,
                     st)
    assert int(st.item()) == 0
    assert np.array_equal(y.cpu().numpy(), P.linear_i8(a, w, [rows]))


@pytest.mark.parametrize("rows,K", [(2, 512), (6000, 32)])
def test_weights_far_apart(ep, rows, K):
    N, stride = 24, 1 << 28
    rng = np.random.default_rng(rows)
    a, w = _codes(rng, (rows, K)), _codes(rng, (1, N, K))
    wd = torch.empty((1, N, stride), dtype=torch.int8, device="cuda")
    wd[0, :, :K] = torch.from_numpy(w[0]).cuda()
    y = torch.empty((rows, N), dtype=torch.int32, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    ep.moe_linear_i8(torch.from_numpy(a).cuda(), wd, K, None, None, None, None, y, st)
    assert int(st.item()) == 0
    assert np.array_equal(y.cpu().numpy(), P.linear_i8(a, w, [rows]))


def test_a_result_of_more_than_two_to_the_31_elements(ep):
    rows, N, K = 33000, 65536, 16
    rng = np.random.default_rng(1)
    a, w = _codes(rng, (rows, K)), _codes(rng, (1, N, K))
    col = (rng.random((1, N)) + 0.5).astype(np.float32)
    scale = (rng.random(rows) + 0.5).astype(np.float32)
    y = torch.zeros((rows, N), dtype=torch.bfloat16, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    ep.moe_linear_i8(torch.from_numpy(a).cuda(), torch.from_numpy(w).cuda(), K, None,
                     torch.from_numpy(col).cuda(), (torch.from_numpy(scale).cuda(), 0, 4), None, y,
                     st)
    assert int(st.item()) == 0
    for some in (slice(0, 3), slice(32760, 32772), slice(rows - 5, rows)):
        part = a[some]
        want = P.linear_i8(part, w, [len(part)], col, scale[some])
        want = torch.from_numpy(want).to(torch.bfloat16)
        assert torch.equal(y[some].cpu().view(torch.int16), want.view(torch.int16))
