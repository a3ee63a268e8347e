"""Renormalised and plain sigmoid weights, and their gradients, of tokens whose
chosen logits are all far below 0, where the scores themselves leave fp32's normal
range: against the float64 definition.

Tolerances.  A renormalised weight is a quotient of exponentials of differences of
chosen logits: the relative error of test_route_gpu (exp within 2 ulp, the difference
rounded to |difference| 2^-24 in the exponent, sums of positive terms, two rounded
operations).  A plain score below 2^-126 is a multiple of 2^-149 and its products
with the scale and the gradient too, so it has a few units of 2^-149 besides."""
import numpy as np
import pytest
import torch

import plain_ops as P

pytestmark = pytest.mark.gpu

W_RTOL = 2e-6
TINY = 2.0 ** -149
DT = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}


@pytest.fixture(scope="module")
def ep():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a CUDA device")
    import combine_moe_dispatch_layout_gb300 as ep
    return ep


def _route(ep, dev, k, renorm, scale):
    T = dev.shape[0]
    ids = torch.full((T, k), -77, dtype=torch.int32, device="cuda")
    w = torch.full((T, k), -77.0, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    ep.moe_route(dev, None, "sigmoid", k, ids, w, st, renormalise=renorm, scale=scale)
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    return ids.cpu().numpy(), w.double().cpu().numpy()


def _backward(ep, dev, ids, dw, renorm, scale):
    out = torch.full(dev.shape, 33.0, dtype=dev.dtype, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    ep.moe_route_backward(dev, torch.from_numpy(ids).cuda(), torch.from_numpy(dw).cuda(),
                          "sigmoid", out, st, renormalise=renorm, scale=scale)
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    return out.double().cpu().numpy()


def _rows(E, dtype, seed):
    """Logits around each of several depths, a row that reaches from 0 down to
    each, and what float64 makes of the rounded values."""
    rng = np.random.default_rng(seed)
    rows = []
    for depth in (-60.0, -80.0, -88.0, -88.73, -90.0, -95.0, -103.0, -104.5, -110.0, -200.0,
                  -700.0):
        for spread in (0.0, 0.8, 6.0):
            rows.append(depth - np.abs(rng.standard_normal(E)) * spread)
    for depth in (-90.0, -103.0):
        rows.append(np.where(np.arange(E) == 1, 0.5, depth - rng.random(E)))
        rows.append(np.where(np.arange(E) == 1, -20.0, depth - rng.random(E)))
    x = torch.from_numpy(np.stack(rows).astype(np.float32)).to(DT[dtype])
    return x.double().numpy(), x.cuda()


@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("E,k,dtype", [(1, 1, "fp32"), (16, 1, "fp32"), (16, 8, "fp32"),
                                       (256, 8, "fp32"), (40, 13, "bf16"), (64, 40, "fp32"),
                                       (300, 6, "fp16"), (1500, 8, "fp32")])
def test_chosen_logits_far_below_zero(ep, renorm, E, k, dtype):
    scale = 2.5
    l, dev = _rows(E, dtype, seed=E + k)
    ids, w = _route(ep, dev, k, renorm, scale)
    ref_ids, ref_w = P.route(l, None, "sigmoid", k, renormalise=renorm, scale=scale)
    np.testing.assert_array_equal(ids, ref_ids)
    chosen = np.take_along_axis(l, ids, 1)
    deep = chosen.max(axis=1, keepdims=True) - chosen.min(axis=1, keepdims=True)
    rel = 2 * (W_RTOL + 2.0 ** -24 * deep)
    assert np.isfinite(w).all()
    assert (np.abs(w - ref_w) <= rel * np.abs(ref_w) + 4 * scale * TINY).all()
    if renorm:
        np.testing.assert_allclose(w.sum(axis=1), scale, rtol=1e-5)

    dw = np.random.default_rng(k).standard_normal((l.shape[0], k)).astype(np.float32)
    got = _backward(ep, dev, ids, dw, renorm, scale)
    ref = P.route_backward(l, ids, dw, "sigmoid", renorm, scale)
    p = ref_w / scale                                # (a plain weight is the score itself)
    g = np.abs(dw) * scale
    size = p * (g + (p * g).sum(axis=1, keepdims=True) * renorm)
    bound = np.zeros_like(l)
    np.add.at(bound, (np.arange(l.shape[0])[:, None], ids),
              8 * (W_RTOL + 2.0 ** -24 * deep) * size + 8 * (1 + g) * TINY)
    lo, hi = (torch.from_numpy(v).to(DT[dtype]).double().numpy()
              for v in (ref - bound, ref + bound))
    assert np.isfinite(got).all()
    assert ((got >= lo) & (got <= hi)).all()


@pytest.mark.parametrize("dtype", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("E", [24, 1500])
def test_logits_of_the_types_lowest_value(ep, dtype, E):
    """Masked by the type's lowest value instead of -inf: such experts are available,
    and where nothing else is they share the token evenly; beside any other one they
    weigh nothing.  -inf alone leaves nothing."""
    k = 6
    x = torch.full((3, E), torch.finfo(DT[dtype]).min, dtype=DT[dtype], device="cuda")
    x[1, 7] = -100.0
    x[2] = float("-inf")
    ids, w = _route(ep, x, k, True, 1.0)
    assert ids[0].tolist() == list(range(k)) and ids[1, 0] == 7
    np.testing.assert_allclose(w[0], 1.0 / k, rtol=2 * W_RTOL)
    np.testing.assert_array_equal(w[1], [1.0] + [0.0] * (k - 1))
    assert (ids[2] == -1).all() and (w[2] == 0).all()
    dw = np.arange(3 * k, dtype=np.float32).reshape(3, k)
    d = _backward(ep, x, ids, dw, True, 1.0)
    want = (dw[0] - dw[0].mean()) / k
    tol = {"fp32": 8 * W_RTOL, "bf16": 2.0 ** -8, "fp16": 2.0 ** -11}[dtype]
    np.testing.assert_allclose(d[0, :k], want, rtol=tol, atol=8 * W_RTOL)
    assert (d[0, k:] == 0).all() and (d[1] == 0).all() and (d[2] == 0).all()
