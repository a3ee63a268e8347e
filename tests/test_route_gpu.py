"""moe_route and moe_route_backward on the GPU against float64 plain forms.

Tolerances, from the arithmetic.  A choice is an fp32 score within 3 ulp
(scores are at most 1) plus one rounded add: two choices further apart than
KEY_TOL * (1 + |choice|) are ordered as in float64; ids are compared exactly
where no bias is given and no group cut is that close, because the order is
then taken on the logits themselves.  A weight is exp within 2 ulp, a
difference l - max rounded to |l - max| 2^-24 in the exponent, sums of at most
E positive terms that each carry the same relative error, and two rounded
operations: W_RTOL + 2^-24 * (max l - min l) relative, doubled for the
quotient.  A gradient is a sum of at most k + 1 products of such weights with
the incoming gradients, so its error is that relative error times the sum of
the products' magnitudes."""
import numpy as np
import pytest
import torch

import plain_ops as P

pytestmark = pytest.mark.gpu

KEY_TOL = 1e-6
W_RTOL = 2e-6
DT = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}


@pytest.fixture(scope="module")
def ep():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a CUDA device")
    import combine_moe_dispatch_layout_gb300 as ep
    return ep


def _logits(T, E, dtype, seed, spread=1.5, pad=0, masked=0.0):
    rng = np.random.default_rng(seed)
    x = torch.from_numpy(rng.standard_normal((T, E)).astype(np.float32) * spread)
    if masked:
        x[torch.from_numpy(rng.random((T, E)) < masked)] = float("-inf")
    x = x.to(DT[dtype])
    dev = torch.full((T, E + pad), 77.0, dtype=DT[dtype], device="cuda")[:, :E]
    dev.copy_(x)
    return x.double().numpy(), dev


def _bias(E, seed):
    return np.round(np.random.default_rng(seed + 1).standard_normal(E) * 30).astype(
        np.float32) * np.float32(0.001)


def _run(ep, dev, bias, score, k, **kw):
    T = dev.shape[0]
    guard = 32
    ids = torch.full((T * k + guard,), -77, dtype=torch.int32, device="cuda")
    w = torch.full((T * k + guard,), -77.0, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    b = None if bias is None else torch.from_numpy(bias).cuda()
    ep.moe_route(dev, b, score, k, ids, w, st, **kw)
    torch.cuda.synchronize()
    assert (ids[T * k:] == -77).all() and (w[T * k:] == -77.0).all()
    return (ids[:T * k].view(T, k).cpu().numpy(), w[:T * k].view(T, k).cpu().numpy(),
            int(st.item()))


def _spread(l):
    fin = l[np.isfinite(l)]
    return float(fin.max() - fin.min()) if fin.size else 0.0


def _check(l, bias, score, k, ids, w, n_group=1, topk_group=1, group_top=1, renormalise=True,
           scale=1.0):
    ref_ids, _ = P.route(l, bias, score, k, n_group, topk_group, group_top, renormalise, scale)
    key, group, s = P.route_keys(l, bias, score, n_group, group_top)
    T, E = key.shape
    per = E // n_group
    differ = (ids != ref_ids).any(axis=1)
    if topk_group == n_group and bias is None:
        assert not differ.any(), "the order of the logits themselves"
    for t in np.nonzero(differ)[0]:
        got, want = ids[t], ref_ids[t]
        assert (got >= -1).all() and (got < E).all()
        real = got[got >= 0]
        assert len(set(real)) == len(real)
        assert (key[t, real] > -np.inf).all()
        # every group used is within the tolerance of the last group kept
        if topk_group < n_group:
            cut = np.sort(group[t])[::-1][topk_group - 1]
            used = np.unique(real // per)
            assert len(used) <= topk_group
            if not set(used) <= set(np.argsort(-group[t], kind="stable")[:topk_group]):
                close = np.abs(group[t] - cut) <= 2 * KEY_TOL * (1 + abs(cut))
                assert close.sum() >= 2, "a group that is not among the best"
                continue
        a, b = key[t, got], key[t, want]
        ok = (np.abs(a - b) <= KEY_TOL * (1 + np.abs(b))) | ((got < 0) & (want < 0))
        assert ok.all(), (t, got, want, a, b)
    assert differ.mean() <= 0.02
    ref_w = P.weights_of(s, ids, renormalise, scale)
    rtol = 2 * (W_RTOL + 2.0 ** -24 * _spread(l))
    assert (np.abs(w - ref_w) <= rtol * np.abs(ref_w) + 1e-37).all(), \
        np.max(np.abs(w - ref_w) / np.maximum(np.abs(ref_w), 1e-30))
    assert (w[ids < 0] == 0).all()


CASES = [  # T, E, k, dtype, score, bias, groups (n, keep, top), renorm, scale, pad
    (1, 1, 1, "fp32", "softmax", False, (1, 1, 1), True, 1.0, 0),
    (5, 2, 2, "bf16", "sigmoid", True, (2, 1, 1), True, 1.0, 0),
    (33, 8, 2, "fp32", "softmax", False, (1, 1, 1), False, 1.0, 3),
    (64, 31, 5, "fp16", "sigmoid", True, (1, 1, 1), True, 2.5, 0),
    (64, 60, 4, "bf16", "softmax", False, (1, 1, 1), False, 1.0, 4),
    (257, 256, 8, "fp32", "sigmoid", True, (8, 4, 2), True, 2.5, 0),
    (257, 256, 8, "fp32", "sigmoid", False, (8, 4, 2), True, 2.5, 0),
    (129, 256, 8, "bf16", "softmax", True, (8, 3, 1), True, 16.0, 8),
    (129, 256, 6, "fp16", "softmax", False, (8, 3, 1), False, 16.0, 1),
    (77, 160, 6, "fp32", "softmax", False, (8, 3, 1), False, 16.0, 0),   # 20 per group
    (77, 72, 7, "fp32", "sigmoid", True, (3, 2, 2), False, 1.0, 0),      # 24 per group
    (40, 768, 8, "bf16", "softmax", False, (1, 1, 1), False, 1.0, 0),
    (40, 768, 64, "fp32", "sigmoid", True, (1, 1, 1), True, 1.0, 0),
    (17, 1024, 33, "fp32", "softmax", True, (4, 2, 2), True, 1.0, 0),
    (9, 1025, 40, "bf16", "sigmoid", False, (1, 1, 1), True, 1.0, 0),
    (9, 4096, 64, "fp32", "softmax", True, (64, 7, 2), False, 1.0, 5),
    (3, 4096, 8, "fp16", "sigmoid", True, (2048, 3, 2), True, 1.0, 0),
    (50, 40, 40, "fp32", "sigmoid", False, (1, 1, 1), True, 1.0, 0),     # every expert
    # groups that fill no whole number of lanes
    (60, 488, 4, "fp32", "softmax", True, (8, 2, 1), True, 1.0, 0),
    (60, 480, 7, "bf16", "sigmoid", True, (12, 5, 2), False, 2.5, 0),
    (33, 96, 8, "fp32", "sigmoid", False, (32, 9, 2), True, 1.0, 0),
    (33, 66, 3, "fp16", "softmax", True, (33, 4, 1), True, 1.0, 0),
    (41, 255, 9, "fp32", "softmax", False, (5, 2, 2), False, 1.0, 2),
    (41, 1000, 50, "bf16", "sigmoid", True, (2, 1, 1), True, 1.0, 0),
    (21, 31, 6, "fp32", "sigmoid", True, (31, 30, 1), True, 1.0, 0),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "T%d_E%d_k%d_%s_%s" % c[:5])
@pytest.mark.parametrize("masked", [0.0, 0.15, 0.97])
def test_route(ep, case, masked):
    T, E, k, dtype, score, has_bias, (n, keep, top), renorm, scale, pad = case
    l, dev = _logits(T, E, dtype, seed=E * 7 + T, pad=pad, masked=masked)
    bias = _bias(E, E) if has_bias else None
    kw = dict(n_group=n, topk_group=keep, group_top=top, renormalise=renorm, scale=scale)
    ids, w, st = _run(ep, dev, bias, score, k, **kw)
    assert st == 0
    _check(l, bias, score, k, ids, w, **kw)


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("E", [24, 256, 1500])
def test_special_rows(ep, score, E):
    """Equal logits, signed zeros, one expert left, none left, infinities, huge
    and tiny values; a bias that is -inf or NaN for some experts."""
    rng = np.random.default_rng(3)
    x = np.zeros((12, E), np.float32)
    x[1] = -0.0
    x[1, 1::2] = 0.0                              # zeros of both signs tie
    x[2] = NEG
    x[2, E // 2] = -5.0                           # one expert
    x[3] = NEG                                    # none
    x[4] = rng.standard_normal(E) * 1e30
    x[5] = rng.standard_normal(E) * 1e-30
    x[6] = rng.integers(0, 3, E)                  # many ties
    x[7, ::3] = np.inf                            # read as the largest float
    x[8] = np.finfo(np.float32).min
    x[8, 5] = np.finfo(np.float32).max
    x[9] = -np.arange(E)
    x[10] = np.arange(E)
    x[11] = rng.standard_normal(E) * 50
    dev = torch.from_numpy(x).cuda()
    for kw in (dict(renormalise=True), dict(renormalise=False, scale=3.0),
               dict(n_group=4, topk_group=2, group_top=2)):
        ids, w, st = _run(ep, dev, None, score, 6, **kw)
        assert st == 0 and np.isfinite(w).all()
        ref_ids, _ = P.route(x.astype(np.float64), None, score, 6, **kw)
        rows = [t for t in range(12) if not (kw.get("n_group") and t in (4, 7, 8, 9, 10, 11))]
        # (a group's summed scores saturate there in fp32 as in any fixed precision)
        np.testing.assert_array_equal(ids[rows], ref_ids[rows])
        assert (ids[3] == -1).all() and (w[3] == 0).all()
        assert ids[2, 0] == E // 2 and (ids[2, 1:] == -1).all()
    np.testing.assert_array_equal(_run(ep, dev, None, score, 6)[0][0], np.arange(6))
    np.testing.assert_array_equal(_run(ep, dev, None, score, 6)[0][1], np.arange(6))
    bias = np.zeros(E, np.float32)
    bias[:4] = [-np.inf, np.nan, np.inf, -3.0]
    ids, w, st = _run(ep, dev[:1], bias, score, 6)
    assert st == 0 and ids[0, 0] == 2 and not ({0, 1} & set(ids[0])) and np.isfinite(w).all()


@pytest.mark.parametrize("E", [24, 256, 1500])
def test_nan_logit_is_reported_and_never_chosen(ep, E):
    x = np.random.default_rng(5).standard_normal((3, E)).astype(np.float32)
    x[1, :E - 2] = np.nan
    ids, w, st = _run(ep, torch.from_numpy(x).cuda(), None, "softmax", 4, renormalise=False)
    assert st == ep.MOE_ERR_INVALID_ARG
    ref_ids, ref_w = P.route(x.astype(np.float64), None, "softmax", 4, renormalise=False)
    np.testing.assert_array_equal(ids, ref_ids)
    np.testing.assert_allclose(w, ref_w, rtol=1e-5)


def test_empty_batch_and_side_stream(ep):
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    e = torch.empty((0, 8), device="cuda")
    ep.moe_route(e, None, "softmax", 2, torch.empty((0, 2), dtype=torch.int32, device="cuda"),
                 torch.empty((0, 2), device="cuda"), st)
    l, dev = _logits(300, 64, "fp32", seed=9)
    side = torch.cuda.Stream()
    ids = torch.empty((300, 3), dtype=torch.int32, device="cuda")
    w = torch.empty((300, 3), device="cuda")
    side.wait_stream(torch.cuda.current_stream())
    ep.moe_route(dev, None, "softmax", 3, ids, w, st, stream=side)
    side.synchronize()
    _check(l, None, "softmax", 3, ids.cpu().numpy(), w.cpu().numpy())


# ---- gradient ----------------------------------------------------------------------

def _backward(ep, dev, ids, dw, score, renorm, scale):
    T, E = dev.shape
    out = torch.full((T * E + 64,), 33.0, dtype=dev.dtype, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    ep.moe_route_backward(dev, torch.from_numpy(ids).cuda(), torch.from_numpy(dw).cuda(), score,
                          out, st, renormalise=renorm, scale=scale)
    torch.cuda.synchronize()
    assert (out[T * E:] == 33.0).all()
    return out[:T * E].view(T, E).double().cpu().numpy(), int(st.item())


def _assert_grad(got, ref, bound, dtype):
    """``got`` is the rounding to the output type of some value within ``bound``
    of ``ref`` (rounding is monotone: between the roundings of both ends)."""
    lo, hi = (torch.from_numpy(v).to(DT[dtype]).double().numpy()
              for v in (ref - bound, ref + bound))
    bad = (got < lo) | (got > hi)
    assert not bad.any(), (int(bad.sum()), got[bad][:4], ref[bad][:4], bound[bad][:4])


def _grad_bound(l, ids, dw, score, renorm, scale):
    """Sum of the magnitudes of the products behind each element, times the
    relative error of a weight: the bound of the fp32 value."""
    s = P.scores(l, score)
    p = np.where(ids >= 0, np.take_along_axis(s, np.maximum(ids, 0), 1), 0.0)
    g = np.abs(dw) * scale * (ids >= 0)
    if renorm:
        tot = p.sum(axis=1, keepdims=True)
        p = np.divide(p, tot, out=np.zeros_like(p), where=tot > 0)
    spread = p * (g + (p * g).sum(axis=1, keepdims=True))
    d = np.zeros_like(l)
    np.add.at(d, (np.arange(l.shape[0])[:, None], np.maximum(ids, 0)),
              np.where(ids >= 0, spread, 0.0))
    if score == "softmax" and not renorm:
        d += s * (p * g).sum(axis=1, keepdims=True)
    return (8 * (W_RTOL + 2.0 ** -24 * _spread(l))) * d + 1e-37


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("T,E,k,dtype,pad", [
    (1, 1, 1, "fp32", 0), (7, 2, 2, "bf16", 0), (65, 60, 4, "bf16", 4), (130, 256, 8, "fp32", 0),
    (33, 257, 8, "fp32", 3), (40, 768, 8, "bf16", 0), (9, 1025, 40, "fp16", 0),
    (5, 4096, 64, "fp32", 8), (37, 33, 8, "bf16", 0), (50, 100, 12, "fp16", 0),
    (35, 33, 13, "fp32", 0), (37, 90, 20, "bf16", 6), (6, 5, 5, "fp16", 0)])
def test_route_backward(ep, score, renorm, T, E, k, dtype, pad):
    l, dev = _logits(T, E, dtype, seed=T + E, pad=pad, masked=0.1)
    ids, _ = P.route(l, None, score, k)
    if T > 4:
        l[3] = -np.inf                            # nothing chosen in this row
        dev[3] = float("-inf")
        ids[3] = -1
    dw = np.random.default_rng(T).standard_normal((T, k)).astype(np.float32)
    got, st = _backward(ep, dev, ids, dw, score, renorm, 2.5)
    assert st == 0
    ref = P.route_backward(l, ids, dw, score, renorm, 2.5)
    _assert_grad(got, ref, _grad_bound(l, ids, dw, score, renorm, 2.5), dtype)
    if T > 4:
        assert (got[3] == 0).all()


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("renorm", [True, False])
def test_route_backward_against_differences(ep, score, renorm):
    """Central differences of sum(d_weights * weights) in float64, ids held."""
    T, E, k = 6, 24, 5
    l, dev = _logits(T, E, "fp32", seed=11)
    ids, _ = P.route(l, None, score, k)
    dw = np.random.default_rng(2).standard_normal((T, k)).astype(np.float32)
    h = 1e-5
    num = np.zeros_like(l)
    for e in range(E):
        up, dn = l.copy(), l.copy()
        up[:, e] += h
        dn[:, e] -= h
        f = [(P.weights_of(P.scores(v, score), ids, renorm, 2.5) * dw).sum(axis=1)
             for v in (up, dn)]
        num[:, e] = (f[0] - f[1]) / (2 * h)
    got, st = _backward(ep, dev, ids, dw, score, renorm, 2.5)
    assert st == 0
    # h^2 times a third derivative of order one, float64 cancellation 1e-16 / h,
    # and the fp32 result's own error
    bound = 1e-9 + _grad_bound(l, ids, dw, score, renorm, 2.5)
    assert (np.abs(got - num) <= bound).all(), np.max(np.abs(got - num) / bound)


def test_route_backward_bad_and_repeated_ids(ep):
    l, dev = _logits(3, 40, "fp32", seed=4)
    ids = np.array([[1, 40, 2], [5, 5, 7], [-1, -2, 3]], np.int32)
    dw = np.array([[1.0, 2.0, 3.0], [4.0, 5.0, 6.0], [7.0, 8.0, 9.0]], np.float32)
    got, st = _backward(ep, dev, ids, dw, "sigmoid", False, 1.0)
    assert st == ep.MOE_ERR_EXPERT_ID
    clean = np.where((ids < 0) | (ids >= 40), -1, ids)
    ref = P.route_backward(l, clean, dw, "sigmoid", False, 1.0)
    _assert_grad(got, ref, _grad_bound(l, clean, dw, "sigmoid", False, 1.0), "fp32")


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("k", [5, 8, 12, 16, 20, 40])
def test_route_backward_repeated_ids(ep, score, renorm, k):
    """Tokens that name experts several times and others not at all, among
    tokens that do not."""
    T, E = 23, 48
    l, dev = _logits(T, E, "fp32", seed=k)
    rng = np.random.default_rng(k)
    ids = np.stack([rng.permutation(E)[:k] for _ in range(T)]).astype(np.int32)
    ids[2] = ids[2, 0]
    ids[5, k - 1] = ids[5, 1]
    ids[6, ::2] = -1
    ids[22, 1:4] = ids[22, 0]
    dw = rng.standard_normal((T, k)).astype(np.float32)
    got, st = _backward(ep, dev, ids, dw, score, renorm, 1.5)
    assert st == 0
    ref = P.route_backward(l, ids, dw, score, renorm, 1.5)
    _assert_grad(got, ref, _grad_bound(l, ids, dw, score, renorm, 1.5), "fp32")


NEG = float("-inf")


@pytest.mark.parametrize("kw,err", [
    (dict(score="relu"), ValueError), (dict(k=0), Exception), (dict(k=9), Exception),
    (dict(n_group=3), Exception), (dict(n_group=2, topk_group=3), Exception),
    (dict(group_top=3), Exception), (dict(scale=float("inf")), Exception),
    (dict(scale=float("nan")), Exception)])
def test_route_refusals(ep, kw, err):
    args = dict(score="sigmoid", k=2, n_group=1, topk_group=1, group_top=1, scale=1.0)
    args.update(kw)
    x = torch.zeros((4, 8), device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    ids = torch.full((4, 16), -77, dtype=torch.int32, device="cuda")
    w = torch.zeros((4, 16), device="cuda")
    score, k = args.pop("score"), args.pop("k")
    with pytest.raises(ValueError if err is ValueError else ep.MoeError):
        ep.moe_route(x, None, score, k, ids, w, st, **args)
    torch.cuda.synchronize()
    assert (ids == -77).all()
    with pytest.raises(TypeError):
        ep.moe_route(x.double(), None, "sigmoid", 2, ids, w, st)
    with pytest.raises(ValueError):
        ep.moe_route(x.t(), None, "sigmoid", 2, ids, w, st)       # columns, not rows
    with pytest.raises(ValueError):
        ep.moe_route(x, torch.zeros(7, device="cuda"), "sigmoid", 2, ids, w, st)
    with pytest.raises(TypeError):
        ep.moe_route(x.cpu(), None, "sigmoid", 2, ids, w, st)
