"""Groups ranked without a bias, by sums of small scores: which groups stay must
follow the definition's sums in float64 wherever two of them differ by more than an
fp32 sum of two exponentials is good for.

Tolerances, on the logarithm of a group's score.  Scores of 2^-100 and more: exp
within 2 ulp, one division, one sum: 3 ulp, of at most 2^-23 each, for either of the
two compared groups; a softmax takes exp of l - max, whose rounding adds |l - max|
2^-24 (nothing where max is 0).  Below, the logarithm itself is compared, rounded
to |l| 2^-24 after the same steps and a logarithm of a number between 1 and 2."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu
ULP = 2.0 ** -23


@pytest.fixture(scope="module")
def ep():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a CUDA device")
    import combine_moe_dispatch_layout_gb300 as ep
    return ep


def _kept(ep, x, score, n, keep, top):
    """The groups whose experts are chosen, when all of theirs are."""
    T, E = x.shape
    per = E // n
    k = keep * per
    ids = torch.zeros((T, k), dtype=torch.int32, device="cuda")
    w = torch.zeros((T, k), device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    ep.moe_route(x.cuda(), None, score, k, ids, w, st, n_group=n, topk_group=keep,
                 group_top=top)
    torch.cuda.synchronize()
    assert int(st.item()) == 0 and (ids >= 0).all()
    used = torch.zeros((T, n), dtype=torch.bool)
    return used.scatter_(1, (ids.cpu() // per).long(), True).numpy()


def _check(ep, x, score, n, keep, top, at_zero=False):
    l = x.double().numpy()
    T, E = l.shape
    best = -np.sort(-l.reshape(T, n, E // n), axis=2)[:, :, :top]
    log = best if score == "softmax" else -np.logaddexp(0.0, -best)   # log of a score
    log = np.logaddexp.reduce(log, axis=2)
    used = _kept(ep, x, score, n, keep, top)
    assert (used.sum(axis=1) == keep).all()
    order = np.argsort(-log, axis=1, kind="stable")
    want = np.zeros_like(used)
    np.put_along_axis(want, order[:, :keep], True, axis=1)
    m = l.max(axis=1) if score == "softmax" else np.zeros(T)
    deep = np.abs(best).max(axis=(1, 2)) + np.abs(m)          # the largest exponent
    off = np.nonzero((used != want).any(axis=1))[0]
    for t in off:
        lost = log[t][want[t] & ~used[t]].max()
        got = log[t][used[t] & ~want[t]].min()
        small = lost - m[t] < -69.0                            # (2^-100 and about)
        tol = 2 * (3 * ULP + (0.0 if at_zero and not small else deep[t] * 2.0 ** -23))
        assert lost - got <= tol, (t, lost, got, tol)
    return len(off)


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("n,per", [(8, 4), (8, 2), (40, 2), (12, 3)])
def test_sums_of_two_scores_near_minus_forty(ep, score, n, per):
    """Sums a few 1e-7 apart: pairs of logits moved by single ulps."""
    if score == "softmax" and per < 2:
        pytest.skip("no group left for the largest logit")
    rng = np.random.default_rng(n * per)
    T, ulp = 4000, 2.0 ** -18                                  # of [32, 64)
    x = np.full((T, n, per), -60.0)
    x[:, :, 0] = -40.0 - np.round(rng.random((T, 1)) / ulp) * ulp
    x[:, :, 1] = x[:, :, 0] - np.round(rng.random((T, 1)) / ulp) * ulp
    x[:, :, :2] += rng.integers(-3, 4, (T, n, 2)) * ulp
    if score == "softmax":
        x[:, 0, 0] = 0.0                                       # the maximum: l - 0 is exact
    x = torch.from_numpy(x.reshape(T, n * per).astype(np.float32))
    _check(ep, x, score, n, n // 2, 2, at_zero=True)


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("depth", [-60.0, -72.0, -86.0, -90.0, -104.0, -150.0, -600.0])
@pytest.mark.parametrize("n,per,top,dtype", [(8, 4, 2, "fp32"), (8, 4, 1, "fp32"),
                                             (40, 3, 2, "fp32"), (16, 2, 2, "bf16")])
def test_scores_below_the_normal_range(ep, score, depth, n, per, top, dtype):
    """Scores that fp32 holds as subnormals, or not at all, still rank their groups."""
    rng = np.random.default_rng(int(-depth) + n + top)
    T = 500
    x = (depth - rng.random((T, n, per)) * 9).astype(np.float32)
    if score == "softmax":
        x[:, n - 1, per - 1] = 0.25
    x = torch.from_numpy(x.reshape(T, n * per))
    if dtype == "bf16":
        x = x.bfloat16()
    _check(ep, x, score, n, n // 2, top)
