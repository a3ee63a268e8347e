"""moe_combine_backward on the GPU.  Gradient rows are one fp32 product rounded
to the token dtype: compared bit for bit.  A weight's gradient is an fp32 dot
product over H: its error is at most (number of rounded steps on the longest
path) * 2^-24 times the sum of |d_out * y|; a path has at most 8 steps per
16-byte chunk of a thread, 5 in a warp and 16 across warps."""
import numpy as np
import pytest
import torch

import workloads as W

pytestmark = pytest.mark.gpu
SENT = -12345.0


@pytest.fixture(scope="module")
def pl():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a CUDA device")
    from combine_moe_dispatch_layout_gb300 import pipeline
    return pipeline


def _setup(pl, w, rows=None):
    import combine_moe_dispatch_layout_gb300 as ep
    idx, wt = W.routing(w)
    b = pl.PipelineBuffers(w.R, w.bs, w.k, w.epr, w.H, w.dtype, False)
    idx_d = idx.cuda()
    pl.run_layout_notify(b, idx_d)
    y = W.expert_outputs(w, rows)
    d_out = W.tokens(w.with_(seed=w.seed + 5))
    d_y = torch.full(y.shape, SENT, dtype=y.dtype, device="cuda")
    d_w = torch.full((w.T * w.k + 32,), SENT, device="cuda")
    torch.cuda.synchronize()
    assert b.status() == 0
    ep.moe_combine_backward(b.shape, d_out.cuda(), y.cuda(), idx_d, wt.cuda(), b.send_idx,
                            b.put_offset, b.rank_recv_base, d_y, d_w, b.dev_status)
    torch.cuda.synchronize()
    s, put, base = (t.cpu().numpy() for t in (b.send_idx, b.put_offset, b.rank_recv_base))
    e = idx.numpy()
    src = np.arange(w.T)[:, None] // w.bs
    row = base[e // w.epr] + put[e * w.R + src] + s
    assert (d_w[w.T * w.k:] == SENT).all()
    return dict(row=row, wt=wt, y=y, d_out=d_out, d_y=d_y.cpu(), status=b.status(),
                d_w=d_w[:w.T * w.k].view(w.T, w.k).cpu().numpy())


def _check(w, r, valid=None):
    valid = np.ones(r["row"].shape, bool) if valid is None else valid
    want = torch.full(r["y"].shape, SENT, dtype=r["y"].dtype)
    t, k = np.nonzero(valid)
    rows = torch.from_numpy(r["row"][t, k])
    prod = r["wt"][t, k][:, None] * r["d_out"][t].float()
    want[rows] = prod.to(want.dtype)
    assert torch.equal(r["d_y"].view(torch.int16), want.view(torch.int16))
    d = r["d_out"][t].double().numpy()
    y = r["y"][rows].double().numpy()
    ref, mag = (d * y).sum(axis=1), np.abs(d * y).sum(axis=1)
    chunks = -(-w.H // 8)
    steps = 8 * -(-chunks // max(32, min(480, chunks // 2))) + 5 + 16
    got = r["d_w"][t, k]
    assert (np.abs(got - ref) <= steps * 2.0 ** -24 * mag + 1e-37).all()
    assert (r["d_w"][~valid] == 0).all()


CASES = [W.Workload("one", R=1, epr=1, bs=1, k=1, H=8),
         W.Workload("narrow", R=3, epr=5, bs=77, k=7, H=72, dtype=W.FP16),
         W.Workload("ragged", R=5, epr=3, bs=200, k=4, H=1000),
         W.Workload("deep", R=2, epr=40, bs=50, k=64, H=256, dtype=W.FP16),
         W.Workload("half", R=2, epr=7, bs=65, k=6, H=504),
         W.Workload("nine", R=4, epr=6, bs=111, k=9, H=520),
         W.Workload("model", R=8, epr=32, bs=64, k=8, H=7168, outlier_p=0.01),
         W.Workload("wide", R=1, epr=4, bs=9, k=3, H=65536)]


@pytest.mark.parametrize("w", CASES, ids=lambda w: w.name)
def test_combine_backward(pl, w):
    r = _setup(pl, w)
    assert r["status"] == 0
    _check(w, r)


def test_short_buffer_and_run_twice(pl):
    """Rows past the buffer: status, weight gradient 0, nothing written there;
    and two runs give the same bits."""
    w = CASES[2]
    n = w.P - 700
    r = _setup(pl, w, rows=n)
    assert r["status"] == 3
    _check(w, r, valid=r["row"] < n)
    again = _setup(pl, w, rows=n)
    assert np.array_equal(r["d_w"].view(np.int32), again["d_w"].view(np.int32))


def test_gradient_against_differences(pl):
    """The gradients of f = sum(d_out * out) in float64: out is linear in y and
    in the weights, so a difference quotient is exact up to rounding."""
    w = W.Workload("diff", R=2, epr=3, bs=5, k=2, H=16)
    r = _setup(pl, w)
    wt, y, d = r["wt"].double().numpy(), r["y"].double().numpy(), r["d_out"].double().numpy()

    def f(wt, y):
        return (d * (wt[:, :, None] * y[r["row"]]).sum(axis=1)).sum()

    base = f(wt, y)
    for t, k in ((0, 0), (3, 1), (9, 0)):
        up = wt.copy()
        up[t, k] += 0.5
        mag = np.abs(d[t] * y[r["row"][t, k]]).sum()
        assert abs((f(up, y) - base) / 0.5 - r["d_w"][t, k]) <= 32 * 2.0 ** -24 * mag + 1e-9
        for h in (0, 7, 15):
            up = y.copy()
            up[r["row"][t, k], h] += 0.5
            num = (f(wt, up) - base) / 0.5
            got = float(r["d_y"][r["row"][t, k], h])
            assert abs(num - got) <= 2.0 ** -8 * abs(num) + 1e-9    # one bf16 rounding


def test_empty_batch_and_refusals(pl):
    import combine_moe_dispatch_layout_gb300 as ep
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    z = torch.zeros((4, 64), dtype=torch.bfloat16, device="cuda")
    i = torch.zeros(64, dtype=torch.int32, device="cuda")
    f = torch.zeros(64, device="cuda")
    base = torch.zeros(3, dtype=torch.int64, device="cuda")
    empty = ep.make_shape(2, 0, 2, 2, 64)
    assert ep.moe_combine_backward(empty, z, z, i, f, i, i, base, z, f, st) == 0
    good = ep.make_shape(2, 1, 2, 2, 64)
    with pytest.raises(TypeError):
        ep.moe_combine_backward(good, z.float(), z, i, f, i, i, base, z, f, st)
    with pytest.raises(ValueError):
        ep.moe_combine_backward(good, z[:1], z, i, f, i, i, base, z, f, st)
    with pytest.raises(ep.MoeError):
        ep.moe_combine_backward(ep.make_shape(2, 1, 2, 2, 60), z, z, i, f, i, i, base, z, f, st)
