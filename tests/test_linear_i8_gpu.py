"""moe_linear_i8 on the GPU, bit for bit: the accumulators are exact integers,
and every later step is one fp32 rounding that numpy repeats."""
import numpy as np
import pytest
import torch

import plain_ops as P

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32,
      "int32": torch.int32}


@pytest.fixture(scope="module")
def ep():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a CUDA device")
    import combine_moe_dispatch_layout_gb300 as ep
    return ep


def _case(sizes, N, K, seed, images=False, a_pad=0, w_pad=0, extra_rows=0, codes=None):
    """Host codes and device operands; the bytes past K hold garbage."""
    rng = np.random.default_rng(seed)
    rows, G = int(sum(sizes)), len(sizes)
    lo, hi = codes or (-128, 128)
    a = rng.integers(lo, hi, (rows + extra_rows, K)).astype(np.int8)
    w = rng.integers(lo, hi, (G, N, K)).astype(np.int8)
    wide = (K + 15) // 16 * 16
    row = (rng.random(rows + extra_rows).astype(np.float32) * 3 + 0.1) / 127
    at = (K + 31) // 32 * 32
    stride = at + 32 if images else wide + a_pad
    ah = rng.integers(0, 256, (rows + extra_rows, stride)).astype(np.uint8)
    ah[:, :K] = a.view(np.uint8)
    if images:
        ah[:, at:at + 4] = row.view(np.uint8).reshape(-1, 4)
    wh = rng.integers(0, 256, (G, N, wide + w_pad)).astype(np.uint8)
    wh[:, :, :K] = w.view(np.uint8)
    col = ((rng.random((G, N)) + 0.5) / (73.6 * K ** 0.5)).astype(np.float32)
    bias = rng.standard_normal((G, N)).astype(np.float32)
    dev = dict(a=torch.from_numpy(ah).cuda(), w=torch.from_numpy(wh).cuda(),
               col=torch.from_numpy(col).cuda(), bias=torch.from_numpy(bias).cuda(),
               sizes=torch.tensor(list(sizes), dtype=torch.int32, device="cuda"),
               row=torch.from_numpy(row).cuda())
    dev["scale"] = (dev["a"], at, stride) if images else (dev["row"], 0, 4)
    return dict(a=a, w=w, row=row, col=col, bias=bias, sizes=list(sizes), K=K, N=N, dev=dev)


def _run(ep, c, out, bias=False, group_rows=True, st=None, stream=None):
    d = c["dev"]
    rows, N = d["a"].shape[0], c["N"]
    item = torch.empty((), dtype=DT[out]).element_size()
    guard = 256 // item
    buf = torch.zeros(guard + rows * N + guard, dtype=DT[out], device="cuda")
    raw = buf.view(torch.uint8)
    raw.fill_(0xA5)
    y = buf[guard:guard + rows * N].view(rows, N)
    st = torch.zeros(1, dtype=torch.int32, device="cuda") if st is None else st
    plain = out == "int32"
    torch.cuda.synchronize()
    ep.moe_linear_i8(d["a"], d["w"], c["K"], d["sizes"] if group_rows else None,
                     None if plain else d["col"], None if plain else d["scale"],
                     d["bias"] if bias else None, y, st, stream=stream)
    torch.cuda.synchronize()
    raw = raw.cpu().numpy()
    assert (raw[:256] == 0xA5).all() and (raw[-256:] == 0xA5).all(), "a write outside c"
    return y.cpu(), int(st.item())


def _want(c, out, bias=False):
    if out == "int32":
        return torch.from_numpy(P.linear_i8(c["a"], c["w"], c["sizes"]).astype(np.int32))
    v = P.linear_i8(c["a"], c["w"], c["sizes"], c["col"], c["row"],
                    c["bias"] if bias else None)
    return torch.from_numpy(v).to(DT[out])


def _same(got, want):
    n = want.shape[0]
    bits = torch.int16 if want.element_size() == 2 else torch.int32
    g, w = got[:n].contiguous().view(bits), want.view(bits)
    if not torch.equal(g, w):
        bad = (g != w).nonzero()
        raise AssertionError("%d of %d differ, first at %s: got %s, want %s" % (
            len(bad), w.numel(), bad[0].tolist(), got[tuple(bad[0])], want[tuple(bad[0])]))


SHAPES = [  # sizes, N, K
    ((1,), 1, 1), ((1,), 8, 16), ((1,), 257, 100), ((1,), 512, 2048), ((2,), 130, 7168),
    ((3,), 1000, 33), ((7,), 64, 64), ((8,), 4096, 1040), ((9,), 96, 4000),
    ((16,), 129, 1024), ((17,), 255, 1025), ((33,), 640, 520), ((64,), 128, 128),
    ((65,), 300, 96), ((127,), 1001, 1992), ((128,), 256, 256), ((129,), 257, 130),
    ((197,), 1001, 1992), ((255,), 48, 640), ((256,), 1024, 512), ((300,), 1536, 1100),
    ((1100,), 520, 2064), ((2000,), 264, 72),
    ((3, 0, 5), 72, 96), ((0, 0, 4), 40, 200), ((1,) * 40, 100, 160),
    ((100, 1, 0, 31, 260), 200, 1030), ((0, 700, 45), 264, 1104),
    ((5, 0, 17, 130, 64, 1, 0, 300), 384, 2048), ((0, 0), 64, 64),
    # past the limits of small products
    ((9,), 14600, 40), ((12,), 11000, 300), ((16,), 8208, 1024), ((17,), 8200, 1025),
    ((33,), 4100, 520), ((64,), 2056, 128), ((65,), 2040, 96), ((128,), 1100, 256),
    ((129,), 1027, 130), ((255,), 1000, 640), ((300,), 600, 1), ((20, 1, 0, 44), 96, 32800),
    ((40,) * 8, 1001, 33), ((100, 1, 0, 31, 260), 1000, 1030), ((4,) * 40, 1001, 161)]


@pytest.mark.parametrize("sizes,N,K", SHAPES, ids=lambda v: str(v).replace(" ", "")[:40])
def test_types_and_sizes(ep, sizes, N, K):
    c = _case(sizes, N, K, seed=sum(sizes) + N + K)
    for out in ("int32", "bf16", "fp16", "fp32"):
        got, st = _run(ep, c, out)
        assert st == 0
        _same(got, _want(c, out))
    got, st = _run(ep, c, "bf16", bias=True)
    assert st == 0
    _same(got, _want(c, "bf16", bias=True))
    got, st = _run(ep, c, "int32", bias=True)           # accumulators: the bias is not read
    assert st == 0
    _same(got, _want(c, "int32"))


@pytest.mark.parametrize("sizes,N,K", [((2,), 200, 300), ((40,), 136, 1000),
                                       ((130, 3), 300, 2050), ((130, 3), 1100, 2050),
                                       ((600,), 520, 1500)],
                         ids=lambda v: str(v).replace(" ", ""))
def test_strides_images_and_rows_past_the_groups(ep, sizes, N, K):
    """Row images, padded strides of both operands, garbage past K, and a
    buffer with more rows than the groups: those rows are not written."""
    for kw in (dict(images=True), dict(a_pad=16, w_pad=48), dict(a_pad=4096, extra_rows=70)):
        c = _case(sizes, N, K, seed=N + K, **kw)
        for out in ("int32", "fp32", "bf16"):
            got, st = _run(ep, c, out)
            assert st == 0
            _same(got, _want(c, out))
            rest = got[sum(sizes):].contiguous().view(torch.uint8)
            assert (rest == 0xA5).all()


@pytest.mark.parametrize("rows", [1, 12, 40, 150, 411, 700])
def test_one_group_without_counts(ep, rows):
    c = _case((rows,), 320, 1300, seed=rows)
    for out in ("bf16", "int32"):
        got, st = _run(ep, c, out, group_rows=False, bias=out == "bf16")
        assert st == 0
        _same(got, _want(c, out, bias=out == "bf16"))


@pytest.mark.parametrize("rows,K", [(1, 65536), (9, 65536), (40, 20000), (90, 65536), (200, 65536)])
@pytest.mark.parametrize("code", [-128, 127])
def test_extreme_codes_stay_exact(ep, rows, K, code):
    """Every product 2^14 (or 127^2): sums far beyond 2^24 in one row."""
    c = _case((rows,), 24, K, seed=1, codes=(code, code + 1))
    got, st = _run(ep, c, "int32")
    assert st == 0 and (got == K * code * code).all()
    c["a"][0, ::3] = -code - 1 if code < 0 else -code       # cancel part of it
    c["dev"]["a"][:, :K] = torch.from_numpy(c["a"].view(np.uint8)).cuda()
    got, st = _run(ep, c, "int32")
    assert st == 0
    _same(got, _want(c, "int32"))


@pytest.mark.parametrize("G,rows", [(4096, 300), (500, 4000), (64, 64)])
def test_many_groups(ep, G, rows):
    rng = np.random.default_rng(G)
    sizes = rng.multinomial(rows, rng.dirichlet(np.full(G, 0.3)))
    c = _case(sizes.tolist(), 40, 80, seed=G)
    got, st = _run(ep, c, "fp32")
    assert st == 0
    _same(got, _want(c, "fp32"))


def test_device_errors(ep):
    for sizes, N in (((3, 2), 72), ((200, 300), 72), ((200, 300), 520)):
        c = _case(sizes, N, 96, seed=5)
        st = torch.zeros(1, dtype=torch.int32, device="cuda")
        c["dev"]["sizes"][0] += 1                            # more rows than a holds
        got, code = _run(ep, c, "fp32", st=st)
        assert code == ep.MOE_ERR_CAPACITY
        assert (got.view(torch.uint8) == 0xA5).all()
        c["dev"]["sizes"][0] = -4                            # read as 0
        st.zero_()
        got, code = _run(ep, c, "int32", st=st)
        assert code == ep.MOE_ERR_INVALID_ARG
        n = sizes[1]
        ref = c["a"][:n].astype(np.int64) @ c["w"][1].T.astype(np.int64)
        assert np.array_equal(got[:n].numpy(), ref)
        assert (got[n:].contiguous().view(torch.uint8) == 0xA5).all()


def test_streams_and_repeats(ep):
    """On a side stream, and twice: the same bits."""
    c = _case((70, 5, 300), 500, 1200, seed=3)
    side = torch.cuda.Stream()
    a, st = _run(ep, c, "fp16", stream=side)
    b, st2 = _run(ep, c, "fp16")
    assert st == st2 == 0
    _same(a, _want(c, "fp16"))
    _same(b, _want(c, "fp16"))


def test_non_finite_scales_and_overflow(ep):
    """Infinite and NaN scales go through to their row or column alone; a value
    beyond fp16's range becomes infinite."""
    c = _case((5,), 40, 64, seed=8)
    c["col"][0, 3], c["col"][0, 4], c["row"][2] = np.inf, np.nan, 1e30
    c["dev"]["col"].copy_(torch.from_numpy(c["col"]))
    c["dev"]["row"].copy_(torch.from_numpy(c["row"]))
    with np.errstate(all="ignore"):
        want = _want(c, "fp16")
    got, st = _run(ep, c, "fp16")
    assert st == 0
    nan = torch.isnan(want)
    assert torch.equal(torch.isnan(got), nan)
    assert torch.equal(got[~nan], want[~nan])


@pytest.mark.parametrize("bad", ["K", "short_w", "c_shape", "c_dtype", "a_dtype", "no_counts", "no_scale", "a_cols", "scale_short", "misaligned"])
def test_refusals(ep, bad):
    c = _case((4, 2), 24, 64, seed=2)
    d = c["dev"]
    y = torch.zeros((6, 24), device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    a, w, K, n, col, scale, bias = d["a"], d["w"], 64, d["sizes"], d["col"], d["scale"], None
    if bad == "K":
        K = 0
    elif bad == "short_w":
        w = w[:, :, :48].contiguous()
    elif bad == "c_shape":
        y = y[:5]
    elif bad == "c_dtype":
        y = y.double()
    elif bad == "a_dtype":
        a = a.to(torch.int16)
    elif bad == "no_counts":
        n = None
    elif bad == "no_scale":
        col = None
    elif bad == "a_cols":
        a = a.t()
    elif bad == "scale_short":
        scale = (d["row"][:5].contiguous(), 0, 4)
    elif bad == "misaligned":
        a = torch.zeros((6, 100), dtype=torch.uint8, device="cuda")[:, 4:68]
    with pytest.raises((ep.MoeError, ValueError, TypeError)):
        ep.moe_linear_i8(a, w, K, n, col, scale, bias, y, st)
    assert (y == 0).all()
