"""The e4m3 product's forms under what can go wrong in each: pairs of SMs with tiles of 256,
128 and 64 channels, pairs that share K, SMs by themselves, and the kernel for few rows.  The
shapes are pinned to their forms, so that a change of the plan shows here."""
import ctypes

import pytest
import torch

import plain_f8 as P
import test_serve_f8_gpu as S
import workloads as W
from test_linear_f8_gpu import Problem
from test_linear_f8_plans import SMS, _ids
from test_linear_f8_types import _plan

pytestmark = pytest.mark.gpu

PLAIN = {(256, 2): [([3000], 800, 1000)], (128, 2): [([600], 2048, 1000)],
         (64, 2): [([129], 1500, 700)], (128, 4): [([130], 2328, 2591)],
         (64, 4): [([300], 1000, 2000)], (0, 0): [([8], 1000, 4100)]}
GROUPED = {(256, 2): [([700, 0, 1157, 900, 1], 2000, 500)],
           (128, 2): [([130, 126, 0, 256], 2000, 2600)],
           (64, 2): [([60, 2, 90], 1501, 1100)],
           (256, 1): [([3, 0, 40, 129, 7] * 9, 1000, 1200), ([40] * 40, 1032, 2992)],
           (0, 0): [([6, 0, 9] * 9, 512, 512)]}


def _cases(*tables):
    return [(form,) + s for t in tables for form, some in t.items() for s in some]


@pytest.fixture(scope="module")
def ep():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a CUDA device")
    import combine_moe_dispatch_layout_gb300 as ep
    assert torch.cuda.get_device_properties(0).multi_processor_count == SMS
    return ep


def _problem(ep, form, sizes, N, K, dtype=torch.float32, **more):
    p = Problem(ep, sizes, N, K, dtype, **more)
    code = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}[dtype]
    rows = sum(sizes) + more.get("extra", 0)
    lib = ctypes.CDLL(ep.LIB_PATH)
    assert _plan(lib, [rows] + [0] * (len(sizes) - 1), N, K, code) == form
    return p


@pytest.mark.parametrize("form,sizes,N,K", _cases(PLAIN, GROUPED), ids=_ids)
def test_codes_and_scales_that_are_no_numbers(ep, form, sizes, N, K):
    """NaN codes in a row and in a channel of one group, an infinite scale of a row and a NaN
    scale of a weight block: in their rows and columns alone, the rest bit for bit."""
    off = [sum(sizes[:g]) for g in range(len(sizes))]
    g = max(range(len(sizes)), key=lambda i: sizes[i])
    first, last = off[g], off[g] + sizes[g]
    clean = _problem(ep, form, sizes, N, K)
    clean.run()
    row, bad_row = first + sizes[g] // 2, first + sizes[g] // 3
    for k, col in ((1, N - 1), (K - 1, N // 2), (K // 2, 3)):
        p = _problem(ep, form, sizes, N, K)
        p.a[row, k] = 0x7F
        p.w[g, col, k] = 0xFF
        p.run()
        torch.cuda.synchronize()
        assert int(p.st.item()) == 0
        assert bool(p.c[row].isnan().all()) and bool(p.c[first:last, col].isnan().all())
        keep = torch.ones_like(p.c, dtype=torch.bool)
        keep[row] = False
        keep[first:last, col] = False
        assert torch.equal(p.c[keep], clean.c[keep])
    p = _problem(ep, form, sizes, N, K)
    kb, nb = P.blocks(K), P.blocks(N)
    at = P.align32(K) + 4 * (kb - 1)
    p.a[bad_row, at:at + 4].view(torch.float32)[0] = float("inf")
    p.w_scale[g, nb // 2, kb // 2] = float("nan")
    p.run()
    torch.cuda.synchronize()
    cols = slice(128 * (nb // 2), min(N, 128 * (nb // 2) + 128))
    assert bool((~p.c[bad_row].isfinite()).all()) and bool(p.c[first:last, cols].isnan().all())
    keep = torch.ones_like(p.c, dtype=torch.bool)
    keep[bad_row] = False
    keep[first:last, cols] = False
    assert torch.equal(p.c[keep], clean.c[keep])


@pytest.mark.parametrize("form,sizes,N,K", _cases(GROUPED), ids=_ids)
def test_bad_counts(ep, form, sizes, N, K):
    """More rows than the buffer: nothing is written; a negative count reads as 0; rows
    past the last group are left."""
    p = _problem(ep, form, sizes, N, K)
    p.group_rows[-1] += 1
    p.run()
    torch.cuda.synchronize()
    assert int(p.st.item()) == ep.MOE_ERR_CAPACITY
    assert bool((p.c.contiguous().view(torch.uint8) == 0xA5).all())
    p = _problem(ep, form, sizes, N, K)
    p.group_rows[-1] = -(1 << 31)
    p.run()
    torch.cuda.synchronize()
    assert int(p.st.item()) == ep.MOE_ERR_INVALID_ARG
    p.sizes = sizes[:-1] + [0]
    p.st.zero_()
    p.check()
    p = _problem(ep, form, sizes, N, K)
    p.group_rows.zero_()
    p.run()
    torch.cuda.synchronize()
    assert int(p.st.item()) == 0
    assert bool((p.c.contiguous().view(torch.uint8) == 0xA5).all())


@pytest.mark.parametrize("form,sizes,N,K", _cases(PLAIN, GROUPED), ids=_ids)
def test_the_same_bits_every_time(ep, form, sizes, N, K):
    """Also on another stream, and from a captured graph."""
    p = _problem(ep, form, sizes, N, K, bias=True)
    p.run()
    torch.cuda.synchronize()
    want = p.c.clone()
    side = torch.cuda.Stream()
    for i in range(20):
        p.c.zero_()
        side.wait_stream(torch.cuda.current_stream())
        p.run(side if i % 2 else None)
        torch.cuda.current_stream().wait_stream(side)
        assert torch.equal(p.c, want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        side.synchronize()
        with torch.cuda.graph(g, stream=side):
            p.run()
            p.run()
    for _ in range(5):
        p.c.zero_()
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(p.c, want)
    assert int(p.st.item()) == 0


@pytest.mark.parametrize("form,sizes,N,K", [
    ((256, 2), [3000], 800, 2992), ((256, 2), [700, 0, 2500, 130, 1000, 300], 500, 2992),
    ((128, 2), [600], 2048, 2000), ((64, 2), [129], 1500, 700),
    ((256, 1), [40] * 40, 1032, 2992), ((256, 1), [3, 0, 200, 129, 7] * 9, 1000, 2992),
    ((256, 1), [100, 0, 64, 1] * 40, 700, 1000)], ids=_ids)
def test_rows_written_just_before(ep, form, sizes, N, K):
    """Operands that arrive late and out of order: rows written just before by a copy,
    weights fallen out of the cache, again and again, the same bits each time."""
    p = [_problem(ep, form, sizes, N, K, torch.bfloat16, seed=s) for s in (0, 1)]
    want = []
    for q in p:
        q.w, q.w_scale = p[0].w, p[0].w_scale
        q.run()
        q.check()
        want.append(q.c.clone())
    flush = torch.zeros(200 << 20, dtype=torch.uint8, device="cuda")
    q, src = p[0], [p[0].a.clone(), p[1].a.clone()]
    wrong = 0
    for i in range(200):
        if i % 3 == 0:
            flush.add_(1)
        q.a.copy_(src[i % 2])
        q.c.zero_()
        q.run()
        wrong += int(not torch.equal(q.c, want[i % 2]))
    assert wrong == 0 and int(q.st.item()) == 0


def test_two_streams_at_once(ep):
    """Two products of different forms on two streams, call after call."""
    shapes = [((256, 1), [40] * 40, 1032, 2992), ((256, 2), [3000], 800, 1000),
              ((64, 4), [300], 1000, 2000), ((128, 2), [600], 2048, 1000)]
    for i in range(len(shapes)):
        pair = [_problem(ep, *shapes[j % len(shapes)]) for j in (i, i + 1)]
        want = []
        for p in pair:
            p.run()
            torch.cuda.synchronize()
            want.append(p.c.clone())
            p.c.zero_()
        streams = [torch.cuda.Stream() for _ in pair]
        torch.cuda.synchronize()
        for _ in range(40):
            for p, s in zip(pair, streams):
                p.run(s)
        torch.cuda.synchronize()
        for p, w in zip(pair, want):
            assert int(p.st.item()) == 0 and torch.equal(p.c, w)


@pytest.mark.parametrize("R,epr,bs,k,H,I,up,down", [
    (2, 20, 160, 4, 2048, 512, (256, 1), (256, 1)),      # tens of rows for many experts
    (1, 4, 2048, 2, 1024, 512, (256, 2), (256, 2)),      # a thousand for each of a few
    (2, 4, 32, 2, 7168, 256, (128, 2), (256, 1))],       # few rows of a few, wide
    ids=_ids)
def test_serving_layer(ep, R, epr, bs, k, H, I, up, down):
    """The whole layer where its products run by tiles."""
    from combine_moe_dispatch_layout_gb300 import pipeline as pl
    lib = ctypes.CDLL(ep.LIB_PATH)
    rows = [R * bs * k] + [0] * (R * epr - 1)
    assert (_plan(lib, rows, 2 * I, H, 0), _plan(lib, rows, H, I, 0)) == (up, down)
    S.test_serving_layer(pl, R, epr, bs, k, H, I, W.BF16)


@pytest.mark.parametrize("form,sizes,extra,N,K", [
    ((256, 2), [5, 0, 7, 1] * 8, 20000, 512, 1000), ((256, 1), [2, 0, 3] * 20, 5000, 1032, 1000),
    ((128, 2), [1, 2, 0, 1], 508, 2000, 2600)], ids=_ids)
def test_a_buffer_for_far_more_rows(ep, form, sizes, extra, N, K):
    """The form goes by the buffer's rows; the counts on the device say that there are few."""
    p = _problem(ep, form, sizes, N, K, bias=True, extra=extra)
    p.run()
    p.check()
