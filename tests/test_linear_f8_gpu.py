"""The e4m3 product against float64: every kernel and tile width it chooses, groups empty and
uneven, odd sizes and strides, every output type (bounds: plain_f8.linear_bound)."""
import numpy as np
import pytest
import torch

import plain_f8 as P

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ep():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a CUDA device")
    import combine_moe_dispatch_layout_gb300 as ep
    return ep


def _codes(shape, g):
    """e4m3 codes of normal values (about +-300 at most), as uint8."""
    v = torch.randn(shape, generator=g, device="cuda") * 90
    return v.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)


class Problem:
    """Operands with NaN codes in every byte that must not count: past K in the rows of a
    (its row images hold scales there) and, past the next multiple of 16, of w."""

    def __init__(self, ep, sizes, N, K, dtype=torch.float32, bias=False, images=True, extra=0,
                 w_gap=0, seed=0):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed + sum(sizes) + N + K)
        self.ep, self.sizes, self.N, self.K, self.dtype = ep, sizes, N, K, dtype
        G, rows = len(sizes), sum(sizes) + extra
        kb, nb = P.blocks(K), P.blocks(N)
        codes = _codes((rows, K), g)
        scale = torch.exp2(torch.randn((rows, kb), generator=g, device="cuda"))
        if images:
            size = ep.f8_row_bytes(K)
            self.a = torch.full((rows, size), 0x7F, dtype=torch.uint8, device="cuda")
            at = P.align32(K)
            self.a[:, at:at + 4 * kb] = scale.view(torch.uint8).view(rows, 4 * kb)
            self.a_scale = (self.a, at, size)
        else:                      # codes alone; scales 4 bytes off every 16, rows apart
            self.a = torch.full((rows, (K + 15) // 16 * 16 + 16), 0x7F, dtype=torch.uint8,
                                device="cuda")
            pitch = kb + 2
            raw = torch.full((rows * pitch + 1,), float("nan"), device="cuda")
            raw[1:].view(rows, pitch)[:, :kb] = scale
            self.a_scale = (raw, 4, 4 * pitch)
        self.a[:, :K] = codes
        wide = (K + 15) // 16 * 16
        self.w = torch.full((G, N, wide + w_gap), 0x7F, dtype=torch.uint8, device="cuda")
        self.w[:, :, :K] = _codes((G, N, K), g)
        self.w_scale = torch.exp2(torch.randn((G, nb, kb), generator=g, device="cuda"))
        self.w_scale *= 1e-5
        self.bias = torch.randn((G, N), generator=g, device="cuda") if bias else None
        self.group_rows = torch.tensor(sizes, dtype=torch.int32, device="cuda")
        self.scale = scale
        item = torch.empty((), dtype=dtype).element_size()
        raw = torch.empty((rows * N + 2 * N + 64,), dtype=dtype, device="cuda")
        raw.view(torch.uint8).fill_(0xA5)
        at = -(-N * item // 16) * 16 // item         # c starts on 16 bytes
        self.c = raw[at:at + rows * N].view(rows, N)
        self.margins = [raw[:at], raw[at + rows * N:]]
        self.st = torch.zeros(1, dtype=torch.int32, device="cuda")

    def run(self, stream=None):
        grouped = self.group_rows if len(self.sizes) > 1 or sum(self.sizes) < len(self.c) else None
        self.ep.moe_linear_f8(self.a, self.w, self.K, grouped, self.w_scale, self.a_scale,
                              self.bias, self.c, self.st, stream)

    def check(self):
        torch.cuda.synchronize()
        assert int(self.st.item()) == 0
        for m in self.margins:
            assert bool((m.contiguous().view(torch.uint8) == 0xA5).all())
        want, mag = P.linear(self.a, self.scale, self.w, self.w_scale, self.K, self.sizes,
                             self.bias)
        n = sum(self.sizes)
        err = (self.c[:n].double().cpu() - want[:n]).abs()
        bound = P.linear_bound(want[:n], mag[:n], self.K, self.dtype)
        bad = ~(err <= bound)
        assert not bool(bad.any()), (bad.nonzero()[:3], err[bad][:3], bound[bad][:3])
        rest = self.c[n:].contiguous().view(torch.uint8)
        assert bool((rest == 0xA5).all())


# plain products: one token, few rows, small products, narrow and wide tiles, odd everything
PLAIN = [(1, 1, 1), (1, 64, 128), (1, 500, 300), (3, 33, 1000), (8, 512, 4096), (9, 100, 257),
         (16, 1000, 2000), (17, 4096, 512), (33, 300, 130), (127, 64, 640), (128, 128, 128),
         (129, 130, 255), (197, 1001, 1992), (256, 256, 384), (257, 513, 1024), (300, 8192, 128),
         (700, 1536, 1664), (1024, 2048, 512), (1100, 2999, 700), (5000, 5000, 96)]


@pytest.mark.parametrize("rows,N,K", PLAIN)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
def test_plain(ep, rows, N, K, dtype):
    p = Problem(ep, [rows], N, K, dtype, bias=rows % 2 == 1, images=K % 3 != 1, w_gap=16 * (N % 3))
    p.run()
    p.check()


@pytest.mark.parametrize("sizes", [
    [0, 0, 5, 0], [1] * 40, [3, 0, 9, 1, 0, 30], [7] * 33, [16, 0, 17, 8, 9, 120],
    [128, 1, 0, 127, 129], [256, 300, 0, 5, 511, 512, 513], [0, 2000, 0, 3], [40] * 64,
    list(range(60))], ids=lambda v: "-".join(map(str, v))[:24])
@pytest.mark.parametrize("N,K,dtype", [(260, 400, torch.float32), (1024, 256, torch.bfloat16),
                                       (999, 1032, torch.float16)])
def test_groups(ep, sizes, N, K, dtype):
    p = Problem(ep, sizes, N, K, dtype, bias=True, extra=9, images=N % 2 == 0)
    p.run()
    p.check()


@pytest.mark.parametrize("rows,N,K", [(1, 256, 512), (200, 600, 512)])
def test_one_group_of_fewer_rows_than_the_buffer(ep, rows, N, K):
    p = Problem(ep, [rows], N, K, extra=70)
    p.run()
    p.check()


@pytest.mark.parametrize("sizes,K", [([4], 600), ([300], 600), ([2, 3, 1], 600), ([150, 90], 600)])
def test_codes_and_scales_that_are_no_numbers(ep, sizes, K):
    """A NaN code of a row or of a channel, an infinite scale of a row, a NaN scale of a
    weight block: in their rows and columns alone."""
    N = 300
    p = Problem(ep, sizes, N, K)
    clean = Problem(ep, sizes, N, K)
    p.a[1, 5] = 0x7F
    p.w[0, 7, 130] = 0xFF
    clean.run()
    p.run()
    torch.cuda.synchronize()
    first = sizes[0]
    assert bool(p.c[1].isnan().all()) and bool(p.c[:first, 7].isnan().all())
    keep = torch.ones_like(p.c, dtype=torch.bool)
    keep[1] = False
    keep[:first, 7] = False
    assert torch.equal(p.c[keep], clean.c[keep])
    p = Problem(ep, sizes, N, K)
    at = P.align32(K)
    p.a[0, at:at + 4].view(torch.float32)[0] = float("inf")
    p.w_scale[0, 1, 2] = float("nan")
    p.run()
    torch.cuda.synchronize()
    assert bool((~p.c[0].isfinite()).all()) and bool(p.c[:first, 128:256].isnan().all())
    keep = torch.ones_like(p.c, dtype=torch.bool)
    keep[0] = False
    keep[:first, 128:256] = False
    assert torch.equal(p.c[keep], clean.c[keep])


@pytest.mark.parametrize("sizes", [[4, 5], [300, 300]])
def test_bad_counts(ep, sizes):
    """More rows than the buffer: nothing is written; a negative count reads as 0."""
    p = Problem(ep, sizes, 128, 256)
    p.group_rows[1] += 50
    p.run()
    torch.cuda.synchronize()
    assert int(p.st.item()) == ep.MOE_ERR_CAPACITY
    assert bool((p.c.contiguous().view(torch.uint8) == 0xA5).all())
    p = Problem(ep, sizes, 128, 256)
    p.group_rows[1] = -3
    p.run()
    torch.cuda.synchronize()
    assert int(p.st.item()) == ep.MOE_ERR_INVALID_ARG
    p.sizes = [sizes[0], 0]
    p.st.zero_()
    p.check()


# sizes whose K two pairs of SMs share: whole tiles, a tile that ends in either half of either
# SM's rows, groups of fewer rows than the buffer (and clusters without a tile), uneven parts
@pytest.mark.parametrize("rows,extra,N,K", [
    (256, 0, 1024, 2048), (30, 226, 1000, 3000), (70, 0, 1500, 3500), (130, 0, 4096, 4000),
    (200, 312, 1032, 2600), (17, 1, 4600, 4500), (321, 0, 72, 16000), (512, 0, 2304, 7168)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_parts_of_k(ep, rows, extra, N, K, dtype):
    for bias, images in ((False, True), (True, False)):
        p = Problem(ep, [rows], N, K, dtype, bias=bias, images=images, extra=extra)
        p.run()
        p.check()


def test_parts_of_k_and_bad_counts(ep):
    for rows, N, K in ((300, 1000, 2000), (40, 4096, 3500)):
        p = Problem(ep, [rows], N, K, extra=20)
        for count, status in ((rows + 21, ep.MOE_ERR_CAPACITY), (-1, ep.MOE_ERR_INVALID_ARG),
                              (0, 0)):
            p.group_rows[0] = count
            p.st.zero_()
            p.run()
            torch.cuda.synchronize()
            assert int(p.st.item()) == status
            assert bool((p.c.contiguous().view(torch.uint8) == 0xA5).all())
        p.group_rows[0] = rows
        p.st.zero_()
        p.run()
        p.check()


def test_parts_of_k_and_codes_that_are_no_numbers(ep):
    """In either part, of either half of the rows."""
    rows, N, K = 256, 1024, 2048
    for row, col, k in ((3, 7, 5), (100, 600, 2000), (200, 1023, 1023), (255, 64, 1024)):
        p, clean = Problem(ep, [rows], N, K), Problem(ep, [rows], N, K)
        p.a[row, k] = 0x7F
        p.w[0, col, k] = 0xFF
        clean.run()
        p.run()
        torch.cuda.synchronize()
        assert bool(p.c[row].isnan().all()) and bool(p.c[:, col].isnan().all())
        keep = torch.ones_like(p.c, dtype=torch.bool)
        keep[row] = False
        keep[:, col] = False
        assert torch.equal(p.c[keep], clean.c[keep])


def test_the_same_bits_every_time(ep):
    for sizes, N, K in (([1], 4096, 7168), ([3] * 30, 512, 2048), ([500], 1000, 4096),
                        ([90, 300, 7], 700, 1500)):
        p = Problem(ep, sizes, N, K, bias=True)
        p.run()
        torch.cuda.synchronize()
        want = p.c.clone()
        for _ in range(20):
            p.c.zero_()
            p.run()
        torch.cuda.synchronize()
        assert torch.equal(p.c, want)


def test_far_weights(ep):
    """Weights past 2^32 bytes: the last of 200 experts of 4096 x 7168, by both kernels."""
    G, N, K = 200, 4096, 7168
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    w = torch.zeros((G, N, K), dtype=torch.uint8, device="cuda")
    w[G - 1] = _codes((N, K), g)
    w_scale = torch.ones((G, P.blocks(N), P.blocks(K)), device="cuda") * 1e-5
    for rows in (3, 40 * G):
        size = ep.f8_row_bytes(K)
        a = torch.zeros((rows, size), dtype=torch.uint8, device="cuda")
        few = min(rows, 40)
        a[-few:, :K] = _codes((few, K), g)
        at = P.align32(K)
        a.view(torch.float32)[:, at // 4:at // 4 + P.blocks(K)] = 1.0
        counts = torch.zeros(G, dtype=torch.int32, device="cuda")
        counts[0], counts[G - 1] = rows - few, few
        c = torch.empty((rows, N), dtype=torch.float32, device="cuda")
        st = torch.zeros(1, dtype=torch.int32, device="cuda")
        ep.moe_linear_f8(a, w, K, counts, w_scale, (a, at, size), None, c, st)
        assert int(st.item()) == 0
        ones = torch.ones((few, P.blocks(K)))
        want, mag = P.linear(a[-few:, :], ones, w[G - 1:], w_scale[G - 1:], K, [few])
        err = (c[-few:].double().cpu() - want).abs()
        assert bool((err <= P.linear_bound(want, mag, K, torch.float32)).all())
        assert bool((c[:-few] == 0).all())


@pytest.mark.parametrize("sizes,N,K,calls", [
    ([1], 4096, 4096, 200), ([5, 0, 3, 8], 512, 4096, 200), ([600], 1000, 4096, 200),
    ([24576], 64, 2048, 200), ([700, 0, 2500, 130, 1000, 300], 500, 2992, 200),
    ([197], 1001, 1992, 200), ([90] * 12, 700, 2100, 200), ([100], 4096, 4096, 200)],
    ids=lambda v: str(v).replace(" ", "")[:30])
def test_rows_written_just_before(ep, sizes, N, K, calls):
    """Operands that arrive late and out of order: rows written just before by a copy,
    weights fallen out of the cache, again and again, the same bits each time."""
    p = [Problem(ep, sizes, N, K, torch.bfloat16, seed=s) for s in (0, 1)]
    a, w_scale = torch.zeros_like(p[0].a), p[0].w_scale
    want = []
    for q in p:
        q.w, q.w_scale, q.bias = p[0].w, w_scale, None
        q.run()
        q.check()
        want.append(q.c.clone())
    flush = torch.zeros(200 << 20, dtype=torch.uint8, device="cuda")
    q = p[0]
    src = [p[0].a.clone(), p[1].a.clone()]
    q.a, q.a_scale = a, (a, q.a_scale[1], q.a_scale[2])
    wrong = 0
    for i in range(calls):
        if i % 3 == 0:
            flush.add_(1)
        a.copy_(src[i % 2])
        q.c.zero_()
        q.run()
        wrong += int(not torch.equal(q.c, want[i % 2]))
    assert wrong == 0 and int(q.st.item()) == 0
