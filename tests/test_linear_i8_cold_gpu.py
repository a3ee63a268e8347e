"""The INT8 product on operands that arrive late and out of order: rows written just
before by a copy, weights fallen out of the cache, hundreds of times, every
accumulator against the exact product."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ep():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a CUDA device")
    import combine_moe_dispatch_layout_gb300 as ep
    return ep


def _exact(a, w, K):
    out = torch.empty((a.shape[0], w.shape[0]), dtype=torch.int32, device="cuda")
    for at in range(0, a.shape[0], 4096):       # products of codes: exact in float64
        out[at:at + 4096] = torch.round(
            a[at:at + 4096, :K].double() @ w[:, :K].double().t()).int()
    return out


@pytest.mark.parametrize("sizes,N,K,calls", [
    ([24576], 40, 4096, 600), ([36000], 40, 2000, 600), ([6000], 520, 4096, 300),
    ([700, 0, 2500, 130, 1000, 300], 500, 3000, 300), ([197], 1001, 2000, 300),
    ([600], 1000, 4096, 300), ([90] * 12, 700, 2100, 300)],
    ids=lambda v: str(v).replace(" ", "")[:30])
def test_rows_written_just_before(ep, sizes, N, K, calls):
    g = torch.Generator(device="cuda")
    g.manual_seed(sum(sizes) + N)
    wide = (K + 15) // 16 * 16
    rows, G = sum(sizes), len(sizes)
    src = [torch.randint(-128, 128, (rows, wide), generator=g, dtype=torch.int8, device="cuda")
           for _ in range(2)]
    w = torch.randint(-128, 128, (G, N, wide), generator=g, dtype=torch.int8, device="cuda")
    want = []
    for a in src:
        parts, at = [], 0
        for e, n in enumerate(sizes):
            parts.append(_exact(a[at:at + n], w[e], K))
            at += n
        want.append(torch.cat(parts))
    counts = torch.tensor(sizes, dtype=torch.int32, device="cuda") if G > 1 else None
    a = torch.zeros_like(src[0])
    c = torch.zeros((rows, N), dtype=torch.int32, device="cuda")
    flush = torch.zeros(200 << 20, dtype=torch.uint8, device="cuda")    # more than the cache
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    wrong = 0
    for i in range(calls):
        if i % 3 == 0:
            flush.add_(1)
        a.copy_(src[i % 2])
        c.fill_(-7)
        ep.moe_linear_i8(a, w, K, counts, None, None, None, c, st)
        wrong += int(not torch.equal(c, want[i % 2]))
    assert wrong == 0 and int(st.item()) == 0
