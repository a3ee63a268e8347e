"""Plain float64 (numpy and torch) forms of the norm, its gradient, SwiGLU to e4m3 rows and
the e4m3 product, written from the definitions in ``include/moe_ep.h``, and e4m3
itself from its definition; shared by the tests of those operators.  They share
nothing with the CUDA code."""
import numpy as np
import torch

U32 = 2.0 ** -24                     # half a step of fp32, relative
HALF = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: U32}
TINY = 1e-12


def blocks(n):
    return (n + 127) // 128


def align32(n):
    return (n + 31) // 32 * 32


def f8_row_bytes(H):
    return align32(H) + align32(4 * blocks(H))


def e4m3_table():
    """The value of each of the 256 codes (sign, 4 exponent bits of bias 7, 3
    fraction bits, no infinities, all ones NaN)."""
    c = np.arange(256)
    s = np.where(c & 0x80, -1.0, 1.0)
    e, m = (c >> 3) & 15, c & 7
    v = np.where(e > 0, (1 + m / 8.0) * 2.0 ** (e - 7.0), m / 8.0 * 2.0 ** -6)
    return s * np.where((e == 15) & (m == 7), np.nan, v)


TABLE = e4m3_table()


def split_image(image, H):
    """uint8 [rows, f8_row_bytes(H)] -> code values float64 [rows, H], scales float64
    [rows, blocks], and the padding bytes."""
    raw = image.cpu().numpy()
    codes, rest = raw[:, :H], raw[:, align32(H):]
    nb = blocks(H)
    scales = rest[:, :4 * nb].copy().view(np.float32).astype(np.float64)
    pad = np.concatenate([raw[:, H:align32(H)], rest[:, 4 * nb:]], axis=1)
    return TABLE[codes], scales, pad


def check_image(image, y, rel):
    """An image of float64 rows y that the kernel knew within rel * |y|: every scale is
    max|block| / 448, every value within half an e4m3 step (2^-4 of it, at least 2^-10
    of the scale), the padding zero."""
    y = np.asarray(y, np.float64)
    rows, H = y.shape
    codes, scales, pad = split_image(image, H)
    assert not pad.any()
    full = np.zeros((rows, 128 * blocks(H)))
    full[:, :H] = np.abs(y)
    top = np.maximum(full.reshape(rows, -1, 128).max(axis=2), TINY)
    np.testing.assert_allclose(scales, top / 448.0, rtol=rel + 4 * U32, atol=0)
    sc = np.repeat(scales, 128, axis=1)[:, :H]
    # the scale's and the quotient's own errors (a few ulp) move a value as `rel` does
    tol = np.maximum(2.0 ** -4 * np.abs(y), 2.0 ** -10 * sc) * (1 + 2.0 ** -10)
    tol = tol + (rel + 16 * U32) * np.abs(y)
    bad = np.abs(codes * sc - y) > tol
    assert not bad.any(), (np.argwhere(bad)[:3], (codes * sc)[bad][:3], y[bad][:3])


def norm(x, residual, gamma, eps):
    """s, rstd and y in float64; x, residual: torch rows, s rounded to their type."""
    s = x.double()
    if residual is not None:
        s = (s + residual.double()).to(x.dtype).double()
    rstd = 1.0 / torch.sqrt((s * s).mean(1, keepdim=True) + eps)
    return s, rstd, s * rstd * gamma.double()


def norm_backward(d_out, s, gamma, eps, d_sum=None):
    """d_x and d_gamma in float64, by the chain rule on y = s (mean(s^2) + eps)^-1/2 gamma."""
    s, g = s.double(), d_out.double() * gamma.double()
    r = (s.pow(2).mean(1, keepdim=True) + eps) ** -0.5
    d = g * r - s * r ** 3 * (g * s).mean(1, keepdim=True)
    if d_sum is not None:
        d = d + d_sum.double()
    return d, (d_out.double() * s * r).sum(0)


def swiglu(h):
    h = h.double()
    I = h.shape[1] // 2
    gate, up = h[:, :I], h[:, I:]
    e = torch.exp(-gate.abs())
    return gate * torch.where(gate >= 0, torch.ones_like(e), e) / (1 + e) * up


def dequant(codes, scale, K):
    """float64 rows of e4m3 codes (uint8) with a scale per 128 of a row."""
    v = torch.from_numpy(TABLE)[codes.cpu().long()]
    return v[:, :K] * scale.double().cpu().repeat_interleave(128, 1)[:, :K]


def linear(a, a_scale, w, w_scale, K, sizes, bias=None):
    """c and the sum of the products' magnitudes, both float64, of uint8 codes a [rows,
    >= K] (scales [rows, blocks(K)]) and w [G, N, >= K] (scales [G, blocks(N),
    blocks(K)]); rows past the groups' total stay 0."""
    rows, (G, N) = a.shape[0], w.shape[:2]
    av = dequant(a, a_scale, K)
    c = torch.zeros((rows, N), dtype=torch.float64)
    mag = torch.zeros_like(c)
    at = 0
    for g, n in enumerate(sizes):
        if n:
            wv = dequant(w[g], w_scale[g].repeat_interleave(128, 0)[:N], K)
            c[at:at + n] = av[at:at + n] @ wv.t()
            mag[at:at + n] = av[at:at + n].abs() @ wv.abs().t()
            if bias is not None:
                c[at:at + n] += bias[g].double().cpu()
                mag[at:at + n] += bias[g].double().cpu().abs()
            at += n
    return c, mag


def linear_bound(c, mag, K, dtype):
    """How far a result may be off.  A block's 128 products are exact and are added in four
    steps, of 32 products and the sum so far: each term is cut at 2^-24 of the largest
    at worst, 33 of them four times (2^-16.9 of the magnitudes' sum at the very most, for
    one term that is the largest; 2^-19 where the magnitudes' sum is 4 of the largest, which
    the tests' rows are far above), and a step's sum is rounded.  The scales' product, the
    multiply-add of each block, the bias and the sums of K's parts are a rounding each."""
    return (2.0 ** -19 + (blocks(K) + 8) * U32) * mag + HALF[dtype] * c.abs() * (1 + 2.0 ** -8)
