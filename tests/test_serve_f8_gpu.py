"""The norm and the e4m3 operators together, as a user runs them (``pipeline.py``): an MoE
layer from the residual stream to its output, every stage against its float64 form on what
the stage before gave; a training step of norm and verbatim pipeline, gradients against
float64; late inputs, other streams, captured graphs and two host threads."""
import threading

import numpy as np
import pytest
import torch

import plain_f8 as F
import plain_ops as P
import workloads as W

pytestmark = pytest.mark.gpu
EPS = 1e-6


@pytest.fixture(scope="module")
def pl():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a CUDA device")
    from combine_moe_dispatch_layout_gb300 import pipeline
    return pipeline


def _weights(E, H, I, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def codes(*shape):
        v = torch.randn(shape, generator=g, device="cuda") * 90
        return v.clamp(-448, 448).to(torch.float8_e4m3fn)

    def scales(rows, cols, k):
        s = torch.exp2(torch.randn((E, F.blocks(rows), F.blocks(cols)), generator=g,
                                   device="cuda"))
        return s / (90 * k ** 0.5)

    return codes(E, 2 * I, H), scales(2 * I, H, H), codes(E, H, I), scales(H, I, I)


class Layer:
    def __init__(self, pl, R, epr, bs, k, H, I, dtype, seed=0):
        self.pl, self.R, self.epr, self.bs, self.k, self.H, self.I = pl, R, epr, bs, k, H, I
        self.T, self.E = R * bs, R * epr
        self.w = _weights(self.E, H, I, seed + 1)
        self.wts = pl.Fp8MoeWeights(*self.w)
        self.routing = pl.Routing(self.T, self.E, k, "sigmoid", scale=1.5)
        self.b = pl.ServeF8Buffers(R, bs, k, epr, H, I, dtype)
        g = torch.Generator(device="cuda")
        g.manual_seed(seed + 2)
        self.g = g
        self.gamma = 1 + 0.2 * torch.randn(H, generator=g, device="cuda")
        self.x, self.res = (torch.zeros((self.T, H), dtype=self.b.torch_dtype, device="cuda")
                            for _ in range(2))
        self.logits = torch.zeros((self.T, self.E), device="cuda")
        self.src = [self.draw() for _ in range(2)]

    def draw(self):
        def rows():
            return torch.randn((self.T, self.H), generator=self.g,
                               device="cuda").to(self.b.torch_dtype)
        return rows() * 2, rows(), torch.randn((self.T, self.E), generator=self.g, device="cuda")

    def write(self, n):
        for to, src in zip((self.x, self.res, self.logits), self.src[n]):
            to.copy_(src)

    def run(self, stream=None):
        self.pl.run_norm_f8(self.b, self.x, self.res, self.gamma, EPS, stream)
        self.pl.run_serve_moe_f8(self.b, self.wts, self.routing, self.logits, stream)

    def results(self):
        torch.cuda.synchronize()
        assert self.b.status() == 0
        return [t.clone() for t in (self.b.sum, self.b.normed, self.b.images, self.b.out)]


def _same(a, b):
    return all(torch.equal(x.contiguous().view(torch.uint8), y.contiguous().view(torch.uint8))
               for x, y in zip(a, b))


@pytest.mark.parametrize("R,epr,bs,k,H,I,dtype", [
    (1, 8, 1, 2, 128, 64, W.BF16),             # one decoded token
    (2, 4, 16, 2, 256, 96, W.FP16),            # a few rows per expert
    (2, 3, 40, 3, 320, 160, W.BF16),           # tens of rows per expert
    (4, 2, 300, 2, 528, 272, W.BF16)])         # hundreds, odd blocks
def test_serving_layer(pl, R, epr, bs, k, H, I, dtype):
    L = Layer(pl, R, epr, bs, k, H, I, dtype)
    L.write(0)
    L.run()
    torch.cuda.synchronize()
    b, half = L.b, F.HALF[L.b.torch_dtype]
    assert b.status() == 0
    s, _, y = F.norm(L.x, L.res, L.gamma, EPS)
    assert torch.equal(b.sum.double(), s)
    assert bool(((b.normed.double() - y).abs() <= (half + 64 * F.U32) * y.abs() + 1e-7).all())
    F.check_image(b.images, y.cpu().numpy(), 64 * F.U32)
    ids, wt = P.route(L.logits.double().cpu().numpy(), None, "sigmoid", k, scale=1.5)
    np.testing.assert_array_equal(L.routing.topk_idx.cpu().numpy(), ids)
    # every pair's row is its token's image, bit for bit
    e = torch.from_numpy(ids).long().cuda()
    src = (torch.arange(L.T, device="cuda") // bs)[:, None]
    row = b.rank_recv_base[e // epr] + b.put_offset[e * R + src] + b.send_idx
    assert torch.equal(b.recv[row.reshape(-1)], b.images.repeat_interleave(k, 0))
    sizes = b.recv_per_expert.tolist()
    w1, s1, w2, s2 = L.w

    def product(image, K, w, sc, got):
        at, kb = F.align32(K), F.blocks(K)
        scale = image.view(torch.float32)[:, at // 4:at // 4 + kb]
        want, mag = F.linear(image, scale, w.view(torch.uint8), sc, K, sizes)
        bound = F.linear_bound(want, mag, K, got.dtype)
        assert bool(((got.double().cpu() - want).abs() <= bound + 1e-7).all())

    product(b.recv, H, w1, s1, b.h1)
    F.check_image(b.x2, F.swiglu(b.h1).cpu().numpy(), 2.0 ** -16)
    product(b.x2, I, w2, s2, b.y2)
    rows = b.y2.double()[row.reshape(-1)].view(L.T, k, H)
    gate = L.routing.topk_weights.double()[:, :, None]
    want = (rows * gate).sum(1)
    tol = half * (1 + half) * want.abs() + 2 * (k + 1) * F.U32 * (rows * gate).abs().sum(1)
    assert bool(((b.out.double() - want).abs() <= tol + 1e-7).all())
    np.testing.assert_allclose(L.routing.topk_weights.cpu().numpy(), wt, rtol=1e-5)


def test_late_inputs_other_streams_and_graphs(pl):
    """Inputs that a copy writes just before, calls on a side stream while the current one
    is another, one captured graph replayed on new inputs, and two graphs at once."""
    L = Layer(pl, 2, 8, 40, 2, 512, 256, W.BF16)
    want = []
    for n in range(2):
        L.write(n)
        torch.cuda.synchronize()
        L.run()
        want.append(L.results())
    assert not _same(want[0], want[1])
    for i in range(30):
        L.write(i % 2)
        L.run()
        if i % 7 == 0:
            assert _same(L.results(), want[i % 2])
    side = torch.cuda.Stream()
    for i in range(6):
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            L.write(i % 2)
        L.run(side)
        torch.cuda.current_stream().wait_stream(side)
        assert _same(L.results(), want[i % 2])
    M = Layer(pl, 2, 8, 40, 2, 512, 256, W.BF16, seed=50)
    graphs = []
    for X in (L, M):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.stream(side):
            X.run()
            side.synchronize()
            with torch.cuda.graph(g, stream=side):
                X.run()
        graphs.append(g)
    other = []
    for n in range(2):
        M.write(n)
        torch.cuda.synchronize()
        M.run()
        other.append(M.results())
    second = torch.cuda.Stream()
    for i in range(8):
        L.write(i % 2)
        M.write(1 - i % 2)
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            graphs[0].replay()
        with torch.cuda.stream(second):
            graphs[1].replay()
        assert _same(L.results(), want[i % 2]) and _same(M.results(), other[1 - i % 2])


def test_two_host_threads(pl):
    """Two threads, each with its buffers and its stream."""
    layers = [Layer(pl, 2, 4, n, 2, 256, 128, W.FP16, seed=n) for n in (5, 60)]
    want = []
    for L in layers:
        L.write(0)
        torch.cuda.synchronize()
        L.run()
        want.append(L.results())
    errors = []

    def work(L, ref):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(60):
                    L.run()
                torch.cuda.current_stream().synchronize()
            if not _same([L.b.sum, L.b.normed, L.b.images, L.b.out], ref):
                errors.append("differs")
        except Exception as e:        # reported by the main thread
            errors.append(repr(e))

    threads = [threading.Thread(target=work, args=a) for a in zip(layers, want)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors


def test_training_step(pl):
    """loss = <c, combine(tanh(dispatch(norm(x + r))), weights)> + <c2, x + r>: gradients of
    the stream and of the norm's weights against float64.  What comes between the stages is
    rounded to fp16 (2^-11) and counted as the rows' gradient's own error."""
    import combine_moe_dispatch_layout_gb300 as ep
    R, epr, bs, k, H = 2, 4, 24, 3, 128
    T, E = R * bs, R * epr
    g = torch.Generator().manual_seed(4)
    x, r, c, c2 = (torch.randn((T, H), generator=g).half().cuda() for _ in range(4))
    gamma = (1 + 0.2 * torch.randn(H, generator=g)).cuda()
    logits = torch.randn((T, E), generator=g).cuda()
    b = pl.PipelineBuffers(R, bs, k, epr, H, W.FP16, False)
    routing = pl.Routing(T, E, k)
    s, normed, rstd = torch.empty_like(x), torch.empty_like(x), torch.empty(T, device="cuda")
    ep.moe_rms_norm(x, r, gamma, EPS, s, normed, None, rstd, b.dev_status)
    pl.run_route(b, routing, logits)
    pl.run_layout_notify(b, routing.topk_idx)
    pl.run_dispatch(b, normed, routing.topk_idx)
    y = torch.tanh(b.recv.view(torch.float16).view(T * k, H).float()).half()
    pl.run_combine(b, y, routing.topk_idx, routing.topk_weights)
    d_y, d_w = torch.empty_like(y), torch.empty((T, k), device="cuda")
    pl.run_combine_backward(b, c, y, routing.topk_idx, routing.topk_weights, d_y, d_w)
    d_rows = (d_y.float() * (1 - y.float() ** 2)).half()
    d_n, d_x = torch.empty_like(x), torch.empty_like(x)
    pl.run_dispatch_backward(b, d_rows, routing.topk_idx, torch.ones((T, k), device="cuda"), d_n)
    d_gamma = torch.empty(H, device="cuda")
    ws = torch.empty(ep.rms_norm_backward_workspace_bytes(T, H), dtype=torch.uint8, device="cuda")
    ep.moe_rms_norm_backward(d_n, s, gamma, rstd, c2, d_x, d_gamma, ws, b.dev_status)
    torch.cuda.synchronize()
    assert b.status() == 0

    sr = s.double().cpu().requires_grad_()
    gr = gamma.double().cpu().requires_grad_()
    wt = routing.topk_weights.double().cpu()
    n = sr * (sr.pow(2).mean(1, keepdim=True) + EPS) ** -0.5 * gr
    out = wt.sum(1, keepdim=True) * torch.tanh(n)
    cd = c.double().cpu()
    ((cd * out).sum() + (c2.double().cpu() * sr).sum()).backward()
    u = 2.0 ** -11
    # the normed rows are rounded (tanh's slope changes by as much), then as in the pipeline's
    # own training step 6 roundings of the rows' gradient
    e = (6 * u + 2 * u * n.detach().abs()) * (cd.abs() * wt.sum(1, keepdim=True)) + 1e-6
    rs = rstd.double().cpu()[:, None]
    ge, xh = gr.detach().abs() * e, (sr.detach() * rs).abs()
    tol = rs * (ge + xh * (ge * xh).mean(1, keepdim=True)) + 2 * u * sr.grad.abs()
    assert bool(((d_x.double().cpu() - sr.grad).abs() <= tol).all())
    assert bool(((d_gamma.double().cpu() - gr.grad).abs() <= (e * xh).sum(0) + 1e-6).all())
