"""The operators together, as a user runs them (``pipeline.py``): an MoE layer
from logits to output on 8-bit weights, against the deep MoE on the same ids
(bit for bit) and against the plain forms; and one training step of a verbatim
pipeline, gradients of tokens and logits against float64."""
import numpy as np
import pytest
import torch

import plain_ops as P
import workloads as W

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pl():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a CUDA device")
    from combine_moe_dispatch_layout_gb300 import pipeline
    return pipeline


@pytest.mark.parametrize("R,epr,bs,k,H,I,dtype", [
    (1, 8, 1, 2, 128, 64, W.BF16),            # one decoded token
    (2, 4, 16, 2, 256, 96, W.FP16),           # a few rows per expert
    (2, 3, 40, 3, 320, 160, W.BF16),          # tens of rows per expert
    (4, 2, 300, 2, 512, 256, W.BF16)])        # hundreds
def test_serving_layer_is_the_deep_moe(pl, R, epr, bs, k, H, I, dtype):
    E, T = R * epr, R * bs
    w = W.Workload("serve", R=R, epr=epr, bs=bs, k=k, H=H, dtype=dtype, seed=31 + T)
    x = W.tokens(w).cuda()
    w1, ws1, w2, ws2 = (t.cuda() for t in W.moe_weights(E, H, I, seed=3))
    logits = torch.randn((T, E), generator=torch.Generator().manual_seed(T)).cuda()
    bias = (torch.arange(E, device="cuda") % 3 - 1) * 0.001
    routing = pl.Routing(T, E, k, "sigmoid", bias, scale=1.5)
    b = pl.ServeBuffers(R, bs, k, epr, H, I, dtype)
    pl.run_serve_moe(b, pl.Int8MoeWeights(w1, ws1, w2, ws2), routing, x, logits)
    torch.cuda.synchronize()
    assert b.status() == 0
    ids, wt = P.route(logits.double().cpu().numpy(), bias.double().cpu().numpy(), "sigmoid", k,
                      scale=1.5)
    np.testing.assert_array_equal(routing.topk_idx.cpu().numpy(), ids)
    np.testing.assert_allclose(routing.topk_weights.cpu().numpy(), wt, rtol=1e-5)
    d = pl.DeepMoeBuffers(R, bs, k, epr, H, I, dtype)
    pl.run_deep_moe(d, pl.DeepMoeWeights(w1, ws1, w2, ws2), x, routing.topk_idx,
                    routing.topk_weights)
    torch.cuda.synchronize()
    assert d.status() == 0
    assert torch.equal(b.out.view(torch.int16), d.out.view(torch.int16))


def test_serving_layer_in_a_cuda_graph(pl):
    """Captured once, replayed on new tokens and logits in the same buffers."""
    R, epr, bs, k, H, I = 2, 8, 8, 2, 256, 128
    T, E = R * bs, R * epr
    w1, ws1, w2, ws2 = (t.cuda() for t in W.moe_weights(E, H, I, seed=5))
    wts = pl.Int8MoeWeights(w1, ws1, w2, ws2)
    routing = pl.Routing(T, E, k)
    b = pl.ServeBuffers(R, bs, k, epr, H, I, W.BF16)
    x = torch.zeros((T, H), dtype=torch.bfloat16, device="cuda")
    logits = torch.zeros((T, E), device="cuda")
    side = torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        pl.run_serve_moe(b, wts, routing, x, logits)
        side.synchronize()
        with torch.cuda.graph(g, stream=side):
            pl.run_serve_moe(b, wts, routing, x, logits)
    for seed in (1, 2):
        gen = torch.Generator().manual_seed(seed)
        x.copy_(torch.randn((T, H), generator=gen))
        logits.copy_(torch.randn((T, E), generator=gen))
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        replayed = b.out.clone()
        pl.run_serve_moe(b, wts, routing, x, logits)
        torch.cuda.synchronize()
        assert b.status() == 0
        assert torch.equal(replayed.view(torch.int16), b.out.view(torch.int16))


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("renorm", [True, False])
def test_training_step(pl, score, renorm):
    """loss = <c, combine(tanh(dispatch(x)), weights(logits))>: gradients of x and
    of the logits against float64 on the same ids.  The fp16 rows between the
    stages (rows, outputs, row gradients) are rounded to 2^-11 relative each."""
    R, epr, bs, k, H = 2, 4, 24, 3, 64
    T, E = R * bs, R * epr
    w = W.Workload("train", R=R, epr=epr, bs=bs, k=k, H=H, dtype=W.FP16, quant=False, seed=77)
    x = W.tokens(w).cuda()
    gen = torch.Generator().manual_seed(8)
    logits = torch.randn((T, E), generator=gen).cuda()
    c = torch.randn((T, H), generator=gen).half().cuda()
    b = pl.PipelineBuffers(R, bs, k, epr, H, W.FP16, False)
    routing = pl.Routing(T, E, k, score, renormalise=renorm, scale=2.0)

    pl.run_route(b, routing, logits)
    pl.run_layout_notify(b, routing.topk_idx)
    pl.run_dispatch(b, x, routing.topk_idx)
    rows = b.recv.view(torch.float16).view(T * k, H)
    y = torch.tanh(rows.float()).half()
    pl.run_combine(b, y, routing.topk_idx, routing.topk_weights)

    d_y, d_w = torch.empty_like(y), torch.empty((T, k), device="cuda")
    pl.run_combine_backward(b, c, y, routing.topk_idx, routing.topk_weights, d_y, d_w)
    d_rows = (d_y.float() * (1 - y.float() ** 2)).half()
    d_x = torch.empty_like(x)
    pl.run_dispatch_backward(b, d_rows, routing.topk_idx, torch.ones((T, k), device="cuda"), d_x)
    d_logits = torch.empty_like(logits)
    pl.run_route_backward(b, routing, logits, d_w, d_logits)
    torch.cuda.synchronize()
    assert b.status() == 0

    l = logits.double().cpu().requires_grad_()
    xr = x.double().cpu().requires_grad_()
    ids = routing.topk_idx.long().cpu()
    s = torch.sigmoid(l) if score == "sigmoid" else torch.softmax(l, 1)
    wt = s.gather(1, ids)
    wt = 2.0 * (wt / wt.sum(1, keepdim=True) if renorm else wt)
    t = torch.tanh(xr)
    out = wt.sum(1, keepdim=True) * t        # every expert is the same tanh
    (c.double().cpu() * out).sum().backward()
    u = 2.0 ** -11
    ref = xr.grad
    # k row gradients of two rounded factors and one rounded product each, a sum
    mag = (c.double().cpu().abs() * wt.abs().sum(1, keepdim=True)).detach()
    assert ((d_x.double().cpu() - ref).abs() <= 6 * u * mag + 1e-6).all()
    # the weights' gradients: H products with outputs rounded to 2^-11
    err = (u * (c.double().cpu() * t.detach()).abs().sum(1, keepdim=True)).numpy()
    bound = 2.0 * err * k            # scale 2, k slots, |d weight / d logit| <= 1
    assert (np.abs(d_logits.double().cpu().numpy() - l.grad.numpy()) <= bound + 1e-6).all()
