"""Every operator as the first thing that a host thread does: a thread has no CUDA
context of its own until a call makes one current."""
import threading

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ep():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a CUDA device")
    import combine_moe_dispatch_layout_gb300 as ep
    return ep


def _calls(ep):
    """name -> (call, outputs)"""
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    x = torch.randn((300, 64), device="cuda")
    ids = torch.zeros((300, 4), dtype=torch.int32, device="cuda")
    w = torch.zeros((300, 4), device="cuda")
    d = torch.zeros((300, 64), device="cuda")
    a = torch.randint(-128, 128, (300, 512), dtype=torch.int8, device="cuda")
    wt = torch.randint(-128, 128, (1, 1000, 512), dtype=torch.int8, device="cuda")
    c = torch.zeros((300, 1000), dtype=torch.int32, device="cuda")
    one = torch.zeros((1, 1000), dtype=torch.int32, device="cuda")
    shape = ep.make_shape(1, 300, 4, 64, 256, torch.bfloat16)
    idx = torch.rand((300, 64), device="cuda").topk(4, dim=1).indices.int().contiguous()
    key = idx.reshape(-1).long()
    row = torch.empty_like(key)
    row[key.sort(stable=True).indices] = torch.arange(1200, device="cuda")
    count = torch.bincount(key, minlength=64)
    start = count.cumsum(0) - count
    send, put = (row - start[key]).int(), start.int()
    base = torch.tensor([0, 1200], device="cuda")
    g = torch.randn((300, 256), device="cuda").bfloat16()
    y = torch.randn((1200, 256), device="cuda").bfloat16()
    d_y, d_w = torch.zeros_like(y), torch.zeros((300, 4), device="cuda")
    ep.moe_route(x, None, "softmax", 4, ids, w, st)
    keep = ids.clone()
    gates = w.clone()
    return {
        "linear_i8": (lambda s: ep.moe_linear_i8(a, wt, 512, None, None, None, None, c, st,
                                                 stream=s), [c]),
        "linear_i8, one row": (lambda s: ep.moe_linear_i8(a[:1], wt, 512, None, None, None, None,
                                                          one, st, stream=s), [one]),
        "route": (lambda s: ep.moe_route(x, None, "softmax", 4, ids, w, st, stream=s), [ids, w]),
        "route_backward": (lambda s: ep.moe_route_backward(x, keep, gates, "softmax", d, st,
                                                           stream=s), [d]),
        "combine_backward": (lambda s: ep.moe_combine_backward(shape, g, y, idx, gates, send, put,
                                                               base, d_y, d_w, st, stream=s),
                             [d_y, d_w]),
    }, st


@pytest.mark.parametrize("name", ["linear_i8", "linear_i8, one row", "route", "route_backward",
                                  "combine_backward"])
def test_first_call_of_a_host_thread(ep, name):
    calls, st = _calls(ep)
    call, outs = calls[name]
    call(torch.cuda.current_stream())              # what the process looks up once is known
    torch.cuda.synchronize()
    want = [t.clone() for t in outs]
    for t in outs:
        t.zero_()
    stream = torch.cuda.Stream()
    torch.cuda.synchronize()
    errors = []

    def work():
        try:
            call(stream)
        except Exception as e:
            errors.append(repr(e))

    t = threading.Thread(target=work)
    t.start()
    t.join()
    torch.cuda.synchronize()
    assert not errors, errors
    assert int(st.item()) == 0
    for a, b in zip(outs, want):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
