"""Routing, the gradients and the INT8 product behind what other streams and captured
graphs do, and between guard regions on both sides of everything they write."""
import numpy as np
import pytest
import torch

import plain_ops as P

pytestmark = pytest.mark.gpu
GUARD = 256            # bytes


@pytest.fixture(scope="module")
def ep():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a CUDA device")
    import combine_moe_dispatch_layout_gb300 as ep
    return ep


class Out:
    """An output of `shape` between two guard regions, all bytes 0xA5."""

    def __init__(self, shape, dtype):
        n = int(np.prod(shape)) * torch.empty((), dtype=dtype).element_size()
        self.raw = torch.full((n + 2 * GUARD,), 0xA5, dtype=torch.uint8, device="cuda")
        self.t = self.raw[GUARD:GUARD + n].view(dtype).view(shape)

    def check(self):
        assert (self.raw[:GUARD] == 0xA5).all() and (self.raw[-GUARD:] == 0xA5).all()


def _plan(idx, R, bs, k, epr):
    key = idx.reshape(-1).astype(np.int64) * R + np.repeat(np.arange(idx.shape[0]) // bs, k)
    order = np.argsort(key, kind="stable")
    row = np.empty_like(order)
    row[order] = np.arange(len(order))
    count = np.bincount(key, minlength=R * epr * R)
    start = np.cumsum(count) - count
    base = np.concatenate([start[::epr * R], [len(order)]])
    put = start - np.repeat(base[:R], epr * R)
    return [torch.from_numpy(v).cuda() for v in
            ((row - start[key]).astype(np.int32), put.astype(np.int32), base.astype(np.int64))]


class Layer:
    """The four operators on inputs `x` (logits), `a` (codes), `g` (gradient rows), which
    `write(n)` fills, and what they give, each from its inputs alone."""

    def __init__(self, ep, T, E, H, K, N, k=5):
        self.ep, self.T, self.E, self.H, self.K, self.N, self.k = ep, T, E, H, K, N, k
        rng = np.random.default_rng(T + E + H)
        gen = torch.Generator(device="cuda")
        gen.manual_seed(T)
        self.src = [(torch.randn((T, E), generator=gen, device="cuda"),
                     torch.randint(-128, 128, (T, K), generator=gen, dtype=torch.int8,
                                   device="cuda"),
                     torch.randn((T, H), generator=gen, device="cuda").half())
                    for _ in range(2)]
        self.x, self.a, self.g = (torch.zeros_like(t) for t in self.src[0])
        self.w = torch.randint(-128, 128, (1, N, K), generator=gen, dtype=torch.int8,
                               device="cuda")
        self.idx = np.stack([rng.permutation(E)[:k] for _ in range(T)]).astype(np.int32)
        self.plan = _plan(self.idx, 1, T, k, E)
        self.ids_in = torch.from_numpy(self.idx).cuda()
        self.gates = torch.rand((T, k), generator=gen, device="cuda")
        self.y = torch.randn((T * k, H), generator=gen, device="cuda").half()
        self.shape = ep.make_shape(1, T, k, E, H, torch.float16)
        self.st = torch.zeros(1, dtype=torch.int32, device="cuda")
        f = torch.float32
        self.outs = dict(ids=Out((T, k), torch.int32), wt=Out((T, k), f), d_l=Out((T, E), f),
                         d_y=Out((T * k, H), torch.float16), d_w=Out((T, k), f),
                         c=Out((T, N), torch.int32), one=Out((min(T, 2), N), torch.int32))

    def write(self, n):
        for to, src in zip((self.x, self.a, self.g), self.src[n]):
            to.copy_(src)

    def run(self):
        ep, o, st = self.ep, {n: v.t for n, v in self.outs.items()}, self.st
        ep.moe_route(self.x, None, "sigmoid", self.k, o["ids"], o["wt"], st)
        ep.moe_route_backward(self.x, self.ids_in, self.gates, "softmax", o["d_l"], st,
                              renormalise=False)
        ep.moe_combine_backward(self.shape, self.g, self.y, self.ids_in, self.gates, *self.plan,
                                o["d_y"], o["d_w"], st)
        ep.moe_linear_i8(self.a, self.w, self.K, None, None, None, None, o["c"], st)
        ep.moe_linear_i8(self.a[:2], self.w, self.K, None, None, None, None, o["one"], st)

    def take(self):
        torch.cuda.synchronize()
        assert int(self.st.item()) == 0
        for v in self.outs.values():
            v.check()
        return {n: v.t.clone() for n, v in self.outs.items()}

    def alone(self):
        """What each of the two inputs gives, with everything waited for."""
        want = []
        for n in range(2):
            self.write(n)
            torch.cuda.synchronize()
            self.run()
            want.append(self.take())
        return want


def _same(got, want):
    for n in want:
        a, b = (t.contiguous().view(torch.uint8) for t in (got[n], want[n]))
        assert torch.equal(a, b), n


SIZES = [(700, 64, 1000, 512, 300), (37, 33, 8, 48, 1), (1, 8, 64, 16, 7), (130, 1100, 2056, 80, 520),
         (515, 256, 256, 2000, 1001)]


@pytest.mark.parametrize("size", SIZES, ids=str)
def test_nothing_is_written_outside_the_outputs(ep, size):
    layer = Layer(ep, *size)
    want = layer.alone()                            # checks the guards
    l = layer.src[1][0].double().cpu().numpy()
    ids, w = P.route(l, None, "sigmoid", layer.k)
    assert np.array_equal(want[1]["ids"].cpu().numpy(), ids)
    np.testing.assert_allclose(want[1]["wt"].cpu().numpy(), w, rtol=1e-5)
    acc = layer.src[1][1].double() @ layer.w[0].double().t()
    assert torch.equal(want[1]["c"].double(), acc)
    assert torch.equal(want[1]["one"].double(), acc[:2])
    g = layer.src[1][2].double()
    row = torch.from_numpy(np.argsort(np.argsort(layer.idx.reshape(-1), kind="stable"),
                                      kind="stable")).cuda()
    dots = (layer.y.double()[row].view(-1, layer.k, layer.H) * g[:, None]).sum(2)
    torch.testing.assert_close(want[1]["d_w"].double(), dots, rtol=1e-5,
                               atol=1e-5 * layer.H ** 0.5)


@pytest.mark.parametrize("size", SIZES[:1] + SIZES[3:], ids=str)
def test_inputs_that_another_stream_writes_late(ep, size):
    """The consumer's stream has work of its own right before it waits for the event
    of the stream that writes the inputs, long after the calls were made."""
    layer = Layer(ep, *size)
    want = layer.alone()
    other, mine = torch.cuda.Stream(), torch.cuda.Stream()
    slow = torch.randn((4096, 4096), device="cuda")
    torch.cuda.synchronize()
    for n in (0, 1, 0, 1):
        with torch.cuda.stream(other):
            for _ in range(6):
                slow = torch.nn.functional.normalize(slow @ slow)
            layer.write(n)
            written = torch.cuda.Event()
            written.record()
        with torch.cuda.stream(mine):
            ep.moe_route(layer.src[0][0], None, "softmax", layer.k, layer.outs["ids"].t,
                         layer.outs["wt"].t, layer.st)
            mine.wait_event(written)
            layer.run()
        _same(layer.take(), want[n])


@pytest.mark.parametrize("size", SIZES[:1] + SIZES[3:], ids=str)
def test_captured_with_what_writes_the_inputs(ep, size):
    """One graph of the writes and the calls, and one whose writes are on a branch of
    their own; replayed without a pause."""
    layer = Layer(ep, *size)
    want = layer.alone()
    for branch in (False, True):
        graph = torch.cuda.CUDAGraph()
        took = []
        with torch.cuda.graph(graph):
            for n in (0, 1, 0):
                if branch:
                    side = torch.cuda.Stream()
                    side.wait_stream(torch.cuda.current_stream())
                    with torch.cuda.stream(side):
                        layer.write(n)
                    ep.moe_route(layer.src[0][0], None, "softmax", layer.k, layer.outs["ids"].t,
                                 layer.outs["wt"].t, layer.st)
                    torch.cuda.current_stream().wait_stream(side)
                else:
                    layer.write(n)
                layer.run()
                took.append({m: v.t.clone() for m, v in layer.outs.items()})
        for _ in range(20):
            graph.replay()
        torch.cuda.synchronize()
        layer.take()
        for got, n in zip(took, (0, 1, 0)):
            _same(got, want[n])
