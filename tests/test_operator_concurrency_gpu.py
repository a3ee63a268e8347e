"""Routing, the gradients and the INT8 product from two host threads on two
streams, with problems that share a kernel but ask for different amounts of
shared memory, or that share the GPU's tensor memory and clusters: every call is
taken, and every result is that of the same call alone."""
import threading

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ep():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a CUDA device")
    import combine_moe_dispatch_layout_gb300 as ep
    return ep


def _together(jobs, rounds, calls):
    """jobs: (call, outputs).  Runs every job `calls` times in a row from its own
    thread and stream, all at once, `rounds` times over."""
    want = []
    for call, outs in jobs:
        call(torch.cuda.current_stream())
        torch.cuda.synchronize()
        want.append([t.clone() for t in outs])
    streams = [torch.cuda.Stream() for _ in jobs]
    for _ in range(rounds):
        for _, outs in jobs:
            for t in outs:
                t.zero_()
        torch.cuda.synchronize()
        errors = []

        def work(call, stream):
            try:
                for _ in range(calls):
                    call(stream)
                stream.synchronize()
            except Exception as e:        # reported below
                errors.append(repr(e))

        threads = [threading.Thread(target=work, args=(c, s))
                   for (c, _), s in zip(jobs, streams)]
        for t in threads:
            t.start()
        for t in threads:
            t.join()
        torch.cuda.synchronize()
        assert not errors, errors[0]
        for (_, outs), ref in zip(jobs, want):
            for a, b in zip(outs, ref):
                assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


def _product(ep, sizes, N, K, out, seed):
    rng = np.random.default_rng(seed)
    rows, G = int(sum(sizes)), len(sizes)
    a = torch.from_numpy(rng.integers(-128, 128, (rows, K)).astype(np.int8)).cuda()
    w = torch.from_numpy(rng.integers(-128, 128, (G, N, K)).astype(np.int8)).cuda()
    col = torch.from_numpy(rng.random((G, N)).astype(np.float32)).cuda()
    row = torch.from_numpy(rng.random(rows).astype(np.float32)).cuda()
    n = torch.tensor(list(sizes), dtype=torch.int32, device="cuda") if G > 1 else None
    c = torch.zeros((rows, N), dtype=out, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")

    def call(stream):
        ep.moe_linear_i8(a, w, K, n, col, (row, 0, 4), None, c, st, stream=stream)
    return call, [c, st]


def test_products_of_different_shared_memory(ep):
    """One kernel, group tables of 1, 32 and 1000 groups."""
    jobs = [_product(ep, [3300], 256, 64, torch.bfloat16, 1),
            _product(ep, [104] * 32, 256, 64, torch.bfloat16, 2),
            _product(ep, [130] * 1000, 64, 64, torch.bfloat16, 3)]
    _together(jobs[:2], 4, 3000)
    _together(jobs, 2, 1500)


def test_wide_routings_of_different_shared_memory(ep):
    """Both above the default limit of a block."""
    jobs = []
    for E in (4096, 4080):
        x = torch.randn((2, E), device="cuda")
        ids = torch.zeros((2, 4), dtype=torch.int32, device="cuda")
        w = torch.zeros((2, 4), device="cuda")
        st = torch.zeros(1, dtype=torch.int32, device="cuda")

        def call(stream, x=x, ids=ids, w=w, st=st, E=E):
            ep.moe_route(x, None, "softmax", 4, ids, w, st, n_group=E, topk_group=9,
                         stream=stream)
        jobs.append((call, [ids, w, st]))
    _together(jobs, 4, 1500)


def test_clusters_and_tensor_memory_of_two_streams(ep):
    """Products over clusters of different sizes (K split and not, both tile
    widths), the kernel for few rows, routing and combine's gradient."""
    jobs = [_product(ep, [197], 1001, 2000, torch.float32, 4),
            _product(ep, [600], 2000, 1024, torch.float16, 5),
            _product(ep, [100, 1, 0, 31, 260], 1000, 1040, torch.bfloat16, 6),
            _product(ep, [2], 700, 4096, torch.bfloat16, 7)]
    x = torch.randn((3000, 256), device="cuda")
    ids = torch.zeros((3000, 8), dtype=torch.int32, device="cuda")
    w = torch.zeros((3000, 8), device="cuda")
    d = torch.zeros((3000, 256), device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")

    def route(stream):
        ep.moe_route(x, None, "sigmoid", 8, ids, w, st, stream=stream)
        ep.moe_route_backward(x, ids, w, "sigmoid", d, st, stream=stream)
    jobs.append((route, [ids, w, d, st]))
    _together(jobs, 4, 150)
