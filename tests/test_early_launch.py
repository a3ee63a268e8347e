"""Kernels that may be put on the GPU while the stream's previous kernel still
writes: their loads are ordinary ones behind the wait (the read-only path asks that
nobody write the data for the kernel's whole life), and chains of such kernels
without a synchronisation give what the same calls give one at a time."""
import glob
import os
import re

import numpy as np
import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "combine_moe_dispatch_layout_gb300", "csrc")


def _code(path):
    return re.sub(r"//[^\n]*", "", open(path).read())


def _early_units():
    units = {os.path.basename(p): _code(p) for p in glob.glob(os.path.join(CSRC, "*.cu"))}
    early = {n: s for n, s in units.items()
             if "launch_early(" in s or "ProgrammaticStreamSerialization" in s}
    assert len(early) >= 5
    return early


def test_loads_of_early_kernels_are_ordinary_ones():
    shared = ["route_math.cuh", "group_tiles.cuh", "tcgen05.cuh"]
    units = dict(_early_units(), **{n: _code(os.path.join(CSRC, n)) for n in shared})
    for name, text in units.items():
        for word in ("__ldg", "ld_stream_16", ".nc", "__ldcs", "__ldlu"):
            assert word not in text, (name, word)
        assert not re.search(r"const\s+[\w:<> ]+\*\s*(const\s*)?__restrict__", text), name
        for call in re.findall(r"resolve_token\w*\s*(<[^>]*>)?\s*\(", text):
            assert call == "<true>", (name, call)
    # what those call of the shared header: the early form has no read-only load
    head = _code(os.path.join(CSRC, "moe_ep_internal.cuh"))
    body = head[head.index("void resolve_token("):]
    body = body[:body.index("\n}\n")]
    assert "__ldg" not in body and "__restrict__" not in body
    once = head[head.index("uint4 ld_once_16("):]
    assert ".nc" not in once[:once.index("\n}\n")]


def test_every_early_kernel_waits_first():
    """The wait is the first statement that is not a declaration of the kernel's own
    (no global load, no store, no call of another function stands before it)."""
    for name, text in _early_units().items():
        kernels = re.split(r"__global__", text)[1:]
        assert kernels, name
        for k in kernels:
            body = k[k.index("{"):]
            wait = body.index("wait_for_stream();")
            before = body[:wait]
            for word in ("= *", "atomic", "asm", "tensor_", "cluster_store", "smem_store",
                         "load_logit", "resolve_token", "__sync"):
                assert word not in before, (name, word)


# ---- chains on the GPU ---------------------------------------------------------------

@pytest.fixture(scope="module")
def ep():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a CUDA device")
    import combine_moe_dispatch_layout_gb300 as ep
    return ep


def _plan(idx, R, bs, k, epr):
    """Send index, put offsets and partition bases as layout and notify give them."""
    T, E = idx.shape[0], R * epr
    key = idx.reshape(-1).astype(np.int64) * R + np.repeat(np.arange(T) // bs, k)
    order = np.argsort(key, kind="stable")
    row = np.empty_like(order)
    row[order] = np.arange(len(order))
    count = np.bincount(key, minlength=E * R)
    start = np.cumsum(count) - count
    base = np.concatenate([start[::epr * R], [len(order)]])
    put = start - np.repeat(base[:R], epr * R)
    return (torch.from_numpy((row - start[key]).astype(np.int32)).cuda(),
            torch.from_numpy(put.astype(np.int32)).cuda(),
            torch.from_numpy(base.astype(np.int64)).cuda())


@pytest.mark.gpu
@pytest.mark.parametrize("T,E,H", [(6000, 256, 1000), (4096, 64, 2048), (3000, 1500, 64)])
def test_chain_of_early_kernels(ep, T, E, H):
    """Product -> routing -> its gradient -> combine's gradient -> product, each on what
    the one before it wrote, round after round over the same buffers with other
    data, and nothing in between; against the same calls with a synchronisation
    after each."""
    R, k, K, rounds = 4, 6, 256, 6
    bs, epr = T // R, E // R
    rng = np.random.default_rng(T)
    g = torch.Generator(device="cuda")
    g.manual_seed(T)

    def codes(*shape):
        return torch.randint(-127, 128, shape, generator=g, dtype=torch.int8, device="cuda")

    x = [codes(T, K) for _ in range(rounds)]
    w = [codes(1, E, K) for _ in range(rounds)]
    col = torch.full((1, E), 1.0 / (73.6 * 73.6 * K ** 0.5), device="cuda")
    row = torch.full((T,), 1.5, device="cuda")
    idx = np.stack([rng.permutation(E)[:k] for _ in range(T)]).astype(np.int32)
    send, put, base = _plan(idx, R, bs, k, epr)
    idx = torch.from_numpy(idx).cuda()
    y = torch.randn((T * k, H), generator=g, device="cuda").bfloat16()
    d_out = [torch.randn((T, H), generator=g, device="cuda").bfloat16() for _ in range(rounds)]
    shape = ep.make_shape(R, bs, k, epr, H, torch.bfloat16)
    wide = codes(1, 40, (H + 15) // 16 * 32)

    def run(sync):
        st = torch.zeros(1, dtype=torch.int32, device="cuda")
        logits = torch.zeros((T, E), device="cuda")
        ids = torch.zeros((T, k), dtype=torch.int32, device="cuda")
        wt = torch.zeros((T, k), device="cuda")
        d_l = torch.zeros((T, E), device="cuda")
        d_y = torch.zeros((T * k, H), dtype=torch.bfloat16, device="cuda")
        d_w = torch.zeros((T, k), device="cuda")
        acc = torch.zeros((T * k, 40), dtype=torch.int32, device="cuda")
        few = torch.zeros((8, 40), dtype=torch.int32, device="cuda")
        out = []

        def done():
            if sync:
                torch.cuda.synchronize()

        torch.cuda.synchronize()
        for r in range(rounds):
            ep.moe_linear_i8(x[r], w[r], K, None, col, (row, 0, 4), None, logits, st)
            done()
            ep.moe_route(logits, None, "softmax", k, ids, wt, st, renormalise=r % 2 == 0)
            done()
            # the weights (not the ids, which need their own plan) go on
            ep.moe_combine_backward(shape, d_out[r], y, idx, wt, send, put, base, d_y, d_w, st)
            done()
            ep.moe_route_backward(logits, ids, d_w, "softmax", d_l, st, renormalise=r % 2 == 0)
            done()
            rows = d_y.view(torch.int8)              # the bytes of the gradient rows as codes
            if H * 2 % 16 == 0:
                ep.moe_linear_i8(rows, wide, H * 2, None, None, None, None, acc, st)
                done()
                ep.moe_linear_i8(rows[:8], wide, H * 2, None, None, None, None, few, st)
                done()
            out.append([t.clone() for t in (logits, ids, wt, d_l, d_y, d_w, acc, few)])
        torch.cuda.synchronize()
        assert int(st.item()) == 0
        return out

    want = run(True)
    for _ in range(3):
        got = run(False)
        for r in range(rounds):
            for i, (a, b) in enumerate(zip(got[r], want[r])):
                a, b = a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8)
                assert torch.equal(a, b), (r, i)
    assert int((want[0][0] != want[1][0]).sum()) > T * E // 2      # the rounds differ
