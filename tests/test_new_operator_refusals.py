"""Host-side refusals of routing, its gradient, combine's gradient and the INT8
product, through the C ABI (no GPU: pointers are never dereferenced), and the
plain float64 forms against hand-worked cases and difference quotients."""
import ctypes
import os
import shutil

import numpy as np
import pytest

import plain_ops as P

OK = ctypes.c_void_p(0x10000)
ODD = ctypes.c_void_p(0x10008)


@pytest.fixture(scope="module")
def lib():
    if shutil.which("nvcc") is None and not os.path.exists("/usr/local/cuda/bin/nvcc"):
        pytest.skip("nvcc not available")
    import __graft_entry__
    L = ctypes.CDLL(__graft_entry__._load_builder().build())
    vp, i32, i64, f32 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_float
    L.moe_route.argtypes = [vp, i32, i64, i32, i64, vp, i32, i32, i32, i32, i32, i32, f32,
                            vp, vp, vp, vp]
    L.moe_route_backward.argtypes = [vp, i32, i64, i32, i64, i32, i32, i32, f32, vp, vp, vp,
                                     vp, vp]
    L.moe_linear_i8.argtypes = [vp, i64, i64, vp, i64, i32, i32, i32, vp, vp, vp, i64, vp,
                                vp, i32, vp, vp]
    return L


ROUTE = dict(logits=OK, dtype=2, T=4, E=16, stride=16, bias=OK, score=0, n=4, keep=2, top=2,
             k=4, renorm=1, scale=1.0, idx=OK, w=OK, st=OK, stream=None)


@pytest.mark.parametrize("bad", [
    dict(logits=None), dict(logits=ctypes.c_void_p(0x10002)), dict(dtype=3), dict(dtype=-1),
    dict(T=-1), dict(T=1 << 31), dict(T=1 << 30), dict(E=0), dict(E=4097), dict(stride=15),
    dict(stride=1 << 33), dict(bias=ctypes.c_void_p(0x10001)), dict(score=2), dict(score=-1),
    dict(n=0), dict(n=3), dict(n=32), dict(keep=0), dict(keep=5), dict(top=0), dict(top=3),
    dict(k=0), dict(k=17), dict(scale=float("inf")), dict(scale=float("nan")), dict(idx=None),
    dict(w=None), dict(w=ctypes.c_void_p(0x10002)), dict(st=None)], ids=str)
def test_route(lib, bad):
    assert lib.moe_route(*dict(ROUTE, **bad).values()) == 1


def test_route_empty_batch_touches_nothing(lib):
    a = dict(ROUTE, T=0, logits=None, idx=None, w=None)
    assert lib.moe_route(*a.values()) == 0


BACK = dict(logits=OK, dtype=2, T=4, E=16, stride=16, score=0, k=4, renorm=1, scale=1.0,
            idx=OK, dw=OK, dl=OK, st=OK, stream=None)


@pytest.mark.parametrize("bad", [
    dict(logits=None), dict(dtype=3), dict(T=-1), dict(E=0), dict(stride=8), dict(score=7),
    dict(k=17), dict(k=0), dict(scale=float("nan")), dict(idx=None), dict(dw=None),
    dict(dl=None), dict(dl=ODD), dict(st=None)], ids=str)
def test_route_backward(lib, bad):
    assert lib.moe_route_backward(*dict(BACK, **bad).values()) == 1


LINEAR = dict(a=OK, rows=4, a_stride=64, w=OK, w_stride=64, G=2, N=24, K=60, sizes=OK, col=OK,
              row=OK, row_stride=4, bias=OK, c=OK, dtype=0, st=OK, stream=None)


@pytest.mark.parametrize("bad", [
    dict(a=None), dict(a=ODD), dict(rows=-1), dict(rows=1 << 31), dict(a_stride=48),
    dict(rows=(1 << 31) - 512), dict(rows=1 << 30, N=65536),
    dict(a_stride=72), dict(w=None), dict(w=ODD), dict(w_stride=48), dict(w_stride=60),
    dict(a_stride=1 << 32), dict(w_stride=1 << 32), dict(row_stride=1 << 32),
    dict(G=0), dict(G=4097), dict(N=0), dict(N=65537), dict(K=0), dict(K=65537),
    dict(sizes=None), dict(col=None), dict(row=None), dict(row_stride=2), dict(row_stride=6),
    dict(bias=ctypes.c_void_p(0x10002)), dict(c=None), dict(c=ODD), dict(dtype=4),
    dict(dtype=-1), dict(st=None)], ids=str)
def test_linear_i8(lib, bad):
    assert lib.moe_linear_i8(*dict(LINEAR, **bad).values()) == 1


def test_linear_i8_no_rows(lib):
    assert lib.moe_linear_i8(*dict(LINEAR, rows=0, a=None, c=None).values()) == 0


# ---- the plain forms the GPU tests compare with ---------------------------------

def test_plain_route_by_hand():
    # sigmoid(0) = 0.5, sigmoid(log 3) = 0.75, sigmoid(-log 3) = 0.25
    l = np.array([[0.0, np.log(3.0), -np.log(3.0), -np.inf]])
    ids, w = P.route(l, None, "sigmoid", 2)
    assert ids.tolist() == [[1, 0]]
    np.testing.assert_allclose(w, [[0.6, 0.4]], rtol=1e-15)
    ids, w = P.route(l, np.array([0.0, 0.0, 0.6, 9.0]), "sigmoid", 4, scale=2.0)
    assert ids.tolist() == [[2, 1, 0, -1]]                  # 0.85, 0.75, 0.5; 3 is masked
    np.testing.assert_allclose(w, [[1 / 3, 1.0, 2 / 3, 0.0]], rtol=1e-15)
    # groups of two: sums 1.25 and 0.25; group 0 stays
    ids, _ = P.route(l, None, "sigmoid", 3, n_group=2, topk_group=1, group_top=2)
    assert ids.tolist() == [[1, 0, -1]]
    ids, w = P.route(np.log(np.array([[1.0, 4.0, 3.0, 2.0]])), None, "softmax", 2,
                     renormalise=False)
    assert ids.tolist() == [[1, 2]]
    np.testing.assert_allclose(w, [[0.4, 0.3]], rtol=1e-15)
    ids, _ = P.route(np.zeros((1, 5)), None, "softmax", 3)
    assert ids.tolist() == [[0, 1, 2]]


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("renorm", [True, False])
def test_plain_gradient_is_the_difference_quotient(score, renorm):
    rng = np.random.default_rng(1)
    l = rng.standard_normal((4, 9))
    ids, _ = P.route(l, None, score, 3)
    ids[2, 1] = -1
    g = rng.standard_normal(ids.shape)
    d = P.route_backward(l, ids, g, score, renorm, 1.7)
    h = 1e-6
    for e in range(9):
        up, dn = l.copy(), l.copy()
        up[:, e] += h
        dn[:, e] -= h
        f = [(P.weights_of(P.scores(v, score), ids, renorm, 1.7) * g).sum(axis=1)
             for v in (up, dn)]
        np.testing.assert_allclose((f[0] - f[1]) / (2 * h), d[:, e], atol=2e-9)


def test_plain_product_by_hand():
    a = np.array([[1, -2], [3, 4]], np.int8)
    w = np.array([[[5, 6]], [[-128, 127]]], np.int8)
    assert P.linear_i8(a, w, [1, 1]).tolist() == [[-7], [124]]
    v = P.linear_i8(a, w, [1, 1], np.array([[2.0], [0.5]], np.float32),
                    np.array([3.0, 4.0], np.float32), np.array([[1.0], [-8.0]], np.float32))
    assert v.dtype == np.float32 and v.tolist() == [[-41.0], [240.0]]
