"""Workloads of the routing, gradient and 8-bit matrix product operators.

Four operators are run here, each in a plain form (elementary torch
operations in fp32) and, where ``own`` is true, through the package's entry
points:

* ``route``            logits -> expert ids and gate weights of every token
* ``route_backward``   gradient of the gate weights -> gradient of the logits
* ``combine_backward`` gradient of the combined tokens -> gradients of the
                       experts' output rows and of the gate weights
* ``linear_i8``        INT8 rows x INT8 weights with a scale per row and per
                       output column, rows grouped by expert

The sizes are those of the benchmark workloads (``workloads.py``) and of the
ragged shapes in the tests.
"""
import math

import numpy as np
import torch

own = False

_DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32,
       "int32": torch.int32}
_BIG = torch.finfo(torch.float32).max


def listed():
    return [
        # a serving step of 32 tokens: DeepSeek-V3-shaped routing (sigmoid
        # scores, balance bias, best 4 of 8 groups), all launch latency
        dict(name="route_serve", op="route", T=32, E=256, k=8, dtype="fp32", score="sigmoid",
             bias=True, groups=8, keep=4, best=2, renorm=True, scale=2.5, masked=0.0),
        # the same routing over a training batch (8 ranks x 4096 tokens)
        dict(name="route_train", op="route", T=32768, E=256, k=8, dtype="fp32", score="sigmoid",
             bias=True, groups=8, keep=4, best=2, renorm=True, scale=2.5, masked=0.0),
        # softmax routing over the widest expert set (384 ranks x 2 experts),
        # bf16 logits, some experts switched off
        dict(name="route_wide", op="route", T=49152, E=768, k=8, dtype="bf16", score="softmax",
             bias=False, groups=1, keep=1, best=1, renorm=False, scale=1.0, masked=0.02),
        # the router's gradient for the training batch
        dict(name="route_backward_train", op="route_backward", T=32768, E=256, k=8,
             dtype="fp32", score="sigmoid", renorm=True, scale=2.5, masked=0.0),
        # the dense gradient: softmax without renormalisation touches every logit
        dict(name="route_backward_wide", op="route_backward", T=49152, E=768, k=8,
             dtype="bf16", score="softmax", renorm=False, scale=1.0, masked=0.02),
        # combine's gradient for the training batch: 262,144 rows of 7168
        dict(name="combine_backward_train", op="combine_backward", R=8, epr=32, bs=4096, k=8,
             H=7168, dtype="bf16"),
        # few ranks, odd counts, narrow fp16 rows
        dict(name="combine_backward_ragged", op="combine_backward", R=3, epr=5, bs=777, k=7,
             H=1000, dtype="fp16"),
        # one decoded token through the shared expert's gate/up product
        dict(name="i8_one_token", op="linear_i8", G=1, rows=1, N=4096, K=7168, out="bf16",
             bias=False, images=False, spread="even"),
        # 32 tokens x 8 experts of a serving step over 256 experts: row images
        # as the dispatch writes them, raw accumulators for the SwiGLU stage
        dict(name="i8_experts_serve", op="linear_i8", G=256, rows=256, N=4096, K=7168,
             out="int32", bias=False, images=True, spread="even"),
        # the shared expert over 4096 tokens
        dict(name="i8_dense_prefill", op="linear_i8", G=1, rows=4096, N=4096, K=7168,
             out="bf16", bias=False, images=True, spread="even"),
        # one rank's 32 experts, skewed load, the down product
        dict(name="i8_experts_prefill", op="linear_i8", G=32, rows=32768, N=7168, K=2048,
             out="fp16", bias=False, images=True, spread="zipf"),
        # a small odd-sized product with padded rows and a bias
        dict(name="i8_ragged", op="linear_i8", G=1, rows=197, N=1001, K=1992, out="fp32",
             bias=True, images=False, spread="even"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["route", "route_backward", "combine_backward", "linear_i8", "linear_i8"])
    if op in ("route", "route_backward"):
        groups, per = rng.choice([(1, rng.randint(8, 768)), (8, rng.randint(2, 64)),
                                  (rng.randint(2, 12), rng.randint(3, 40))])
        E = groups * per
        T = _log(rng, 1, max(64, 49152 * 768 // max(E, 256)))
        keep = rng.randint(1, groups)
        k = min(rng.choice([1, 2, 4, 6, 7, 8, 8, 10]), keep * per)
        case = dict(op=op, T=T, E=E, k=k, dtype=rng.choice(["fp32", "fp32", "bf16", "fp16"]),
                    score=rng.choice(["sigmoid", "softmax"]), renorm=rng.random() < 0.5,
                    scale=rng.choice([1.0, 2.5, 16.0]), masked=rng.choice([0.0, 0.0, 0.1]))
        if op == "route":
            case.update(bias=rng.random() < 0.6, groups=groups, keep=keep, best=rng.choice([1, 2]))
        return case
    if op == "combine_backward":
        R, epr = rng.choice([1, 2, 3, 8, 16, 32, 384]), rng.randint(1, 10)
        H = 8 * _log(rng, 8, 896)
        k = min(rng.randint(1, 9), R * epr)
        return dict(op=op, R=R, epr=epr, bs=max(1, _log(rng, 1, 4096 * 256 * 896 // (R * k * H))),
                    k=k, H=H, dtype=rng.choice(["bf16", "fp16"]))
    G = rng.choice([1, 1, rng.randint(2, 64), rng.randint(65, 256)])
    N = _log(rng, 64, 7168)
    K = _log(rng, 64, min(7168, 4096 * 7168 * 256 // (G * N)))
    rows = _log(rng, 1, 8192)
    return dict(op=op, G=G, rows=rows, N=N, K=K,
                out=rng.choice(["bf16", "fp16", "fp32", "int32"]), bias=rng.random() < 0.3,
                images=rng.random() < 0.5, spread=rng.choice(["even", "even", "zipf"]))


def work(case):
    """Bytes: every input that matters read once and every output written
    once.  Flops: the arithmetic of the definition."""
    op = case["op"]
    if op in ("route", "route_backward"):
        T, E, k = case["T"], case["E"], case["k"]
        el = 4 if case["dtype"] == "fp32" else 2
        if op == "route":
            return {"bytes": T * E * el + T * k * 8, "flops": T * E * 6}
        dense = case["score"] == "softmax" and not case["renorm"]
        read = T * E * el if dense else T * k * el
        return {"bytes": read + T * E * el + T * k * 8,
                "flops": T * (E * 6 if dense else k * 10)}
    if op == "combine_backward":
        T = case["R"] * case["bs"]
        P = T * case["k"]
        row = 2 * case["H"]
        return {"bytes": T * row + 2 * P * row + P * 16, "flops": 3 * P * case["H"]}
    G, rows, N, K = (case[n] for n in ("G", "rows", "N", "K"))
    if case["spread"] == "zipf":
        used = min(G, rows)
    else:   # experts that get a row when rows fall evenly at random
        used = G * (1.0 - (1.0 - 1.0 / G) ** rows) if G > 1 else 1
    out = 2 if case["out"] in ("bf16", "fp16") else 4
    return {"bytes": used * N * K + rows * K + rows * N * out, "flops": 2 * rows * N * K}


# ---- inputs ------------------------------------------------------------------

def _gen(seed, salt):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed * 16 + salt)
    return g


def _draw_logits(n, E, dtype, masked, g):
    x = torch.randn((n, E), generator=g, device="cuda") * 1.5
    if masked > 0.0:
        off = torch.rand((n, E), generator=g, device="cuda") < masked
        off |= torch.rand((n, 1), generator=g, device="cuda") < masked / 64   # nothing left
        x = x.masked_fill(off, float("-inf"))
    return x.to(dtype)


def _close_rows(x, bias, case):
    """Rows whose choice hangs on the last bits of a score: two neighbours of
    the ordering, or two groups, that differ by less than a 32-bit sum is
    good for (equal values are no such case: they go to the lowest index)."""
    l = x.double().clamp(max=_BIG)
    on = l > -math.inf
    if case["score"] == "sigmoid":
        s = 1.0 / (1.0 + torch.exp(-l))
    else:
        top = l.amax(1, keepdim=True).clamp(min=-_BIG)
        e = torch.exp(l - top)
        s = e / e.sum(1, keepdim=True).clamp(min=1e-300)
    c = s + bias.double() if bias is not None else s
    c = c.masked_fill(~on, -math.inf)
    bad = torch.zeros(x.shape[0], dtype=torch.bool, device=x.device)

    def close(v, n):
        v = v.sort(1, descending=True).values[:, :n + 1]
        d = v[:, :-1] - v[:, 1:]
        small = 4e-6 * v[:, :1].abs().clamp(min=1e-9)
        return ((d < small) & (d > 0)).any(1)

    if case["groups"] > 1:
        per = c.view(x.shape[0], case["groups"], -1).sort(2, descending=True).values
        per = per[:, :, :case["best"]]
        per = per.masked_fill(per == -math.inf, 0.0).sum(2)
        bad |= close(per, case["groups"] - 1)
    if bias is not None:
        bad |= close(c, min(case["E"] - 1, 64))
    return bad


def _prepare_route(case, seed):
    g = _gen(seed, 1)
    T, E, k, dtype = case["T"], case["E"], case["k"], _DT[case["dtype"]]
    x = _draw_logits(T, E, dtype, case["masked"], g)
    bias = None
    if case["op"] == "route":
        if case["bias"]:
            # a balance bias moves in steps of 0.001
            bias = torch.round(torch.randn(E, generator=g, device="cuda") * 30) * 0.001
        for _ in range(16):
            bad = _close_rows(x, bias, case).nonzero()[:, 0]
            if bad.numel() == 0:
                break
            x[bad] = _draw_logits(bad.numel(), E, dtype, case["masked"], g)
    st = {"case": case, "logits": x, "bias": bias,
          "status": torch.zeros(1, dtype=torch.int32, device="cuda")}
    if case["op"] == "route":
        st["idx"] = torch.empty((T, k), dtype=torch.int32, device="cuda")
        st["weights"] = torch.empty((T, k), dtype=torch.float32, device="cuda")
    else:
        order = x.float().sort(dim=1, descending=True, stable=True)
        st["idx"] = torch.where(order.values[:, :k] > -math.inf, order.indices[:, :k],
                                -1).to(torch.int32).contiguous()
        st["d_weights"] = torch.randn((T, k), generator=g, device="cuda")
        st["d_logits"] = torch.empty_like(x)
    return st


def _plan(idx, R, bs, k, epr):
    """Send index, put offsets and partition bases of a routing, as the
    dispatch layout and notify stages define them."""
    E = R * epr
    src = torch.arange(R * bs, device=idx.device).repeat_interleave(k) // bs
    key = idx.reshape(-1).long() * R + src
    order = key.sort(stable=True).indices
    row = torch.empty_like(order)
    row[order] = torch.arange(order.numel(), device=idx.device)
    count = torch.bincount(key, minlength=E * R)
    start = count.cumsum(0) - count
    base = torch.cat([start[::epr * R], torch.tensor([order.numel()], device=idx.device)])
    put = start - base[:R].repeat_interleave(epr * R)
    send = row - start[key]
    return send.int(), put.int(), base.long().contiguous(), row


def _prepare_combine_backward(case, seed):
    g = _gen(seed, 2)
    R, epr, bs, k, H = (case[n] for n in ("R", "epr", "bs", "k", "H"))
    T, E, dtype = R * bs, R * epr, _DT[case["dtype"]]
    idx = torch.rand((T, E), generator=g, device="cuda").topk(k, dim=1).indices.int().contiguous()
    w = torch.softmax(torch.randn((T, k), generator=g, device="cuda"), dim=1)
    send, put, base, row = _plan(idx, R, bs, k, epr)
    y = torch.empty((T * k, H), dtype=dtype, device="cuda")
    for part in y.split(1 << 15):
        part.copy_(torch.randn(part.shape, generator=g, device="cuda"))
    d_out = torch.randn((T, H), generator=g, device="cuda").to(dtype)
    return {"case": case, "idx": idx, "weights": w, "send": send, "put": put, "base": base,
            "row": row, "y": y, "d_out": d_out, "d_y": torch.zeros_like(y),
            "d_weights": torch.empty((T, k), dtype=torch.float32, device="cuda"),
            "status": torch.zeros(1, dtype=torch.int32, device="cuda")}


def _group_sizes(case, seed):
    G, rows = case["G"], case["rows"]
    rng = np.random.RandomState(seed % (1 << 31))
    p = np.ones(G) if case["spread"] == "even" else (np.arange(G) + 1.0) ** -1.0
    return rng.multinomial(rows, rng.permutation(p) / p.sum())


def _prepare_linear(case, seed):
    g = _gen(seed, 3)
    G, rows, N, K = (case[n] for n in ("G", "rows", "N", "K"))
    sizes = _group_sizes(case, seed)
    wide = (K + 15) // 16 * 16          # weight rows start on 16-byte boundaries
    w = torch.zeros((G, N, wide), dtype=torch.int8, device="cuda")
    for part in w.view(G * N, wide).split(max(1, (1 << 30) // wide)):
        part[:, :K] = torch.randint(-127, 128, (part.shape[0], K), generator=g,
                                    dtype=torch.int8, device="cuda")
    codes = torch.randint(-127, 128, (rows, K), generator=g, dtype=torch.int8, device="cuda")
    scale = (torch.rand(rows, generator=g, device="cuda") * 3 + 0.1) / 127
    at = (K + 31) // 32 * 32            # a dispatched row image keeps its scale here
    if case["images"]:
        a = torch.zeros((rows, at + 32), dtype=torch.uint8, device="cuda")
        a[:, at:at + 4] = scale.view(torch.uint8).view(rows, 4)
    else:
        a = torch.zeros((rows, wide), dtype=torch.uint8, device="cuda")
    a[:, :K] = codes.view(torch.uint8)
    col = (torch.rand((G, N), generator=g, device="cuda") + 0.5) / (73.6 * K ** 0.5)
    bias = torch.randn((G, N), generator=g, device="cuda") if case["bias"] else None
    off = np.concatenate([[0], np.cumsum(sizes)])
    return {"case": case, "a": a, "at": at, "scale": scale, "w": w, "col": col, "bias": bias,
            "group_rows": torch.tensor(sizes, dtype=torch.int32, device="cuda"),
            "group_of": torch.tensor(np.repeat(np.arange(G), sizes), device="cuda"),
            "place": torch.tensor(np.arange(rows) - np.repeat(off[:-1], sizes), device="cuda"),
            "most": int(sizes.max()),
            "c": torch.empty((rows, N), dtype=_DT[case["out"]], device="cuda"),
            "status": torch.zeros(1, dtype=torch.int32, device="cuda")}


def prepare(case, seed):
    if case["op"] in ("route", "route_backward"):
        return _prepare_route(case, seed)
    if case["op"] == "combine_backward":
        return _prepare_combine_backward(case, seed)
    return _prepare_linear(case, seed)


# ---- plain forms ---------------------------------------------------------------

def _scores(l, score):
    if score == "sigmoid":
        return 1.0 / (1.0 + torch.exp(-l))
    top = l.amax(1, keepdim=True).clamp(min=-_BIG)
    e = torch.exp(l - top)
    return e / e.sum(1, keepdim=True).clamp(min=1e-30)


def _plain_route(st):
    case = st["case"]
    T, E, k = case["T"], case["E"], case["k"]
    l = st["logits"].float().clamp(max=_BIG)
    s = _scores(l, case["score"])
    none = torch.full_like(l, -math.inf)
    on = l > -math.inf
    c = s + st["bias"] if st["bias"] is not None else s
    key = torch.where(on, c if st["bias"] is not None else l, none)
    if case["groups"] > 1:
        top = torch.where(on, c, none).view(T, case["groups"], -1)
        top = top.sort(dim=2, descending=True).values[:, :, :case["best"]]
        some = top[:, :, 0] > -math.inf
        total = torch.where(top > -math.inf, top, torch.zeros_like(top)).sum(2)
        total = torch.where(some, total, torch.full_like(total, -math.inf))
        kept = total.sort(dim=1, descending=True, stable=True).indices[:, :case["keep"]]
        use = torch.zeros_like(some).scatter_(1, kept, True)
        key = torch.where(use.repeat_interleave(E // case["groups"], 1), key, none)
    best = key.sort(dim=1, descending=True, stable=True)
    there = best.values[:, :k] > -math.inf
    order = best.indices[:, :k]
    w = torch.where(there, s.gather(1, order), torch.zeros_like(s[:, :k]))
    if case["renorm"]:
        w = w / w.sum(1, keepdim=True).clamp(min=1e-30)
    return [torch.where(there, order, -1).int(), w * case["scale"]]


def _plain_route_backward(st):
    case = st["case"]
    l = st["logits"].float().clamp(max=_BIG)
    there = st["idx"] >= 0
    at = st["idx"].clamp(min=0).long()
    zero = torch.zeros_like(st["d_weights"])
    g = torch.where(there, st["d_weights"], zero) * case["scale"]
    s = _scores(l, case["score"])
    p = torch.where(there, s.gather(1, at), zero)
    d = torch.zeros_like(l)
    if case["renorm"]:
        w = p / p.sum(1, keepdim=True).clamp(min=1e-30)
        v = w * (g - (w * g).sum(1, keepdim=True))
        v = v * (1.0 - p) if case["score"] == "sigmoid" else v
    elif case["score"] == "sigmoid":
        v = g * p * (1.0 - p)
    else:
        v = g * p
        d = -s * v.sum(1, keepdim=True)
    return d.scatter_add_(1, at, torch.where(there, v, zero)).to(st["logits"].dtype)


def _plain_combine_backward(st):
    case = st["case"]
    T, k, H = st["idx"].shape[0], case["k"], case["H"]
    g = st["d_out"].float()
    y = st["y"].float()[st["row"]].view(T, k, H)
    d_w = (y * g[:, None, :]).sum(2)
    d_y = torch.zeros_like(st["y"])
    d_y[st["row"]] = (st["weights"][:, :, None] * g[:, None, :]).view(T * k, H).to(d_y.dtype)
    return [d_y, d_w]


def _plain_linear(st):
    case = st["case"]
    G, K, N = case["G"], case["K"], case["N"]
    codes = st["a"][:, :K].view(torch.int8).float()
    w = st["w"][:, :, :K].float()
    if G == 1:
        acc = codes @ w[0].T
    else:   # every expert's rows in a block of its own, one batched product
        block = torch.zeros((G, st["most"], K), device=codes.device)
        block[st["group_of"], st["place"]] = codes
        acc = torch.bmm(block, w.transpose(1, 2))[st["group_of"], st["place"]]
    if case["out"] == "int32":
        return torch.round(acc).int()
    scale = st["scale"]
    if case["images"]:
        scale = st["a"][:, st["at"]:st["at"] + 4].contiguous().view(torch.float32)[:, 0]
    acc = acc * st["col"][st["group_of"]] * scale[:, None]
    if st["bias"] is not None:
        acc = acc + st["bias"][st["group_of"]]
    return acc.to(_DT[case["out"]])


# ---- the framework's operators -----------------------------------------------------

def _own(st):
    import combine_moe_dispatch_layout_gb300 as ep
    case = st["case"]
    if case["op"] == "route":
        ep.moe_route(st["logits"], st["bias"], case["score"], case["k"], st["idx"],
                     st["weights"], st["status"], n_group=case["groups"],
                     topk_group=case["keep"], group_top=case["best"],
                     renormalise=case["renorm"], scale=case["scale"])
        return [st["idx"], st["weights"]]
    if case["op"] == "route_backward":
        ep.moe_route_backward(st["logits"], st["idx"], st["d_weights"], case["score"],
                              st["d_logits"], st["status"], renormalise=case["renorm"],
                              scale=case["scale"])
        return st["d_logits"]
    if case["op"] == "combine_backward":
        shape = ep.make_shape(case["R"], case["bs"], case["k"], case["epr"], case["H"],
                              _DT[case["dtype"]])
        ep.moe_combine_backward(shape, st["d_out"], st["y"], st["idx"], st["weights"],
                                st["send"], st["put"], st["base"], st["d_y"],
                                st["d_weights"], st["status"])
        return [st["d_y"], st["d_weights"]]
    if case["images"]:
        scale = (st["a"], st["at"], st["a"].shape[1])
    else:
        scale = (st["scale"], 0, 4)
    ep.moe_linear_i8(st["a"], st["w"], case["K"],
                     st["group_rows"] if case["G"] > 1 else None, st["col"], scale,
                     st["bias"], st["c"], st["status"])
    return st["c"]


def run(state):
    if own:
        return _own(state)
    return {"route": _plain_route, "route_backward": _plain_route_backward,
            "combine_backward": _plain_combine_backward,
            "linear_i8": _plain_linear}[state["case"]["op"]](state)


# ---- the definitions in 64 bits -----------------------------------------------------

def _exact_scores(l, score):
    """Scores of numpy float64 logits; a row of -inf alone scores 0."""
    if score == "sigmoid":
        return np.where(l >= 0, 1 / (1 + np.exp(-np.abs(l))),
                        np.exp(-np.abs(l)) / (1 + np.exp(-np.abs(l))))
    top = l.max(axis=1, keepdims=True)
    e = np.exp(l - np.where(np.isfinite(top), top, 0.0))
    total = e.sum(axis=1, keepdims=True)
    return np.divide(e, total, out=np.zeros_like(e), where=total > 0)


def _exact_route(case, st):
    l = st["logits"].double().cpu().numpy()
    T, E = l.shape
    k, n = case["k"], case["groups"]
    s = _exact_scores(l, case["score"])
    c = s if st["bias"] is None else s + st["bias"].double().cpu().numpy()
    rank = np.where(l > -np.inf, l if st["bias"] is None else c, -np.inf)
    if n > 1:
        per = np.where(l > -np.inf, c, -np.inf).reshape(T, n, E // n)
        best = -np.sort(-per, axis=2)[:, :, :case["best"]]
        total = np.where(np.isfinite(best), best, 0).sum(axis=2)
        total[best[:, :, 0] == -np.inf] = -np.inf
        keep = np.argsort(-total, axis=1, kind="stable")[:, :case["keep"]]
        use = np.zeros((T, n), bool)
        np.put_along_axis(use, keep, True, axis=1)
        rank = np.where(np.repeat(use, E // n, axis=1), rank, -np.inf)
    order = np.argsort(-rank, axis=1, kind="stable")[:, :k]
    there = np.take_along_axis(rank, order, 1) > -np.inf
    w = np.where(there, np.take_along_axis(s, order, 1), 0.0)
    if case["renorm"]:
        total = w.sum(axis=1, keepdims=True)
        w = np.divide(w, total, out=np.zeros_like(w), where=total > 0)
    return [np.where(there, order, -1).astype(np.int32), w * case["scale"]]


def _exact_route_backward(case, st):
    """The Jacobian of the definition applied to the weights' gradient:
    weights = scale * s / sum(s) or scale * s, s = sigmoid(l) or softmax(l)."""
    l = st["logits"].double().cpu().numpy()
    idx = st["idx"].cpu().numpy()
    g = st["d_weights"].double().cpu().numpy() * (idx >= 0) * case["scale"]
    at = np.maximum(idx, 0)
    s = _exact_scores(l, case["score"])
    chosen = np.take_along_axis(s, at, 1) * (idx >= 0)
    if case["renorm"]:
        total = chosen.sum(axis=1, keepdims=True)
        total[total == 0] = 1.0
        ds = (g - (g * chosen).sum(axis=1, keepdims=True) / total) / total
    else:
        ds = g
    ds = ds * (idx >= 0)
    if case["score"] == "sigmoid":
        dense = np.zeros_like(l)
        np.add.at(dense, (np.arange(l.shape[0])[:, None], at), ds * chosen * (1 - chosen))
        return dense
    dense = np.zeros_like(l)
    np.add.at(dense, (np.arange(l.shape[0])[:, None], at), ds * chosen)
    if case["renorm"]:       # the softmax's own sum cancels exactly
        return dense
    return dense - s * (ds * chosen).sum(axis=1, keepdims=True)


def _exact_combine_backward(case, st):
    k = case["k"]
    row = st["row"].view(-1, k)
    d_y = torch.zeros(st["y"].shape, dtype=torch.float64, device="cuda")
    d_w = torch.zeros(row.shape, dtype=torch.float64, device="cuda")
    w = st["weights"].double()
    for j in range(k):
        for part in torch.arange(row.shape[0], device="cuda").split(1 << 13):
            g = st["d_out"][part].double()
            to = row[part, j]
            d_w[part, j] = torch.einsum("th,th->t", st["y"][to].double(), g)
            d_y[to] = w[part, j][:, None] * g
    return [d_y, d_w]


def _exact_linear(case, st):
    G, rows, N, K = (case[n] for n in ("G", "rows", "N", "K"))
    sizes = st["group_rows"].tolist()
    c = torch.zeros((rows, N), dtype=torch.float64, device="cuda")
    a = st["a"][:, :K].contiguous().view(torch.int8)
    at = 0
    for g, n in enumerate(sizes):
        if n == 0:
            continue
        acc = a[at:at + n].double() @ st["w"][g, :, :K].double().t()
        if case["out"] != "int32":
            acc = acc * st["scale"][at:at + n].double()[:, None] * st["col"][g].double()
            if st["bias"] is not None:
                acc = acc + st["bias"][g].double()
        c[at:at + n] = acc
        at += n
    return c.round().int() if case["out"] == "int32" else c


def exact(case, seed):
    st = prepare(case, seed)
    return {"route": _exact_route, "route_backward": _exact_route_backward,
            "combine_backward": _exact_combine_backward,
            "linear_i8": _exact_linear}[case["op"]](case, st)
