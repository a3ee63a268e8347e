"""Workloads of the norm in front of an MoE layer and of its FP8 products.

Four operators are run here, each in a plain form (elementary torch
operations in fp32) and, where ``own`` is true, through the package's entry
points:

* ``norm``           residual's addition and root-mean-square norm of token
                     rows, in 16 bits and as e4m3 row images (a scale per 128
                     values)
* ``norm_backward``  gradients of that norm: of the rows and of its weights
* ``swiglu``         [gate | up] rows -> e4m3 row images of silu(gate) * up
* ``linear``         e4m3 row images x e4m3 weights with a scale per 128 x 128
                     block, rows grouped by expert

A row image holds a row's codes, then from the next multiple of 32 bytes on
its fp32 scales, and is a multiple of 32 bytes long.  The sizes are those of
the benchmark workloads (``workloads.py``) and of the ragged shapes in the
tests.
"""
import math

import numpy as np
import torch

own = False

_DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
_F8 = torch.float8_e4m3fn
_EPS = 1e-6
_TINY = 1e-12          # the largest magnitude of a block counts as at least this


def listed():
    return [
        # a serving step of 32 tokens: the residual stream's addition, rows for
        # the router in bf16 and for the products in e4m3; all launch latency
        dict(name="norm_serve", op="norm", T=32, H=7168, dtype="bf16", residual=True, out=True,
             codes=True, rstd=False),
        # the training batch (8 ranks x 4096 tokens): 16-bit rows, and what the
        # gradient needs
        dict(name="norm_train", op="norm", T=32768, H=7168, dtype="bf16", residual=True, out=True,
             codes=False, rstd=True),
        # prefill of narrow fp16 rows straight into row images; odd counts
        dict(name="norm_ragged_codes", op="norm", T=24251, H=1000, dtype="fp16", residual=False,
             out=False, codes=True, rstd=False),
        # the norm's gradient for the training batch, the stream's own gradient added
        dict(name="norm_backward_train", op="norm_backward", T=32768, H=7168, dtype="bf16",
             d_sum=True),
        # a small step of narrow fp16 rows; odd counts
        dict(name="norm_backward_ragged", op="norm_backward", T=777, H=1000, dtype="fp16",
             d_sum=False),
        # 32 tokens x 8 experts between the two products of a serving step
        dict(name="swiglu_serve", op="swiglu", rows=256, I=2048, dtype="bf16"),
        # the same for the training batch's 262,144 rows
        dict(name="swiglu_prefill", op="swiglu", rows=262144, I=2048, dtype="bf16"),
        # one decoded token through the shared expert's gate/up product
        dict(name="f8_one_token", op="linear", G=1, rows=1, N=4096, K=7168, out="bf16", bias=False,
             spread="even"),
        # 32 tokens x 8 experts of a serving step over 256 experts
        dict(name="f8_experts_serve", op="linear", G=256, rows=256, N=4096, K=7168, out="bf16",
             bias=False, spread="even"),
        # the shared expert over 8192 tokens
        dict(name="f8_dense_prefill", op="linear", G=1, rows=8192, N=4096, K=7168, out="bf16",
             bias=False, spread="even"),
        # one rank's 32 experts, skewed load, the down product
        dict(name="f8_experts_prefill", op="linear", G=32, rows=32768, N=7168, K=2048, out="fp16",
             bias=False, spread="zipf"),
        # a small odd-sized product in fp32 with a bias
        dict(name="f8_ragged", op="linear", G=1, rows=197, N=1001, K=1992, out="fp32", bias=True,
             spread="even"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(max(lo, hi))))))


def draw(rng):
    op = rng.choice(["norm", "norm_backward", "swiglu", "linear", "linear", "linear"])
    if op in ("norm", "norm_backward"):
        H = 8 * _log(rng, 8, 1024)
        case = dict(op=op, T=_log(rng, 1, min(65536, 32768 * 7168 // H)), H=H,
                    dtype=rng.choice(["bf16", "fp16"]))
        if op == "norm_backward":
            case.update(d_sum=rng.random() < 0.5)
        else:
            out = rng.random() < 0.7
            case.update(residual=rng.random() < 0.6, out=out,
                        codes=not out or rng.random() < 0.5, rstd=rng.random() < 0.4)
        return case
    if op == "swiglu":
        I = 8 * _log(rng, 8, 512)
        return dict(op=op, rows=_log(rng, 1, 262144 * 1024 // I), I=I,
                    dtype=rng.choice(["bf16", "bf16", "fp16", "fp32"]))
    G = rng.choice([1, 1, rng.randint(2, 64), rng.randint(65, 256)])
    N = _log(rng, 64, 7168)
    K = _log(rng, 64, min(7168, 4096 * 7168 * 256 // (G * N)))
    return dict(op=op, G=G, rows=_log(rng, 1, 8192), N=N, K=K,
                out=rng.choice(["bf16", "fp16", "fp32"]), bias=rng.random() < 0.3,
                spread=rng.choice(["even", "even", "zipf"]))


def _blocks(n):
    return (n + 127) // 128


def work(case):
    """Bytes: every input that matters read once and every output written
    once.  Flops: the arithmetic of the definition."""
    op = case["op"]
    if op == "norm":
        T, H = case["T"], case["H"]
        row = 2 * H * (1 + 2 * case["residual"] + case["out"])
        row += (H + 4 * _blocks(H)) * case["codes"] + 4 * case["rstd"]
        return {"bytes": T * row + 4 * H, "flops": T * H * (5 + 3 * case["codes"])}
    if op == "norm_backward":
        T, H = case["T"], case["H"]
        return {"bytes": T * (2 * H * (3 + case["d_sum"]) + 4) + 8 * H, "flops": 9 * T * H}
    if op == "swiglu":
        rows, I = case["rows"], case["I"]
        el = 4 if case["dtype"] == "fp32" else 2
        return {"bytes": rows * (2 * I * el + I + 4 * _blocks(I)), "flops": 8 * rows * I}
    G, rows, N, K = (case[n] for n in ("G", "rows", "N", "K"))
    if case["spread"] == "zipf":
        used = min(G, rows)
    else:   # experts that get a row when rows fall evenly at random
        used = G * (1.0 - (1.0 - 1.0 / G) ** rows) if G > 1 else 1
    out = 4 if case["out"] == "fp32" else 2
    return {"bytes": used * (N * K + 4 * _blocks(N) * _blocks(K))
            + rows * (K + 4 * _blocks(K)) + rows * N * out, "flops": 2 * rows * N * K}


# ---- inputs ------------------------------------------------------------------

def _gen(seed, salt):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed * 16 + salt)
    return g


def _randn(shape, dtype, g, scale=1.0):
    x = torch.empty(shape, dtype=dtype, device="cuda")
    for part in x.split(1 << 15):
        part.copy_(torch.randn(part.shape, generator=g, device="cuda") * scale)
    return x


def _image_bytes(H):
    return (H + 31) // 32 * 32 + (4 * _blocks(H) + 31) // 32 * 32


def _codes(image, H):
    """The e4m3 codes [rows, H] and the scales [rows, blocks] of row images."""
    at = (H + 31) // 32 * 8
    return image[:, :H].view(_F8), image.view(torch.float32)[:, at:at + _blocks(H)]


def _prepare_norm(case, seed):
    g = _gen(seed, 4)
    T, H, dtype = case["T"], case["H"], _DT[case["dtype"]]
    # rows of a residual stream: some channels much larger than the others
    loud = torch.rand(H, generator=g, device="cuda") < 0.01
    size = torch.where(loud, 20.0, 1.0)
    st = {"case": case, "gamma": 1.0 + 0.2 * torch.randn(H, generator=g, device="cuda"),
          "status": torch.zeros(1, dtype=torch.int32, device="cuda")}
    x = _randn((T, H), dtype, g)
    x.mul_(size.to(dtype))
    if case["op"] == "norm_backward":
        st["x"], st["d_out"] = x, _randn((T, H), dtype, g, 0.1)
        st["d_sum"] = _randn((T, H), dtype, g, 0.1) if case["d_sum"] else None
        rstd = torch.empty(T, device="cuda")
        for part, to in zip(x.split(1 << 15), rstd.split(1 << 15)):
            to.copy_(1.0 / torch.sqrt((part.float() ** 2).mean(1) + _EPS))
        st["rstd"] = rstd
        st["d_x"] = torch.empty_like(x)
        st["d_gamma"] = torch.empty(H, device="cuda")
        return st
    st["x"] = x
    st["residual"] = _randn((T, H), dtype, g) if case["residual"] else None
    st["sum"] = torch.empty_like(x) if case["residual"] else None
    st["out"] = torch.empty_like(x) if case["out"] else None
    st["codes"] = torch.empty((T, _image_bytes(H)), dtype=torch.uint8,
                              device="cuda") if case["codes"] else None
    st["rstd"] = torch.empty(T, device="cuda") if case["rstd"] else None
    return st


def _prepare_swiglu(case, seed):
    g = _gen(seed, 5)
    rows, I = case["rows"], case["I"]
    h = _randn((rows, 2 * I), _DT[case["dtype"]], g, 1.5)
    return {"case": case, "h": h, "status": torch.zeros(1, dtype=torch.int32, device="cuda"),
            "codes": torch.empty((rows, _image_bytes(I)), dtype=torch.uint8, device="cuda")}


def _group_sizes(case, seed):
    G, rows = case["G"], case["rows"]
    rng = np.random.RandomState(seed % (1 << 31))
    p = np.ones(G) if case["spread"] == "even" else (np.arange(G) + 1.0) ** -1.0
    return rng.multinomial(rows, rng.permutation(p) / p.sum())


def _draw_image(rows, K, g):
    """Row images of normal values, as a norm leaves them."""
    image = torch.zeros((rows, _image_bytes(K)), dtype=torch.uint8, device="cuda")
    x = torch.randn((rows, K), generator=g, device="cuda")
    x = torch.nn.functional.pad(x, (0, -K % 128)).view(rows, _blocks(K), 128)
    scale = x.abs().amax(2) / 448
    q = (x / scale[:, :, None]).view(rows, -1)[:, :K].clamp(-448, 448).to(_F8)
    codes, scales = _codes(image, K)
    codes.view(torch.uint8).copy_(q.view(torch.uint8))
    scales.copy_(scale)
    return image


def _prepare_linear(case, seed):
    g = _gen(seed, 6)
    G, rows, N, K = (case[n] for n in ("G", "rows", "N", "K"))
    sizes = _group_sizes(case, seed)
    wide = (K + 15) // 16 * 16          # weight rows start on 16-byte boundaries
    w = torch.zeros((G, N, wide), dtype=torch.uint8, device="cuda")
    flat = w.view(G * N, wide)
    for part in flat.split(max(1, (1 << 29) // wide)):
        v = torch.randn((part.shape[0], K), generator=g, device="cuda") * 110.0
        part[:, :K] = v.clamp(-448, 448).to(_F8).view(torch.uint8)
    # the blocks' scales of a trained matrix lie within a few octaves
    w_scale = torch.exp2(torch.randn((G, _blocks(N), _blocks(K)), generator=g, device="cuda"))
    w_scale *= 1.0 / (110.0 * K ** 0.5)
    bias = torch.randn((G, N), generator=g, device="cuda") if case["bias"] else None
    off = np.concatenate([[0], np.cumsum(sizes)])
    return {"case": case, "a": _draw_image(rows, K, g), "w": w.view(_F8), "w_scale": w_scale,
            "bias": bias,
            "group_rows": torch.tensor(sizes, dtype=torch.int32, device="cuda"),
            "group_of": torch.tensor(np.repeat(np.arange(G), sizes), device="cuda"),
            "place": torch.tensor(np.arange(rows) - np.repeat(off[:-1], sizes), device="cuda"),
            "most": int(sizes.max()),
            "c": torch.empty((rows, N), dtype=_DT[case["out"]], device="cuda"),
            "status": torch.zeros(1, dtype=torch.int32, device="cuda")}


def prepare(case, seed):
    if case["op"] in ("norm", "norm_backward"):
        return _prepare_norm(case, seed)
    if case["op"] == "swiglu":
        return _prepare_swiglu(case, seed)
    return _prepare_linear(case, seed)


# ---- plain forms ---------------------------------------------------------------

def _plain_quant(y):
    """fp32 rows -> e4m3 codes and a scale per 128 values."""
    rows, H = y.shape
    parts = torch.nn.functional.pad(y, (0, -H % 128)).view(rows, _blocks(H), 128)
    scale = parts.abs().amax(2).clamp(min=_TINY) / 448
    codes = (parts / scale[:, :, None]).view(rows, -1)[:, :H].to(_F8)
    return [codes, scale]


def _plain_norm(st):
    case = st["case"]
    s = st["x"]
    outputs = []
    if case["residual"]:
        s = (s.float() + st["residual"].float()).to(s.dtype)
        outputs.append(s)
    v = s.float()
    rstd = 1.0 / torch.sqrt((v * v).sum(1) / case["H"] + _EPS)
    y = v * rstd[:, None] * st["gamma"]
    if case["out"]:
        outputs.append(y.to(s.dtype))
    if case["codes"]:
        outputs += _plain_quant(y)
    if case["rstd"]:
        outputs.append(rstd)
    return outputs


def _plain_norm_backward(st):
    v = st["x"].float() * st["rstd"][:, None]
    dy = st["d_out"].float()
    d_gamma = (dy * v).sum(0)
    a = dy * st["gamma"]
    d = (a - v * ((a * v).sum(1, keepdim=True) / st["case"]["H"])) * st["rstd"][:, None]
    if st["d_sum"] is not None:
        d = d + st["d_sum"].float()
    return [d.to(st["x"].dtype), d_gamma]


def _plain_swiglu(st):
    I = st["case"]["I"]
    gate, up = st["h"][:, :I].float(), st["h"][:, I:].float()
    return _plain_quant(gate / (1.0 + torch.exp(-gate)) * up)


def _plain_linear(st):
    case = st["case"]
    G, K, N = case["G"], case["K"], case["N"]
    codes, scale = _codes(st["a"], K)
    a = codes.float() * scale.repeat_interleave(128, 1)[:, :K]
    w = st["w"][:, :, :K].float()
    w *= st["w_scale"].repeat_interleave(128, 1)[:, :N].repeat_interleave(128, 2)[:, :, :K]
    if G == 1:
        c = a @ w[0].T
    else:   # every expert's rows in a block of its own, one batched product
        block = torch.zeros((G, st["most"], K), device=a.device)
        block[st["group_of"], st["place"]] = a
        c = torch.bmm(block, w.transpose(1, 2))[st["group_of"], st["place"]]
    if st["bias"] is not None:
        c = c + st["bias"][st["group_of"]]
    return c.to(_DT[case["out"]])


# ---- the framework's operators -----------------------------------------------------

def _own(st):
    import combine_moe_dispatch_layout_gb300 as ep
    case = st["case"]
    if case["op"] == "norm":
        ep.moe_rms_norm(st["x"], st["residual"], st["gamma"], _EPS, st["sum"], st["out"],
                        st["codes"], st["rstd"], st["status"])
        outputs = [t for t in (st["sum"], st["out"]) if t is not None]
        if case["codes"]:
            outputs += _codes(st["codes"], case["H"])
        return outputs + ([st["rstd"]] if case["rstd"] else [])
    if case["op"] == "norm_backward":
        if "workspace" not in st:       # made once and kept, as a training program would
            size = ep.rms_norm_backward_workspace_bytes(case["T"], case["H"])
            st["workspace"] = torch.empty(size, dtype=torch.uint8, device="cuda")
        ep.moe_rms_norm_backward(st["d_out"], st["x"], st["gamma"], st["rstd"], st["d_sum"],
                                 st["d_x"], st["d_gamma"], st["workspace"], st["status"])
        return [st["d_x"], st["d_gamma"]]
    if case["op"] == "swiglu":
        ep.moe_swiglu_f8(st["h"], None, st["codes"], st["status"])
        return list(_codes(st["codes"], case["I"]))
    a = st["a"]
    ep.moe_linear_f8(a, st["w"], case["K"], st["group_rows"] if case["G"] > 1 else None,
                     st["w_scale"], (a, (case["K"] + 31) // 32 * 32, a.shape[1]), st["bias"],
                     st["c"], st["status"])
    return st["c"]


def run(state):
    if own:
        return _own(state)
    return {"norm": _plain_norm, "norm_backward": _plain_norm_backward, "swiglu": _plain_swiglu,
            "linear": _plain_linear}[state["case"]["op"]](state)


# ---- the definitions in 64 bits -----------------------------------------------------

def _exact_quant(y):
    """Rows in 64 bits -> what the codes stand for before their rounding, and
    the scales."""
    codes = torch.empty_like(y)
    scale = torch.empty((y.shape[0], _blocks(y.shape[1])), dtype=torch.float64, device=y.device)
    for b in range(scale.shape[1]):
        part = y[:, 128 * b:128 * b + 128]
        scale[:, b] = torch.clamp(part.abs().max(dim=1).values, min=_TINY) / 448.0
        codes[:, 128 * b:128 * b + 128] = part / scale[:, b:b + 1]
    return [codes, scale]


def _exact_norm(case, st):
    s = st["x"].double()
    outputs = []
    if case["residual"]:
        s = (s + st["residual"].double()).to(st["x"].dtype).double()
        outputs.append(s)
    rstd = (torch.einsum("th,th->t", s, s) / case["H"] + _EPS) ** -0.5
    y = torch.einsum("th,t,h->th", s, rstd, st["gamma"].double())
    if case["out"]:
        outputs.append(y)
    if case["codes"]:
        outputs += _exact_quant(y)
    if case["rstd"]:
        outputs.append(rstd)
    return outputs


def _exact_norm_backward(case, st):
    """The Jacobian of y = s * rstd(s) * gamma applied to the rows' gradient:
    d rstd / d s_j = -rstd^3 s_j / H."""
    s, gamma, r = st["x"].double(), st["gamma"].double(), st["rstd"].double()
    dy = st["d_out"].double()
    d_gamma = torch.einsum("th,th,t->h", dy, s, r)
    g = dy * gamma
    along = torch.einsum("th,th->t", g, s) * r ** 3 / case["H"]
    d = g * r[:, None] - s * along[:, None]
    if st["d_sum"] is not None:
        d += st["d_sum"].double()
    return [d, d_gamma]


def _exact_swiglu(case, st):
    I = case["I"]
    outs = []
    for part in st["h"].split(1 << 15):
        gate, up = part[:, :I].double(), part[:, I:].double()
        e = torch.exp(-gate.abs())
        sig = torch.where(gate >= 0, 1.0, e) / (1.0 + e)
        outs.append(_exact_quant(gate * sig * up))
    return [torch.cat([o[i] for o in outs]) for i in range(2)]


def _exact_linear(case, st):
    G, rows, N, K = (case[n] for n in ("G", "rows", "N", "K"))
    sizes = st["group_rows"].tolist()
    c = torch.zeros((rows, N), dtype=torch.float64, device="cuda")
    codes, scale = _codes(st["a"], K)
    at = 0
    for g, n in enumerate(sizes):
        if n == 0:
            continue
        for b in range(_blocks(K)):
            k = slice(128 * b, min(K, 128 * b + 128))
            part = codes[at:at + n, k].double() @ st["w"][g, :, k].double().t()
            by = st["w_scale"][g, :, b].double().repeat_interleave(128)[:N]
            c[at:at + n] += part * scale[at:at + n, b:b + 1].double() * by
        if st["bias"] is not None:
            c[at:at + n] += st["bias"][g].double()
        at += n
    return c


def exact(case, seed):
    st = prepare(case, seed)
    return {"norm": _exact_norm, "norm_backward": _exact_norm_backward,
            "swiglu": _exact_swiglu, "linear": _exact_linear}[case["op"]](case, st)
