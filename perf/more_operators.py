"""The operators between the products of a decoder layer, as their users call them.

  norm, norm_bwd      residual addition (with dropout of the branch that is added) and root-mean-square norm; the
                      output in the operands' type, or as e4m3 numbers with a scale for each row.
  dropout, dropout_bwd   with a counter-based generator, so that no mask is stored.
  linear, linear_bwd  matrix product with bias, activation and residual in its epilogue, and its gradients.
  linear8             the same on e4m3 numbers with a scale for each row of the activations and of the weights; the
                      activations' rows are quantised in the pass, the weights were when they were loaded.

`own` false: elementary torch operations.  `own` true: the library's entry points.
"""
import math

import torch

own = False

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32, "e4m3": torch.float8_e4m3fn}
EPS = 1e-6
SITE = 3  # which dropout of the model it is


# --------------------------------------------------------------------------- cases

def _norm(name, op, T, d, dtype="bf16", residual=True, p=0.0, out=None):
    return {"name": name, "op": op, "T": T, "d": d, "dtype": dtype, "residual": residual, "p": p, "out": out or dtype}


def _dropout(name, op, T, d, dtype="bf16", p=0.1, residual=False):
    return {"name": name, "op": op, "T": T, "d": d, "dtype": dtype, "p": p, "residual": residual}


def _linear(name, op, T, K, N, dtype="bf16", layout="in_out", act="none", bias=True, residual=False):
    return {"name": name, "op": op, "T": T, "K": K, "N": N, "dtype": dtype, "layout": layout, "act": act, "bias": bias,
            "residual": residual}


def listed():
    return [
        # a training batch or a long prompt: the residual stream joined and normalised in front of a product
        _norm("norm_T8192", "norm", 8192, 4096),
        # serving: one new token of each of 64 sequences, in front of an 8-bit product
        _norm("norm_e4m3_T64", "norm", 64, 4096, out="e4m3"),
        # the backward pass of the training batch, the branch behind dropout
        _norm("norm_bwd_T8192", "norm_bwd", 8192, 4096, p=0.1),
        # checked in full precision on a ragged batch and an odd width, without a residual
        _norm("norm_bwd_f32_odd", "norm_bwd", 1000, 1111, dtype="f32", residual=False),
        # dropout of an MLP's hidden activations
        _dropout("dropout_T8192", "dropout", 8192, 14336),
        # its backward on an odd tensor in full precision
        _dropout("dropout_bwd_f32_odd", "dropout_bwd", 1365, 1001, dtype="f32", p=0.25),
        # the first product of an MLP with biases, in training: the pre-activation is kept
        _linear("linear_T8192", "linear", 8192, 4096, 14336, act="gelu_tanh"),
        # serving one token: the product back into the residual stream
        _linear("linear_T1", "linear", 1, 14336, 4096, layout="out_in", residual=True),
        # the backward pass of the training product
        _linear("linear_bwd_T8192", "linear_bwd", 8192, 4096, 14336, act="gelu_tanh"),
        # the same checked in full precision, ragged
        _linear("linear_f32", "linear", 500, 1024, 4100, dtype="f32", layout="out_in", act="gelu"),
        # a long prompt through 8-bit weights
        _linear("linear8_T8192", "linear8", 8192, 4096, 14336, dtype="e4m3", layout="out_in", act="silu"),
        # one new token of each of 64 sequences through them, back into the residual stream
        _linear("linear8_T64", "linear8", 64, 14336, 4096, dtype="e4m3", layout="out_in", bias=False, residual=True),
    ]


def _span(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(("norm", "norm", "dropout", "linear", "linear", "linear8"))
    f32 = rng.random() < 0.25
    dtype = "f32" if f32 else "bf16"
    if kind in ("norm", "dropout"):
        d = _span(rng, 64, 4096)
        d = d if rng.random() < 0.3 else -(-d // 8) * 8
        T = min(_span(rng, 1, 8192), (16 << 20) // d)
        p = rng.choice((0.0, 0.1, 0.25)) if kind == "norm" else rng.choice((0.1, 0.25, 0.5))
        op = rng.choice((kind, kind + "_bwd"))
        case = {"op": op, "T": T, "d": d, "dtype": dtype, "residual": rng.random() < 0.7, "p": p}
        if kind == "norm":
            case["out"] = "e4m3" if op == "norm" and rng.random() < 0.4 else dtype
            case["p"] = p if case["residual"] else 0.0
        elif op == "dropout_bwd":
            case["residual"] = False
        return case
    layout = "out_in" if kind == "linear8" else rng.choice(("in_out", "out_in"))
    K = 16 * _span(rng, 8, 64 if f32 and kind == "linear" else 256)
    N = _span(rng, 100, 4100 if f32 and kind == "linear" else 14336)
    if layout == "in_out" or rng.random() < 0.6:
        N = -(-N // 8) * 8
    case = {"op": kind, "T": _span(rng, 1, 700 if f32 and kind == "linear" else 8192), "K": K, "N": N, "dtype": dtype,
            "layout": layout, "act": rng.choice(("none", "none", "gelu", "gelu_tanh", "silu")),
            "bias": rng.random() < 0.6, "residual": rng.random() < 0.5}
    if kind == "linear8":
        case["dtype"] = "e4m3"
    elif rng.random() < 0.4:
        case["op"], case["residual"] = "linear_bwd", False
    return case


# --------------------------------------------------------------------------- inputs

def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    s = {"case": case, "seed": (seed * 0x9e3779b97f4a7c15 + 12345) & 0x7fffffffffffffff}
    {"n": _prepare_norm, "d": _prepare_dropout, "l": _prepare_linear}[case["op"][0]](s, case, g)
    return s


def _randn(g, *shape):
    return torch.randn(*shape, device=DEV, generator=g)


def _prepare_norm(s, case, g):
    T, d, t = case["T"], case["d"], TYPES[case["dtype"]]
    s["w"] = (1.0 + 0.2 * _randn(g, d)).to(t)
    # the stream's rows differ in size, and a few of its channels stand out
    size = torch.exp(0.5 * _randn(g, T, 1)) * (1.0 + 10.0 * (torch.rand(d, device=DEV, generator=g) < 0.01))
    stream = (_randn(g, T, d) * size).to(t)
    if case["op"] == "norm":
        s["x"], s["res"] = (_randn(g, T, d).to(t), stream) if case["residual"] else (stream, None)
    else:
        s["h"] = stream
        s["rstd"] = (stream.float().square().mean(1) + EPS).rsqrt()
        s["dy"] = (_randn(g, T, d) * 0.01).to(t)
        s["dh"] = (_randn(g, T, d) * 0.01).to(t) if case["residual"] else None


def _prepare_dropout(s, case, g):
    T, d, t = case["T"], case["d"], TYPES[case["dtype"]]
    s["x"] = _randn(g, T, d).to(t)
    s["res"] = _randn(g, T, d).to(t) if case["residual"] else None


def _prepare_linear(s, case, g):
    T, K, N = case["T"], case["K"], case["N"]
    t = torch.bfloat16 if case["dtype"] == "e4m3" else TYPES[case["dtype"]]
    s["x"] = _randn(g, T, K).to(t)
    W = _randn(g, N, K) if case["layout"] == "out_in" else _randn(g, K, N)
    s["W"] = W.mul_(K ** -0.5).to(t)
    s["b"] = (_randn(g, N) * 0.5).to(t) if case["bias"] else None
    s["res"] = _randn(g, T, N).to(t) if case["residual"] else None
    if case["op"] == "linear_bwd":
        s["dy"] = _randn(g, T, N).to(t)
        s["pre"] = None
        if case["act"] != "none":
            z = s["x"].float() @ _in_out(s["W"], case).float()
            s["pre"] = (z if s["b"] is None else z + s["b"].float()).to(t)
    if case["op"] == "linear8":  # the weights as they were loaded
        s["W"], s["ws"] = _to_e4m3(s["W"].float())


# --------------------------------------------------------------------------- one pass

def run(s):
    case = s["case"]
    return {"norm": _run_norm, "norm_bwd": _run_norm_bwd, "dropout": _run_dropout, "dropout_bwd": _run_dropout,
            "linear": _run_linear, "linear_bwd": _run_linear_bwd, "linear8": _run_linear8}[case["op"]](s, case)


def _run_norm(s, case):
    if own:
        from backward_tcgen05_tma_gemms_gb300 import api
        y, scale, h, rstd = api.rmsnorm_fwd(s["x"], s["w"], residual=s["res"], eps=EPS, dropout=case["p"],
                                            seed=s["seed"], site=SITE, out_dtype=TYPES[case["out"]])
        return [x for x in (y, scale, h if s["res"] is not None else None, rstd) if x is not None]
    x = s["x"].float()
    if case["p"] > 0.0:
        x = x * _mask(x, case["p"], s["seed"])
    if s["res"] is not None:
        h = (x + s["res"].float()).to(s["res"].dtype)
        x = h.float()
    rstd = (x.square().mean(1) + EPS).rsqrt()
    y = x * s["w"].float()
    if case["out"] == "e4m3":  # the numbers do not depend on the norm, which all of a row shares
        q, scale = _to_e4m3(y)
        out = [q, scale * rstd]
    else:
        out = [(y * rstd[:, None]).to(TYPES[case["out"]])]
    return [*out, h, rstd] if s["res"] is not None else [*out, rstd]


def _run_norm_bwd(s, case):
    if own:
        from backward_tcgen05_tma_gemms_gb300 import api
        dx, dres, dw = api.rmsnorm_bwd(s["dy"], s["h"], s["w"], s["rstd"], dh=s["dh"], dropout=case["p"],
                                       seed=s["seed"], site=SITE)
        return [dx, dres, dw] if case["p"] > 0.0 else [dx, dw]
    n = s["h"].float() * s["rstd"][:, None]
    dy = s["dy"].float()
    dw = (dy * n).sum(0)
    g = dy * s["w"].float()
    d = (g - n * (g * n).mean(1, keepdim=True)) * s["rstd"][:, None]
    if s["dh"] is not None:
        d = d + s["dh"].float()
    if case["p"] > 0.0:
        return [(d * _mask(d, case["p"], s["seed"])).to(s["h"].dtype), d.to(s["h"].dtype), dw]
    return [d.to(s["h"].dtype), dw]


def _run_dropout(s, case):
    if own:
        from backward_tcgen05_tma_gemms_gb300 import api
        if case["op"] == "dropout_bwd":
            return [api.dropout_bwd(s["x"], case["p"], s["seed"], site=SITE)]
        return [api.dropout_fwd(s["x"], case["p"], s["seed"], site=SITE, residual=s["res"])]
    x = s["x"].float()
    x = x * _mask(x, case["p"], s["seed"])
    if s["res"] is not None:
        x = x + s["res"].float()
    return [x.to(s["x"].dtype)]


def _in_out(W, case):
    return W if case["layout"] == "in_out" else W.t()


def _act_name(case):
    return None if case["act"] == "none" else case["act"]


def _run_linear(s, case):
    keep = case["act"] != "none" and not case["residual"]  # training keeps the pre-activation
    if own:
        from backward_tcgen05_tma_gemms_gb300 import api
        y, pre = api.linear_fwd(s["x"], s["W"], bias=s["b"], residual=s["res"], act=_act_name(case),
                                weight_layout=case["layout"], want_pre=keep)
        return [y, pre] if keep else [y]
    z = s["x"].float() @ _in_out(s["W"], case).float()
    y = _finish(s, case, z)
    return [y.to(s["x"].dtype), z.to(s["x"].dtype)] if keep else [y.to(s["x"].dtype)]


def _finish(s, case, z):
    """Bias (into z), activation and residual."""
    if s["b"] is not None:
        z += s["b"].float()
    y = _act(z, case["act"])
    return y if s["res"] is None else y + s["res"].float()


def _run_linear_bwd(s, case):
    t = s["x"].dtype
    if own:
        from backward_tcgen05_tma_gemms_gb300 import api
        out = api.linear_bwd(s["x"], s["W"], s["dy"], pre=s["pre"], act=_act_name(case), weight_layout=case["layout"],
                             want_dbias=case["bias"], grad_dtype=t)
        return [x for x in out if x is not None]
    dz = s["dy"].float()
    if s["pre"] is not None:
        dz = dz * _act_slope(s["pre"].float(), case["act"])
    x, W = s["x"].float(), s["W"].float()
    if case["layout"] == "in_out":
        out = [(dz @ W.t()).to(t), (x.t() @ dz).to(t)]
    else:
        out = [(dz @ W).to(t), (dz.t() @ x).to(t)]
    return [*out, dz.sum(0).to(t)] if case["bias"] else out


def _run_linear8(s, case):
    if own:
        from backward_tcgen05_tma_gemms_gb300 import api
        q, scale = api.quantize_e4m3(s["x"])
        y, _ = api.linear_fwd(q, s["W"], bias=s["b"], residual=s["res"], act=_act_name(case), weight_layout="out_in",
                              x_scale=scale, w_scale=s["ws"], out_dtype=torch.bfloat16)
        return [q, scale, y]
    q, scale = _to_e4m3(s["x"].float())
    z = (q.float() @ s["W"].float().t()) * scale[:, None] * s["ws"]
    return [q, scale, _finish(s, case, z).to(torch.bfloat16)]


def _act(z, kind):
    if kind == "gelu":
        return 0.5 * z * (1.0 + torch.erf(z * math.sqrt(0.5)))
    if kind == "gelu_tanh":
        return 0.5 * z * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (z + 0.044715 * z * z * z)))
    if kind == "silu":
        return z / (1.0 + torch.exp(-z))
    return z


def _act_slope(z, kind):
    if kind == "gelu":
        return 0.5 * (1.0 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) * (1.0 / math.sqrt(2.0 * math.pi))
    if kind == "gelu_tanh":
        c = math.sqrt(2.0 / math.pi)
        t = torch.tanh(c * (z + 0.044715 * z * z * z))
        return 0.5 * (1.0 + t) + 0.5 * z * (1.0 - t * t) * c * (1.0 + 3 * 0.044715 * z * z)
    s = 1.0 / (1.0 + torch.exp(-z))
    return s + z * s * (1.0 - s)


def _to_e4m3(x):
    """e4m3 numbers and a scale for each row: the row's largest magnitude is 448.  Rows below 1e-30 are zeros.

    448 x / top as (7/8 x) / (top / 512): for bf16 values both are exact, so that ties are ties."""
    top = x.abs().amax(1)
    top = torch.where(top < 1e-30, torch.zeros_like(top), top)
    q = (x * 0.875) / torch.where(top > 0, top / 512, torch.full_like(top, math.inf))[:, None]
    return q.clamp(-448.0, 448.0).to(torch.float8_e4m3fn), top / 448


def _mask(x, p, seed):
    """0 or 1 / (1 - p) for each element of the rows x columns of x, with p in steps of 2^-16.

    Element i takes 16 bits of Philox 4x32-10 (Salmon, Moraes, Dror and Shaw, "Parallel random numbers: as easy as
    1, 2, 3", 2011) with key `seed` and counter (i // 8, site): the low and the high half of the words in turn."""
    n = x.numel()
    step = round(p * 65536)
    i = torch.arange(-(-n // 8), dtype=torch.int64, device=DEV)
    c0, c1 = i & 0xffffffff, i >> 32
    c2, c3 = torch.full_like(i, SITE & 0xffffffff), torch.full_like(i, SITE >> 32)
    k0, k1 = seed & 0xffffffff, (seed >> 32) & 0xffffffff
    for _ in range(10):
        a, b = c0 * 0xd2511f53, c2 * 0xcd9e8d57  # modulo 2^64
        c0, c1, c2, c3 = (((b >> 32) & 0xffffffff) ^ c1 ^ k0, b & 0xffffffff,
                          ((a >> 32) & 0xffffffff) ^ c3 ^ k1, a & 0xffffffff)
        k0, k1 = (k0 + 0x9e3779b9) & 0xffffffff, (k1 + 0xbb67ae85) & 0xffffffff
    u = torch.stack([h for c in (c0, c1, c2, c3) for h in (c & 0xffff, c >> 16)], 1).view(-1)[:n].view(x.shape)
    scale = 65536.0 / (65536 - step) if step < 65536 else 0.0
    return torch.where(u >= step, scale, 0.0)


# --------------------------------------------------------------------------- what a pass cannot do without

def work(case):
    op, T = case["op"], case["T"]
    if op[0] != "l":
        d, n = case["d"], T * case["d"]
        b = 2 if case["dtype"] == "bf16" else 4
        if op.startswith("dropout"):
            return {"bytes": (3 if case["residual"] else 2) * b * n, "flops": 2.0 * n}
        if op == "norm":
            out = 1 if case["out"] == "e4m3" else b
            return {"bytes": ((3 if case["residual"] else 1) * b + out) * n + b * d + 4 * T + (4 * T if out == 1 else 0),
                    "flops": 5.0 * n}
        tensors = 3 + (1 if case["residual"] else 0) + (1 if case["p"] > 0.0 else 0)
        return {"bytes": tensors * b * n + (b + 4) * d + 4 * T, "flops": 10.0 * n}
    K, N = case["K"], case["N"]
    if op == "linear8":
        return {"bytes": 2 * T * K + T * K + N * K + 4 * (T + N) + 2 * T * N * (2 if case["residual"] else 1)
                + (2 * N if case["bias"] else 0), "flops": 2.0 * T * K * N}
    b = 2 if case["dtype"] == "bf16" else 4
    acted = case["act"] != "none"
    if op == "linear_bwd":
        return {"bytes": b * (2 * T * K + 2 * K * N + (2 if acted else 1) * T * N + (N if case["bias"] else 0)),
                "flops": 4.0 * T * K * N}
    tensors = 2 if case["residual"] or acted else 1  # the output, and the residual or the pre-activation
    return {"bytes": b * (T * K + K * N + tensors * T * N + (N if case["bias"] else 0)), "flops": 2.0 * T * K * N}


# --------------------------------------------------------------------------- the definitions in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    return {"norm": _exact_norm, "norm_bwd": _exact_norm_bwd, "dropout": _exact_dropout, "dropout_bwd": _exact_dropout,
            "linear": _exact_linear, "linear_bwd": _exact_linear_bwd, "linear8": _exact_linear8}[case["op"]](s, case)


def _exact_kept(s, case):
    """The mask, its words from products of 16-bit halves."""
    T, d = case["T"], case["d"]
    step, seed = int(math.floor(case["p"] * 65536 + 0.5)), s["seed"]
    low = 0xffff
    i = torch.arange((T * d + 7) // 8, dtype=torch.int64, device=DEV)

    def times(x, m):  # (high, low) word of x m
        x0, x1, m0, m1 = x & low, x >> 16, m & low, m >> 16
        mid = x1 * m0 + ((x0 * m0) >> 16)
        other = x0 * m1 + (mid & low)
        return x1 * m1 + (mid >> 16) + (other >> 16), ((other & low) << 16) | ((x0 * m0) & low)

    ctr = [i & 0xffffffff, i >> 32, torch.zeros_like(i) + SITE, torch.zeros_like(i)]
    for r in range(10):
        key = [(seed % 2 ** 32 + r * 0x9e3779b9) % 2 ** 32, (seed // 2 ** 32 + r * 0xbb67ae85) % 2 ** 32]
        h0, l0 = times(ctr[0], 0xd2511f53)
        h2, l2 = times(ctr[2], 0xcd9e8d57)
        ctr = [h2 ^ ctr[1] ^ key[0], l2, h0 ^ ctr[3] ^ key[1], l0]
    bits = torch.empty(i.numel(), 8, dtype=torch.int64, device=DEV)
    for w in range(4):
        bits[:, 2 * w], bits[:, 2 * w + 1] = ctr[w] & low, ctr[w] >> 16
    kept = (bits.flatten()[:T * d] >= step).reshape(T, d)
    return kept.double() / (1.0 - step / 65536.0)


def _exact_dropout(s, case):
    y = s["x"].double() * _exact_kept(s, case)
    return [y + s["res"].double() if case["residual"] else y]


def _exact_norm(s, case):
    h = s["x"].double()
    if case["p"] > 0.0:
        h = h * _exact_kept(s, case)
    total = None
    if case["residual"]:
        total = h + s["res"].double()
        h = total.to(s["res"].dtype).double()  # the norm is that of the stored sum
    root = torch.sqrt(h.pow(2).sum(1) / case["d"] + EPS)
    out = [h / root[:, None] * s["w"].double()]
    if case["out"] == "e4m3":
        q, scale = _exact_codes(h * s["w"].double())
        out = [q, scale / root]
    return out + ([] if total is None else [total]) + [1.0 / root]


def _exact_codes(y):
    most = torch.linalg.vector_norm(y, ord=math.inf, dim=1)
    codes = (7.0 * y) / torch.where(most > 0, most / 64.0, torch.ones_like(most))[:, None]
    return [codes.float().clamp(-448, 448).to(torch.float8_e4m3fn).double(), most / 448.0]


def _exact_norm_bwd(s, case):
    h, dy, w = s["h"].double(), s["dy"].double(), s["w"].double()
    r = s["rstd"].double()[:, None]
    along = (dy * w * h).sum(1, keepdim=True)
    d = r * dy * w - r ** 3 * h * along / case["d"]
    if case["residual"]:
        d = d + s["dh"].double()
    dw = torch.einsum("td,td->d", dy, h * r)
    return [d * _exact_kept(s, case), d, dw] if case["p"] > 0.0 else [d, dw]


def _exact_act(z, kind):
    if kind == "gelu":
        return z * 0.5 * torch.erfc(-z / math.sqrt(2.0))
    if kind == "gelu_tanh":
        return z * torch.sigmoid(2.0 * math.sqrt(2.0 / math.pi) * (z + 0.044715 * z ** 3))
    return z * torch.sigmoid(z) if kind == "silu" else z


def _exact_after(s, case, z):
    if case["bias"]:
        z = z + s["b"].double()
    y = _exact_act(z, case["act"])
    return (y + s["res"].double() if case["residual"] else y), z


def _exact_linear(s, case):
    W = s["W"].double()
    z = torch.einsum("tk,kn->tn" if case["layout"] == "in_out" else "tk,nk->tn", s["x"].double(), W)
    y, z = _exact_after(s, case, z)
    return [y, z] if case["act"] != "none" and not case["residual"] else [y]


def _exact_linear8(s, case):
    q, scale = _exact_codes(s["x"].double())
    W = s["W"].double() * s["ws"].double()[:, None]
    y, _ = _exact_after(s, case, torch.einsum("tk,nk->tn", q * scale[:, None], W))
    return [q, scale, y]


def _exact_linear_bwd(s, case):
    dz = s["dy"].double()
    if case["act"] != "none":
        with torch.enable_grad():
            z = s["pre"].double().requires_grad_()
            slope, = torch.autograd.grad(_exact_act(z, case["act"]).sum(), z)
        dz = dz * slope
    x, W = s["x"].double(), s["W"].double()
    io = case["layout"] == "in_out"
    dx = torch.einsum("tn,kn->tk" if io else "tn,nk->tk", dz, W)
    dW = torch.einsum("tk,tn->kn" if io else "tk,tn->nk", x, dz)
    return [dx, dW, dz.sum(0)] if case["bias"] else [dx, dW]
