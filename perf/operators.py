"""The operators of a training step around this library's sharded products, as their users call them.

Three operators stand next to the projections, the MLP and the vocabulary cross-entropy of this library:

  ce_fwd, ce_bwd   softmax cross entropy of a language-model head, z = h W, taken in pieces of the vocabulary.
                   Only the log-sum-exp of each token is kept from the forward to the backward pass.
  rope, rope_bwd   rotary positions of the query and key heads between the QKV projections and attention.
  adamw            the update of all tensors of a model part in one call, with the gradient's global norm
                   clipped on the device, and with moments in 32 bits or in 8 (e4m3 with one scale for 256 elements).

`own` false: elementary torch operations.  `own` true: the library's entry points.
"""
import math

import torch

own = False

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
BLOCK = 256  # elements that share a scale of the 8-bit moments


# --------------------------------------------------------------------------- cases

def _ce(name, op, T, d, V, layout="in_out", dtype="bf16", reduction="mean", ignored=0.0, real=0):
    return {"name": name, "op": op, "T": T, "d": d, "V": V, "layout": layout, "dtype": dtype,
            "reduction": reduction, "ignored": ignored, "real": real}


def _rope(name, op, B, S, H, Hkv, D, rot, interleaved=False, scaling="none", factor=1.0, far=0, dtype="bf16",
          packed=False):
    return {"name": name, "op": op, "B": B, "S": S, "H": H, "Hkv": Hkv, "D": D, "rot": rot,
            "interleaved": interleaved, "scaling": scaling, "factor": factor, "far": far, "dtype": dtype,
            "packed": packed}


def _adamw(name, sizes, param, master, grad, state, clip=True):
    return {"name": name, "op": "adamw", "sizes": sizes, "param": param, "master": master, "grad": grad,
            "state": state, "clip": clip}


def listed():
    return [
        # evaluation and the forward half of training: the vocabulary head of the library's own benchmark
        _ce("ce_fwd_T8192", "ce_fwd", 8192, 4096, 128256),
        # the backward half of the same
        _ce("ce_bwd_T8192", "ce_bwd", 8192, 4096, 128256),
        # scoring one token
        _ce("ce_fwd_T1", "ce_fwd", 1, 4096, 128256, reduction="none"),
        # fine-tuning on a short ragged batch: nn.Linear's layout, an odd vocabulary, prompt tokens not supervised
        _ce("ce_bwd_T1000_odd", "ce_bwd", 1000, 2048, 32003, layout="out_in", ignored=0.3),
        # the same loss checked in full precision, a padded vocabulary and a gradient for each token
        _ce("ce_bwd_f32", "ce_bwd", 512, 1024, 8192, dtype="f32", reduction="none", real=8000),
        # a training batch's heads
        _rope("rope_T8192", "rope", 1, 8192, 32, 8, 128, 128),
        # serving: one new token of each of 64 sequences, far into a long context
        _rope("rope_decode64", "rope", 64, 1, 32, 8, 128, 128, scaling="yarn", factor=32.0, far=1 << 20),
        # backward of a part of the head, interleaved pairs, heads inside one packed QKV buffer, odd length
        _rope("rope_bwd_packed", "rope_bwd", 3, 1365, 16, 16, 96, 64, interleaved=True, scaling="linear",
              factor=4.0, packed=True),
        # the weights of one decoder layer, mixed precision: bf16 weights, fp32 master copy and moments
        _adamw("adamw_layer_f32", "layer", "bf16", True, "bf16", "f32"),
        # the same layer with 8-bit moments and no master copy (stochastic rounding)
        _adamw("adamw_layer_e4m3", "layer", "bf16", False, "bf16", "e4m3"),
        # many small and odd tensors (norms, biases, adapters), where launches and latency count
        _adamw("adamw_small", "small", "f32", False, "f32", "f32"),
        _adamw("adamw_adapters_e4m3", "adapters", "f32", False, "f32", "e4m3"),
    ]


def _span(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(("ce", "ce", "rope", "adamw"))
    if kind == "ce":
        f32 = rng.random() < 0.2
        layout = rng.choice(("in_out", "out_in"))
        d = 8 * _span(rng, 16, 192 if f32 else 512)
        V = _span(rng, 300, 12000 if f32 else 128256)
        if layout == "in_out":
            V = -(-V // 8) * 8
        T = _span(rng, 1, 700 if f32 else 8192)
        real = V - rng.randrange(1, 64) if rng.random() < 0.25 else 0
        return {"op": rng.choice(("ce_fwd", "ce_bwd")), "T": T, "d": d, "V": V, "layout": layout,
                "dtype": "f32" if f32 else "bf16", "reduction": rng.choice(("none", "sum", "mean")),
                "ignored": rng.choice((0.0, 0.0, 0.3)), "real": real}
    if kind == "rope":
        D = rng.choice((64, 80, 96, 128, 256))
        H = rng.choice((1, 4, 8, 12, 16, 32))
        B = _span(rng, 1, 64)
        return {"op": rng.choice(("rope", "rope_bwd")), "B": B, "S": _span(rng, 1, max(1, 8192 // B)), "H": H,
                "Hkv": rng.choice([n for n in (1, 2, 4, 8, 16) if H % n == 0 and n <= H]), "D": D,
                "rot": rng.choice((D, D, D // 2)), "interleaved": rng.random() < 0.5,
                "scaling": rng.choice(("none", "linear", "ntk", "yarn")), "factor": rng.choice((2.0, 4.0, 8.0)),
                "far": rng.choice((0, 0, 1 << 17, 1 << 20)), "dtype": rng.choice(("bf16", "bf16", "f32")),
                "packed": rng.random() < 0.5}
    param = rng.choice(("bf16", "f32"))
    return {"op": "adamw", "sizes": "%d x %d" % (_span(rng, 1, 200), _span(rng, 1, 1000000)), "param": param,
            "master": param == "bf16" and rng.random() < 0.5, "grad": param, "state": rng.choice(("f32", "e4m3")),
            "clip": rng.random() < 0.7}


def _sizes(case):
    """The tensors' element counts."""
    if case["sizes"] == "layer":  # d = 4096, F = 14336, 32 query and 8 KV heads of 128, two norms
        return [4096 * 4096, 4096 * 1024, 4096 * 1024, 4096 * 4096, 4096 * 14336, 4096 * 14336, 4096 * 14336,
                4096, 4096]
    if case["sizes"] == "small":
        return [1 + (i * 977) % 5000 for i in range(160)]
    if case["sizes"] == "adapters":
        return [16 * 4096, 16 * 1024, 16 * 14336] * 32 + [4097, 1, 255]
    n, most = (int(x) for x in case["sizes"].split(" x "))
    return [1 + (i * 7919 + most) % most for i in range(n)] if n * most <= 220000000 else [most]


def _starts(sizes):
    """Each tensor's place in the flat buffers: on whole blocks."""
    at = [0]
    for n in sizes:
        at.append(at[-1] + -(-n // BLOCK) * BLOCK)
    return at


# --------------------------------------------------------------------------- inputs

def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def prepare(case, seed):
    g = _gen(seed)
    if case["op"].startswith("ce"):
        return _prepare_ce(case, g)
    if case["op"].startswith("rope"):
        return _prepare_rope(case, g)
    return _prepare_adamw(case, g, seed)


def _ce_inputs(case, g):
    T, d, V, t = case["T"], case["d"], case["V"], TYPES[case["dtype"]]
    h = torch.randn(T, d, device=DEV, generator=g).to(t)
    W = torch.randn(d, V, device=DEV, generator=g).mul_(0.02).to(t)
    if case["layout"] == "out_in":
        W = W.t().contiguous()
    y = torch.randint(0, case["real"] or V, (T,), device=DEV, generator=g)
    y = torch.where(torch.rand(T, device=DEV, generator=g) < case["ignored"], torch.full_like(y, -100), y)
    up = torch.randn(T if case["reduction"] == "none" else 1, device=DEV, generator=g)
    return h, W, y, up


def _prepare_ce(case, g):
    h, W, y, up = _ce_inputs(case, g)
    s = {"case": case, "h": h, "W": W, "y": y, "up": up}
    if case["op"] == "ce_bwd":  # what the forward pass left
        V = case["real"] or case["V"]
        Wv = (W if case["layout"] == "in_out" else W.t())[:, :V].float()
        s["lse"] = torch.logsumexp(h.float() @ Wv, 1)
    return s


def _prepare_rope(case, g):
    B, S, H, Hkv, D, t = (case[k] for k in ("B", "S", "H", "Hkv", "D", "dtype"))
    t = TYPES[t]
    if case["packed"]:  # q, k and v side by side, as one projection leaves them
        x = torch.randn(B, S, H + 2 * Hkv, D, device=DEV, generator=g).to(t)
        q, k = x[:, :, :H], x[:, :, H:H + Hkv]
    else:
        q = torch.randn(B, S, H, D, device=DEV, generator=g).to(t)
        k = torch.randn(B, S, Hkv, D, device=DEV, generator=g).to(t)
    first = torch.randint(0, case["far"] + 1, (B, 1), device=DEV, generator=g)
    pos = (first + torch.arange(S, device=DEV)).to(torch.int64)
    s = {"case": case, "q": q, "k": k, "pos": pos}
    if own:
        from backward_tcgen05_tma_gemms_gb300 import api
        s["plan"] = api.rope_plan(case["rot"], base=10000.0, interleaved=case["interleaved"],
                                  scaling=case["scaling"], factor=case["factor"], original_context=4096)
    else:
        s["freq"], s["amp"] = _frequencies(case)
    return s


def _prepare_adamw(case, g, seed):
    sizes = _sizes(case)
    at = _starts(sizes)
    n = at[-1]
    live = torch.zeros(n, dtype=torch.bool, device=DEV)
    for a, m in zip(at, sizes):
        live[a:a + m] = True
    p32 = torch.randn(n, device=DEV, generator=g).mul_(0.02) * live
    # gradients of different tensors and rows differ by orders of magnitude
    mag = torch.exp(2.0 * torch.randn(n // BLOCK, device=DEV, generator=g)).repeat_interleave(BLOCK) * 1e-3
    grad = torch.randn(n, device=DEV, generator=g).mul_(mag) * live
    m = torch.randn(n, device=DEV, generator=g).mul_(mag * 0.3) * live
    v = (torch.rand(n, device=DEV, generator=g) + 0.1).mul_(mag).mul_(mag) * live
    s = {"case": case, "sizes": sizes, "at": at, "n": n, "step": 100, "seed": seed & 0x7fffffff}
    s["p"] = p32.to(TYPES[case["param"]])
    s["master"] = p32.clone() if case["master"] else None
    s["g"] = grad.to(TYPES[case["grad"]])
    if case["state"] == "e4m3":
        rnd = torch.full((n,), 0x8000, dtype=torch.int64, device=DEV)
        s["m"], s["ms"] = _to_e4m3(m, rnd, False)
        s["v"], s["vs"] = _to_e4m3(v.sqrt(), rnd, True)
    else:
        s["m"], s["v"], s["ms"], s["vs"] = m, v, None, None
    if own:
        from backward_tcgen05_tma_gemms_gb300 import api
        part = lambda x: None if x is None else [x[a:a + k] for a, k in zip(at, sizes)]  # noqa: E731
        blocks = lambda x: None if x is None else [x[a // BLOCK:b // BLOCK] for a, b in zip(at, at[1:])]  # noqa: E731
        s["plan"] = api.adamw_plan(part(s["p"]), master=part(s["master"]), m=part(s["m"]), v=part(s["v"]),
                                   m_scale=blocks(s["ms"]), v_scale=blocks(s["vs"]))
        s["grads"] = part(s["g"])
    return s


# --------------------------------------------------------------------------- one pass

HYPER = {"lr": 1e-3, "beta1": 0.9, "beta2": 0.95, "eps": 1e-8, "weight_decay": 0.1}


def run(s):
    case = s["case"]
    return {"ce_fwd": _run_ce_fwd, "ce_bwd": _run_ce_bwd, "rope": _run_rope, "rope_bwd": _run_rope,
            "adamw": _run_adamw}[case["op"]](s, case)


def _run_ce_fwd(s, case):
    if own:
        from backward_tcgen05_tma_gemms_gb300 import api
        loss, total, lse = api.linear_ce_fwd(s["h"], s["W"], s["y"], weight_layout=case["layout"], ignore_index=-100,
                                             vocab_size=case["real"], reduction=case["reduction"])
        return [loss, lse] if total is None else [loss, lse, total]
    z = _logits(s, case)
    m = z.amax(1, keepdim=True)
    lse = (m + (z - m).exp().sum(1, keepdim=True).log())[:, 0]
    kept = s["y"] != -100
    loss = torch.where(kept, lse - z.gather(1, s["y"].clamp(min=0)[:, None])[:, 0], 0.0)
    if case["reduction"] == "none":
        return [loss, lse]
    return [loss, lse, loss.sum() * _share(kept, case)]


def _logits(s, case):
    W = s["W"].float() if case["layout"] == "in_out" else s["W"].float().t()
    z = s["h"].float() @ W
    if case["real"]:
        z[:, case["real"]:] = -math.inf
    return z


def _share(kept, case):
    """What the sum of the losses is multiplied by."""
    return kept.sum().clamp(min=1).float().reciprocal() if case["reduction"] == "mean" else 1.0


def _run_ce_bwd(s, case):
    t = TYPES[case["dtype"]]
    if own:
        from backward_tcgen05_tma_gemms_gb300 import api
        return list(api.linear_ce_bwd(s["h"], s["W"], s["y"], s["lse"], grad_loss=s["up"], weight_layout=case["layout"],
                                      ignore_index=-100, vocab_size=case["real"], reduction=case["reduction"],
                                      grad_dtype=t))
    z = _logits(s, case)
    kept = s["y"] != -100
    dz = (z - s["lse"][:, None]).exp_()
    y = s["y"].clamp(min=0)[:, None]
    dz.scatter_(1, y, dz.gather(1, y) - 1.0)
    dz.mul_((torch.where(kept, s["up"], 0.0) * _share(kept, case))[:, None])
    dh = (dz @ (s["W"].float().t() if case["layout"] == "in_out" else s["W"].float())).to(t)
    dW = s["h"].float().t() @ dz if case["layout"] == "in_out" else dz.t() @ s["h"].float()
    return [dh, dW.to(t)]


def _run_rope(s, case):
    if own:
        from backward_tcgen05_tma_gemms_gb300 import api
        turn = api.rope_fwd if case["op"] == "rope" else api.rope_bwd
        return list(turn(s["plan"], s["q"], s["k"], s["pos"]))
    a = s["pos"].double()[..., None, None] * s["freq"]
    c, n = a.cos().float() * s["amp"], a.sin().float() * s["amp"]
    if case["op"] == "rope_bwd":
        n = -n
    return [_turned(s["q"], c, n, case), _turned(s["k"], c, n, case)]


def _turned(x, c, n, case):
    r, t = case["rot"], x.dtype
    u = x[..., :r].float()
    if case["interleaved"]:
        u = u.unflatten(-1, (r // 2, 2))
        a, b = u[..., 0], u[..., 1]
        u = torch.stack((a * c - b * n, b * c + a * n), -1).flatten(-2)
    else:
        a, b = u[..., :r // 2], u[..., r // 2:]
        u = torch.cat((a * c - b * n, b * c + a * n), -1)
    return torch.cat((u.to(t), x[..., r:]), -1)


def _frequencies(case, base=10000.0, context=4096.0):
    """Radians a position for each pair, and what the cosines and sines are multiplied by."""
    r, s, kind = case["rot"], case["factor"], case["scaling"]
    if kind == "ntk":
        base = base * s ** (r / (r - 2))
    f = base ** (-torch.arange(0, r, 2, dtype=torch.float64, device=DEV) / r)
    if kind == "linear":
        f = f / s
    if kind != "yarn":
        return f, 1.0
    at = lambda turns: r * math.log(context / (turns * 2 * math.pi)) / (2 * math.log(base))  # noqa: E731
    lo, hi = max(math.floor(at(32.0)), 0), min(math.ceil(at(1.0)), r - 1)
    ramp = ((torch.arange(r // 2, dtype=torch.float64, device=DEV) - lo) / max(hi - lo, 1e-3)).clamp(0, 1)
    return f / s * ramp + f * (1 - ramp), 0.1 * math.log(s) + 1.0


def _run_adamw(s, case):
    s["step"] += 1
    if own:
        from backward_tcgen05_tma_gemms_gb300 import api
        norm = api.grad_norm(s["grads"], max_norm=1.0) if case["clip"] else None
        api.adamw_step(s["plan"], s["grads"], step=s["step"], grad_scale=None if norm is None else norm[1:],
                       seed=s["seed"] + s["step"], **HYPER)
        return _adamw_outputs(s, None if norm is None else norm[0])
    g = s["g"].float()
    norm = g.square().sum().sqrt() if case["clip"] else None
    if case["clip"]:
        g = g * (1.0 / (norm + 1e-6)).clamp(max=1.0)
    lr, b1, b2, eps, wd = HYPER.values()
    if case["state"] == "e4m3":
        m, v = _from_e4m3(s["m"], s["ms"]), _from_e4m3(s["v"], s["vs"]).square()
    else:
        m, v = s["m"], s["v"]
    m = m * b1 + g * (1 - b1)
    v = v * b2 + g * g * (1 - b2)
    root = v.sqrt()
    p = s["p"].float() if s["master"] is None else s["master"]
    p = p * (1 - lr * wd) - m * (lr / (1 - b1 ** s["step"])) / (root * (1 - b2 ** s["step"]) ** -0.5 + eps)
    bits = _dither(s["n"], s["seed"] + s["step"])
    if case["state"] == "e4m3":
        (s["m"], s["ms"]), (s["v"], s["vs"]) = _to_e4m3(m, bits & 0xffff, False), _to_e4m3(root, bits >> 16, True)
    else:
        s["m"], s["v"] = m, v
    if s["master"] is not None:
        s["master"] = p
        s["p"] = p.to(torch.bfloat16)
    else:
        s["p"] = _to_bf16(p, _dither_again(bits)) if case["param"] == "bf16" else p
    return _adamw_outputs(s, norm)


def _adamw_outputs(s, norm):
    """The weights, the master copy and the moments (8-bit ones as the float8 numbers that they are, with their
    scales), and the gradient's norm."""
    return [x for x in (s["p"], s["master"], s["m"], s["v"], s["ms"], s["vs"], norm) if x is not None]


# 32 random bits for each element: its place in the plan and the step's seed, mixed by multiplications and shifts.
def _dither(n, seed):
    x = torch.arange(n, dtype=torch.int64, device=DEV)
    x = (((x & 0xffffffff) * 0x9e3779b1 + (x >> 32) * 0x85ebca77) & 0xffffffff) ^ (seed & 0xffffffff)
    x = ((x ^ (x >> 16)) * 0x2c1b3c6d) & 0xffffffff
    x = ((x ^ (x >> 12)) * 0x297a2d39) & 0xffffffff
    return x ^ (x >> 15)


def _dither_again(x):
    return ((x * 0x9e3779b1) & 0xffffffff) >> 16


def _from_e4m3(q, scale):
    return (q.float().view(-1, BLOCK) * scale[:, None]).view(-1)


def _to_e4m3(x, rnd, keep):
    """x in blocks as e4m3 numbers (values up to 448) and scales; each value goes up or down by 16 random bits.
    keep: what is not zero does not become zero."""
    x = x.view(-1, BLOCK)
    top = x.abs().amax(1)
    top = torch.where(top < 1e-30, torch.zeros_like(top), top)
    inv = torch.where(top > 0, 448.0 / top, torch.zeros_like(top))
    y = (x.abs() * inv[:, None]).clamp(max=448.0)
    rnd = rnd.view(-1, BLOCK)
    if x.dtype == torch.float32:
        big = ((y.view(torch.int32).to(torch.int64) + (rnd << 4)) >> 20) - 960
    else:  # 64 bits
        big = ((y.view(torch.int64) + (rnd << 33)) >> 49) - ((1023 - 7) << 3)
    code = torch.where(y >= 2.0 ** -6, big, (y * 512 + rnd.to(x.dtype) / 65536).floor().to(torch.int64))
    if keep:
        code = torch.where((y > 0) & (code == 0), torch.ones_like(code), code)
    code = code + 128 * ((x < 0) & (code > 0)).to(torch.int64)
    return code.to(torch.uint8).view(-1).view(torch.float8_e4m3fn), (top * (1.0 / 448)).float()


def _to_bf16(x, rnd):
    """fp32 to bf16, up or down by 16 random bits."""
    if x.dtype == torch.float64:
        x = x.float()
    return ((x.view(torch.int32).to(torch.int64) + rnd) >> 16).to(torch.int16).view(torch.bfloat16)


# --------------------------------------------------------------------------- what a pass cannot do without

def work(case):
    if case["op"].startswith("ce"):
        T, d, V = case["T"], case["d"], case["V"]
        b = 2 if case["dtype"] == "bf16" else 4
        if case["op"] == "ce_fwd":
            return {"bytes": b * (T * d + d * V) + 16 * T, "flops": 2.0 * T * d * V}
        return {"bytes": 2 * b * (T * d + d * V) + 16 * T, "flops": 6.0 * T * d * V}
    if case["op"].startswith("rope"):
        rows = case["B"] * case["S"]
        b = 2 if case["dtype"] == "bf16" else 4
        values = rows * (case["H"] + case["Hkv"]) * case["D"]
        return {"bytes": 2 * b * values + 8 * rows, "flops": 3.0 * values}
    n = sum(_sizes(case))
    b = {"bf16": 2, "f32": 4}
    per = b[case["grad"]] + 2 * b[case["param"]] - (2 if case["master"] else 0) + (8 if case["master"] else 0)
    per += 16 if case["state"] == "f32" else 4 + 16.0 / BLOCK
    return {"bytes": per * n, "flops": 20.0 * n}


# --------------------------------------------------------------------------- the definitions in 64 bits

def exact(case, seed):
    if case["op"].startswith("ce"):
        return _exact_ce(case, seed)
    if case["op"].startswith("rope"):
        return _exact_rope(case, seed)
    return _exact_adamw(case, seed)


def _exact_ce(case, seed):
    if case["T"] * case["d"] * case["V"] > 2.0e11:
        return None
    s = prepare(case, seed)
    T, V = case["T"], case["real"] or case["V"]
    W = (s["W"] if case["layout"] == "in_out" else s["W"].t()).double()
    h, y = s["h"].double(), s["y"]
    z = torch.matmul(h, W[:, :V])
    kept = (y >= 0).double()
    div = max(1.0, float(kept.sum())) if case["reduction"] == "mean" else 1.0
    if case["op"] == "ce_fwd":
        lse = torch.logsumexp(z, 1)
        loss = (lse - z[torch.arange(T, device=DEV), y.clamp(min=0)]) * kept
        return [loss, lse] if case["reduction"] == "none" else [loss, lse, loss.sum() / div]
    dz = torch.zeros(T, case["V"], dtype=torch.float64, device=DEV)
    dz[:, :V] = torch.exp(z - s["lse"].double()[:, None])
    dz[torch.arange(T, device=DEV), y.clamp(min=0)] -= 1.0
    dz *= (kept * s["up"].double() / div)[:, None]
    dW = torch.matmul(h.t(), dz)
    return [torch.matmul(dz, W.t()), dW if case["layout"] == "in_out" else dW.t()]


def _exact_rope(case, seed):
    s = prepare(case, seed)
    r, kind, f = case["rot"], case["scaling"], case["factor"]
    amp = 0.1 * math.log(f) + 1.0 if kind == "yarn" else 1.0
    base = 10000.0 * f ** (r / (r - 2)) if kind == "ntk" else 10000.0
    freq = []
    for i in range(r // 2):
        w = base ** (-2.0 * i / r)
        if kind == "linear":
            w /= f
        elif kind == "yarn":
            lo = max(math.floor(r / 2 * math.log(4096 / (2 * math.pi * 32)) / math.log(base)), 0)
            hi = min(math.ceil(r / 2 * math.log(4096 / (2 * math.pi)) / math.log(base)), r - 1)
            t = min(1.0, max(0.0, (i - lo) / max(hi - lo, 1e-3)))
            w = w * (1 - t) + w / f * t
        freq.append(w)
    a = s["pos"].double()[..., None] * torch.tensor(freq, dtype=torch.float64, device=DEV)
    e = torch.polar(torch.full_like(a, amp), a if case["op"] == "rope" else -a)[:, :, None]
    out = []
    for x in (s["q"], s["k"]):
        y = x.double().contiguous()
        u = y[..., :r]
        pairs = u.reshape(*u.shape[:-1], r // 2, 2) if case["interleaved"] else u.reshape(*u.shape[:-1], 2, r // 2).transpose(-1, -2)
        z = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * e)
        y[..., :r] = z.flatten(-2) if case["interleaved"] else z.transpose(-1, -2).flatten(-2)
        out.append(y)
    return out


def _exact_adamw(case, seed):
    s = prepare(case, seed)
    g = s["g"].double()
    norm = torch.linalg.vector_norm(g)
    if case["clip"]:
        g = g * min(1.0, 1.0 / (float(norm) + 1e-6))
    step = s["step"] + 1
    if case["state"] == "e4m3":
        m = s["m"].double() * s["ms"].double().repeat_interleave(BLOCK)
        v = (s["v"].double() * s["vs"].double().repeat_interleave(BLOCK)) ** 2
    else:
        m, v = s["m"].double(), s["v"].double()
    m = 0.9 * m + (1 - 0.9) * g
    v = 0.95 * v + (1 - 0.95) * g ** 2
    p = (s["p"] if s["master"] is None else s["master"]).double()
    p = p - 1e-3 * 0.1 * p - 1e-3 * (m / (1 - 0.9 ** step)) / (torch.sqrt(v / (1 - 0.95 ** step)) + 1e-8)
    out = [p] if s["master"] is None else [p, p]
    if case["state"] == "e4m3":
        bits = _dither(s["n"], s["seed"] + step)
        qm, ms = _to_e4m3(m, bits & 0xffff, False)
        qv, vs = _to_e4m3(torch.sqrt(v), bits >> 16, True)
        out += [qm.double(), qv.double(), ms.double(), vs.double()]
    else:
        out += [m, v]
    return out + ([norm] if case["clip"] else [])
