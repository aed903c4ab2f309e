"""Workloads of the operators around a mixture-of-experts block's products: norms, the router's gate, its balance
loss, and linear layers whose weights are held in four bits.

Each case is one pass through one operator.  ``run`` computes it in a plain
form (elementary torch operations in float32) or, where ``own`` is true, by
the calls that a training or serving program makes of the package.  Sizes are
those of the framework's own workloads (h = 4096 transformer matrices, the
[64, 1408, 2048] expert tensors) or generic.
"""

from __future__ import annotations

import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
ACTS = ("none", "relu", "silu", "gelu", "gelu_tanh")
DEV = "cuda"
BLOCK = 32  # values that share a scale in four bits


# ------------------------------------------------------------------ the cases


def _norm(name, dtype, rows, cols, kind, residual, train):
    return {"name": name, "op": "norm", "dtype": dtype, "rows": rows, "cols": cols, "kind": kind,
            "residual": residual, "train": train}


def _gate(name, dtype, tokens, e, top, normalize, pad, train):
    return {"name": name, "op": "gate", "dtype": dtype, "tokens": tokens, "e": e, "top": top, "normalize": normalize,
            "pad": pad, "train": train}


def _balance(name, dtype, tokens, e, top, pad):
    return {"name": name, "op": "balance", "dtype": dtype, "tokens": tokens, "e": e, "top": top, "pad": pad}


def _quantize(name, dtype, e, k, n, w_t):
    return {"name": name, "op": "quantize", "dtype": dtype, "e": e, "k": k, "n": n, "w_t": w_t}


def _mx(name, dtype, rows, e, k, n, act, bias, residual):
    return {"name": name, "op": "mx", "dtype": dtype, "rows": rows, "e": e, "k": k, "n": n, "act": act, "bias": bias,
            "residual": residual}


def listed():
    return [
        # One token of serving at h = 4096: the residual is added and the sum normalised; latency counts.
        _norm("norm_token", "bf16", 1, 4096, "layer", True, False),
        # Odd sizes in float32: a small probe trained in full precision.
        _norm("norm_odd_f32_train", "f32", 777, 1001, "rms", False, True),
        # The pre-norm of a block in one training step: forward, dx, dW, db, the residual stream's gradient joined.
        _norm("norm_train", "bf16", 16384, 4096, "layer", True, True),
        # 64 tokens of decoding choose 6 of 64 experts.
        _gate("gate_decode", "f32", 64, 64, 6, True, 0.0, False),
        # A training step's router: 16384 tokens, 8 of 64 experts, padding left out.
        _gate("gate_train", "bf16", 16384, 64, 8, False, 0.02, True),
        # The balance loss of a small odd batch, with its gradient.
        _balance("balance_odd", "f32", 5003, 24, 3, 0.1),
        # The balance loss of a large step over many experts.
        _balance("balance_train", "bf16", 65536, 256, 8, 0.02),
        # A probe head of odd sizes taken to four bits, its weight stored [n, k].
        _quantize("quantize_odd", "f32", 0, 1001, 1343, True),
        # The h = 4096 up-projection [h, 4h] taken to four bits for evaluation.
        _quantize("quantize_weight", "bf16", 0, 4096, 16384, False),
        # One token through the up-projection in four bits: the weight is read once.
        _mx("mx_token", "bf16", 1, 0, 4096, 16384, "gelu_tanh", True, False),
        # Evaluation of 8192 tokens through it.
        _mx("mx_eval", "bf16", 8192, 0, 4096, 16384, "gelu", True, True),
        # The experts in four bits: 8192 tokens, 6 of 64 experts a token, skewed loads.
        _mx("mx_experts", "bf16", 49152, 64, 2048, 1408, "silu", False, False),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _size(rng, lo, hi):
    """A size spread over the logarithm of the range: odd, or a multiple of 8 or of 64."""
    v = _log_int(rng, lo, hi)
    step = rng.choice((1, 8, 64))
    return max(lo, min(hi, v // step * step))


def draw(rng):
    op = rng.choice(("norm", "norm", "gate", "balance", "quantize", "mx", "mx"))
    dtype = rng.choice(("bf16", "bf16", "f32"))
    if op == "norm":
        c = _norm("", dtype, _size(rng, 1, 16384), _size(rng, 24, 8192), rng.choice(("layer", "rms")),
                  rng.random() < 0.5, rng.random() < 0.6)
    elif op in ("gate", "balance"):
        e = _log_int(rng, 8, 256)
        tokens, top, pad = _size(rng, 1, 65536), rng.randint(1, 8), rng.choice((0.0, 0.05))
        if op == "gate":
            c = _gate("", dtype, tokens, e, top, rng.random() < 0.5, pad, rng.random() < 0.6)
        else:
            c = _balance("", dtype, tokens, e, top, pad)
    elif op == "quantize":
        e = rng.choice((0, 0, _log_int(rng, 2, 16)))
        hi = 2048 if e else 8192
        c = _quantize("", dtype, e, _size(rng, 24, hi), _size(rng, 24, hi), rng.random() < 0.5)
    else:
        e = rng.choice((0, _log_int(rng, 2, 64)))
        rows, k, n = _size(rng, 1, 8192), _size(rng, 24, 2048 if e else 16384), _size(rng, 24, 2048 if e else 16384)
        while rows * k * n > 2 ** 38:  # at most half of the largest listed case
            rows = max(1, rows // 2)
        c = _mx("", dtype, rows, e, k, n, rng.choice(ACTS), rng.random() < 0.7, not e and rng.random() < 0.5)
    del c["name"]
    return c


# ------------------------------------------------------------------ inputs


def _normal(gen, shape, dtype, std=1.0):
    return (torch.randn(shape, generator=gen, device=DEV) * std).to(dtype)


def _hidden(gen, rows, cols, dtype):
    """Hidden states: tokens of unlike size, a few channels far above the others."""
    v = torch.randn(rows, cols, generator=gen, device=DEV) * torch.exp(
        0.5 * torch.randn(rows, 1, generator=gen, device=DEV))
    loud = torch.rand(cols, generator=gen, device=DEV) < 0.01
    return (v * torch.where(loud, 12.0, 1.0) + 0.1).to(dtype)


def _logits(gen, tokens, e, dtype):
    """A router's scores with a few favoured experts."""
    z = torch.randn(tokens, e, generator=gen, device=DEV) * 1.5 + torch.randn(e, generator=gen, device=DEV) * 0.5
    return z.to(dtype)


def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    dt = DTYPES[case["dtype"]]
    s = {"case": case}
    grads = ()
    if case["op"] == "norm":
        shape = (case["rows"], case["cols"])
        s["x"] = _hidden(gen, *shape, dt)
        s["r"] = _hidden(gen, *shape, dt) if case["residual"] else None
        s["w"] = _normal(gen, shape[1:], torch.float32, 0.2).add(1.0).to(dt)
        s["b"] = _normal(gen, shape[1:], dt, 0.2) if case["kind"] == "layer" else None
        if case["train"]:
            s["gy"] = _normal(gen, shape, dt)
            s["gs"] = _normal(gen, shape, dt) if case["residual"] else None
            grads = ("x", "w", "b")
    elif case["op"] in ("gate", "balance"):
        t, e = case["tokens"], case["e"]
        s["z"] = _logits(gen, t, e, dt)
        s["mask"] = torch.rand(t, generator=gen, device=DEV) >= case["pad"] if case["pad"] else None
        if case["op"] == "gate":
            s["gw"] = _normal(gen, (t, case["top"]), torch.float32) if case["train"] else None
        else:  # the choices that the gate made
            ids = torch.topk(s["z"].float(), case["top"], dim=1)[1].to(torch.int32)
            s["ids"] = ids if s["mask"] is None else torch.where(s["mask"][:, None], ids, -1)
            s["gl"] = torch.rand((), generator=gen, device=DEV) * 0.01 + 0.005  # the loss's share of the total
        grads = ("z",) if case.get("train", True) else ()
    else:
        e, k, n = case["e"], case["k"], case["n"]
        lead = (e,) if e else ()
        t = case.get("w_t", False)
        w = _normal(gen, (*lead, n, k) if t else (*lead, k, n), dt, k ** -0.5)
        s["w"] = w.transpose(-1, -2) if t else w
        if case["op"] == "mx":
            m = case["rows"]
            s["x"] = _hidden(gen, m, k, dt)
            s["b"] = _normal(gen, (*lead, n), dt, 0.5) if case["bias"] else None
            s["r"] = _normal(gen, (m, n), dt) if case["residual"] else None
            s["offsets"] = None
            if e:
                load = torch.softmax(torch.randn(e, generator=gen, device=DEV) * 0.5, 0)
                of = torch.multinomial(load, m, replacement=True, generator=gen)
                counts = (of[:, None] == torch.arange(e, device=DEV)).sum(0)
                s["offsets"] = torch.cat([counts.new_zeros(1), counts.cumsum(0)]).to(torch.int32)
                s["cap"] = int(counts.max())  # the plain form's padded rows an expert
            # The weight as a serving program keeps it: in four bits, or as the values they stand for.
            if own:
                import muon_newton_schulz_05_amd as muon
                s["wq"] = muon.mx_quantize(s["w"])
            else:
                s["wq"] = _plain_blocks(s["w"].float())
    for g in grads:  # the leaves of a training step
        if s.get(g) is not None:
            s[g].requires_grad_()
    return s


# ------------------------------------------------------------------ the plain forms


def _act(z, act):
    if act == "none":
        return z
    if act == "relu":
        return z * (z > 0)
    if act == "silu":
        return z / (1 + torch.exp(-z))
    if act == "gelu":
        return z * 0.5 * (1 + torch.erf(z * 0.5 ** 0.5))
    return 0.5 * z * (1 + torch.tanh((2 / math.pi) ** 0.5 * (z + 0.044715 * z * z * z)))


EPS = {"layer": 1e-5, "rms": 1e-6}


def _plain_norm(s, case):
    dt = DTYPES[case["dtype"]]
    h = s["x"].detach().float()
    out = {}
    if s["r"] is not None:
        h = h + s["r"].float()
        out["s"] = h.to(dt)
    w = s["w"].detach().float()
    c = h - h.mean(1, keepdim=True) if case["kind"] == "layer" else h
    rstd = ((c * c).mean(1, keepdim=True) + EPS[case["kind"]]) ** -0.5
    xhat = c * rstd
    y = xhat * w
    if s["b"] is not None:
        y = y + s["b"].detach().float()
    out["y"] = y.to(dt)
    if case["train"]:
        dy = s["gy"].float()
        g = dy * w
        dx = g - xhat * (g * xhat).mean(1, keepdim=True)
        if case["kind"] == "layer":
            dx = dx - g.mean(1, keepdim=True)
        dx = dx * rstd
        if s["gs"] is not None:
            dx = dx + s["gs"].float()
        out["dx"], out["dw"] = dx.to(dt), (dy * xhat).sum(0).to(dt)
        if s["b"] is not None:
            out["db"] = dy.sum(0).to(dt)
    return out


def _plain_gate(s, case):
    z, top = s["z"].detach().float(), case["top"]
    order = torch.sort(z, dim=1, descending=True, stable=True)[1][:, :top]  # ties: the lowest index first
    zs = torch.gather(z, 1, order)
    peak = zs[:, :1]
    part = torch.exp(zs - peak)
    whole = torch.exp(z - peak)
    total = (part if case["normalize"] else whole).sum(1, keepdim=True)
    w = part / total
    keep = torch.ones_like(w, dtype=torch.bool) if s["mask"] is None else s["mask"][:, None].expand_as(w)
    out = {"weights": torch.where(keep, w, 0.0), "ids": torch.where(keep, order, -1).to(torch.int32)}
    if case["train"]:
        dw = torch.where(keep, s["gw"], 0.0)
        mean = (w * dw).sum(1, keepdim=True)
        if case["normalize"]:
            dz = torch.zeros_like(z).scatter(1, order, w * (dw - mean))
        else:
            dz = (-whole / total * mean).scatter_add(1, order, w * dw)
        out["dz"] = dz.to(s["z"].dtype)
    return out


def _plain_balance(s, case):
    z, e = s["z"].detach().float(), case["e"]
    keep = torch.ones(len(z), device=z.device) if s["mask"] is None else s["mask"].float()
    p = torch.exp(z - z.max(1, keepdim=True)[0])
    p = p / p.sum(1, keepdim=True)
    counted = torch.where(keep[:, None] > 0, s["ids"], -1)
    counts = (counted[:, :, None] == torch.arange(e, device=z.device)).sum((0, 1)).double()
    tokens = keep.sum(dtype=torch.float64).clamp_min(1)  # counts pass 2^24
    f = (counts / (tokens * case["top"])).float()
    share = ((p * keep[:, None]).sum(0, dtype=torch.float64) / tokens).float()
    loss = e * (f * share).sum()
    slope = s["gl"] * e / tokens.float() * p * (f - (p * f).sum(1, keepdim=True)) * keep[:, None]
    return {"loss": loss, "counts": counts.to(torch.int32), "dz": slope.to(s["z"].dtype)}


def _plain_blocks(v):
    """v [..., K, N] float32 with each block of 32 along K taken to four bits: the values they stand for.

    A block's scale is 2^(floor(log2 of its largest magnitude) - 2), down to 2^-127; a value is the nearest of
    0, 0.5, 1, 1.5, 2, 3, 4, 6 in that scale (ties to the even code), 6 where it is larger."""
    k, n = v.shape[-2:]
    full = -(-k // BLOCK) * BLOCK
    b = torch.cat([v, v.new_zeros(*v.shape[:-2], full - k, n)], -2).reshape(*v.shape[:-2], full // BLOCK, BLOCK, n)
    exponent = torch.frexp(b.abs().amax(-2, keepdim=True))[1] - 3
    scale = torch.exp2(exponent.clamp_min(-127).double())
    a = b.abs().double() / scale  # in 64 bits: a small block's inverse scale passes 32
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
    q = (torch.round(a / step) * step).clamp_max(6.0) * torch.sign(b) * scale
    return q.float().reshape(*v.shape[:-2], full, n)[..., :k, :]


def _plain_quantize(s, case):
    return _plain_blocks(s["w"].float()).to(s["w"].dtype)


def _plain_mx(s, case):
    dt = DTYPES[case["dtype"]]
    x = _plain_blocks(s["x"].float().t()).t()
    if not case["e"]:
        z = x @ s["wq"]
        if s["b"] is not None:
            z = z + s["b"].float()
    else:
        off = s["offsets"].long()
        rows = torch.arange(case["rows"], device=x.device)
        of = torch.searchsorted(off[1:], rows, right=True)
        rank = rows - off[of]
        xp = x.new_zeros(case["e"], s["cap"], case["k"])
        xp[of, rank] = x
        z = torch.bmm(xp, s["wq"])
        if s["b"] is not None:
            z = z + s["b"].float()[:, None]
        z = z[of, rank]
    y = _act(z, case["act"])
    if s["r"] is not None:
        y = y + s["r"].float()
    return y.to(dt)


PLAIN = {"norm": _plain_norm, "gate": _plain_gate, "balance": _plain_balance, "quantize": _plain_quantize,
         "mx": _plain_mx}


# ------------------------------------------------------------------ the framework's calls


def _own_norm(s, case):
    import muon_newton_schulz_05_amd as muon
    if case["kind"] == "layer":
        got = muon.layer_norm(s["x"], s["w"], s["b"], eps=EPS["layer"], residual=s["r"])
    else:
        got = muon.rms_norm(s["x"], s["w"], eps=EPS["rms"], residual=s["r"])
    y, total = got if s["r"] is not None else (got, None)
    out = {} if total is None else {"s": total.detach()}
    out["y"] = y.detach()
    if case["train"]:
        leaves = {"dx": s["x"], "dw": s["w"]}
        if s["b"] is not None:
            leaves["db"] = s["b"]
        outs, seeds = ((y,), (s["gy"],)) if total is None else ((y, total), (s["gy"], s["gs"]))
        out.update(zip(leaves, torch.autograd.grad(outs, tuple(leaves.values()), seeds)))
    return out


def _own_gate(s, case):
    import muon_newton_schulz_05_amd as muon
    weights, ids = muon.gate(s["z"], case["top"], normalize=case["normalize"], mask=s["mask"])
    out = {"weights": weights.detach(), "ids": ids}
    if case["train"]:
        out["dz"], = torch.autograd.grad(weights, s["z"], s["gw"])
    return out


def _own_balance(s, case):
    import muon_newton_schulz_05_amd as muon
    loss, counts = muon.balance_loss(s["z"], s["ids"], mask=s["mask"])
    dz, = torch.autograd.grad(loss, s["z"], s["gl"])
    return {"loss": loss.detach(), "counts": counts, "dz": dz}


def _own_quantize(s, case):
    import muon_newton_schulz_05_amd as muon
    return muon.mx_dequantize(muon.mx_quantize(s["w"]), s["w"].dtype)


def _own_mx(s, case):
    import muon_newton_schulz_05_amd as muon
    if case["e"]:
        return muon.mx_expert_linear(s["x"], s["wq"], s["offsets"], s["b"], activation=case["act"])
    return muon.mx_linear(s["x"], s["wq"], s["b"], activation=case["act"], residual=s["r"])


OWN = {"norm": _own_norm, "gate": _own_gate, "balance": _own_balance, "quantize": _own_quantize, "mx": _own_mx}


def run(state):
    case = state["case"]
    return (OWN if own else PLAIN)[case["op"]](state, case)


# ------------------------------------------------------------------ what a pass cannot do without


def work(case):
    b = 2 if case["dtype"] == "bf16" else 4
    if case["op"] == "norm":
        n, c = case["rows"] * case["cols"], case["cols"]
        vectors = 2 if case["kind"] == "layer" else 1
        res, train = case["residual"], case["train"]
        els = n * (2 + 2 * res + train * (2 + res)) + c * vectors * (2 if train else 1)
        return {"bytes": b * els, "flops": n * (20 if train else 8)}
    if case["op"] == "gate":
        n, c = case["tokens"] * case["e"], case["tokens"] * case["top"]
        size = b * n + 8 * c + (case["tokens"] if case["pad"] else 0)
        if case["train"]:
            size += b * n + 4 * c
        return {"bytes": size, "flops": 4 * n * (2 if case["train"] else 1)}
    if case["op"] == "balance":
        n = case["tokens"] * case["e"]
        size = 2 * b * n + 4 * case["tokens"] * case["top"] + 4 * case["e"] + (case["tokens"] if case["pad"] else 0)
        return {"bytes": size, "flops": 10 * n}
    e, k, n = max(case["e"], 1), case["k"], case["n"]
    if case["op"] == "quantize":
        return {"bytes": 2 * b * e * k * n, "flops": 4 * e * k * n}
    m = case["rows"]
    met = min(e, m)  # an expert without rows is not read
    size = b * (m * k + m * n * (2 if case["residual"] else 1) + (met * n if case["bias"] else 0))
    return {"bytes": size + met * n * (-(-k // BLOCK)) * (BLOCK // 2 + 1), "flops": 2 * m * k * n}


# ------------------------------------------------------------------ 64 bits


def _exact_norm(s, case):
    x = s["x"].detach().double().requires_grad_()
    w = s["w"].detach().double().requires_grad_()
    b = None if s["b"] is None else s["b"].detach().double().requires_grad_()
    h = x if s["r"] is None else x + s["r"].double()
    if case["kind"] == "layer":
        var, mean = torch.var_mean(h, 1, correction=0, keepdim=True)
        y = (h - mean) / torch.sqrt(var + EPS["layer"]) * w + b
    else:
        y = h / torch.sqrt(h.square().mean(1, keepdim=True) + EPS["rms"]) * w
    out = {} if s["r"] is None else {"s": h.detach()}
    out["y"] = y.detach()
    if case["train"]:
        outs, seeds = ([y], [s["gy"].double()]) if s["r"] is None else ([y, h], [s["gy"].double(), s["gs"].double()])
        leaves = [x, w] if b is None else [x, w, b]
        out.update(zip(("dx", "dw", "db"), torch.autograd.grad(outs, leaves, seeds)))
    return out


def _exact_gate(s, case):
    z = s["z"].detach().double().requires_grad_()
    t, e, top = case["tokens"], case["e"], case["top"]
    # An expert's rank: how many are larger, or as large and before it.
    v, index = z.detach(), torch.arange(e, device=z.device)
    rank = torch.zeros(t, e, dtype=torch.int64, device=z.device)
    for j in range(e):
        ahead = (v[:, j:j + 1] > v) | ((v[:, j:j + 1] == v) & (j < index))
        rank += ahead
    ids = torch.full((t, top), -1, dtype=torch.int64, device=z.device)
    row, col = (rank < top).nonzero(as_tuple=True)
    ids[row, rank[row, col]] = col
    p = torch.softmax(z, 1)
    w = p.gather(1, ids)
    if case["normalize"]:
        w = w / w.sum(1, keepdim=True)
    if s["mask"] is not None:
        w = w * s["mask"].double()[:, None]
        ids = ids.masked_fill(~s["mask"][:, None], -1)
    out = {"weights": w.detach(), "ids": ids.to(torch.int32)}
    if case["train"]:
        out["dz"], = torch.autograd.grad(w, z, s["gw"].double())
    return out


def _exact_balance(s, case):
    z = s["z"].detach().double().requires_grad_()
    e = case["e"]
    keep = torch.arange(case["tokens"], device=z.device)
    if s["mask"] is not None:
        keep = keep[s["mask"]]
    flat = s["ids"][keep].reshape(-1).long()
    counts = torch.zeros(e, dtype=torch.int64, device=z.device).index_add(0, flat, torch.ones_like(flat))
    n = max(len(keep), 1)
    loss = e * (counts.double() / (n * case["top"]) * torch.softmax(z[keep], 1).sum(0) / n).sum()
    dz, = torch.autograd.grad(loss, z, s["gl"].double())
    return {"loss": loss.detach(), "counts": counts.to(torch.int32), "dz": dz}


def _exact_blocks(v):
    """Four bits along the last dimension, by counting the borders between neighbouring values that |v| passes."""
    k = v.shape[-1]
    v = torch.nn.functional.pad(v.double(), (0, -k % BLOCK)).unflatten(-1, (-1, BLOCK))
    peak = v.abs().max(-1, keepdim=True)[0]
    log = torch.floor(torch.log2(peak.clamp_min(2.0 ** -149)))
    log = torch.where(torch.exp2(log) > peak, log - 1, log)
    log = torch.where(torch.exp2(log + 1) <= peak, log + 1, log)
    scale = torch.exp2((log - 2).clamp_min(-127))
    a = v.abs() / scale
    values = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
    q = torch.zeros_like(a)
    for code in range(1, 8):
        border = (values[code - 1] + values[code]) / 2
        # A value on the border goes to the even code.
        q += (values[code] - values[code - 1]) * ((a >= border) if code % 2 == 0 else (a > border))
    return (torch.copysign(q, v) * scale).flatten(-2)[..., :k]


def _exact_mx(s, case):
    x = _exact_blocks(s["x"])

    def layer(x, w, b):
        z = x @ _exact_blocks(w.transpose(-1, -2)).t()
        if b is not None:
            z = z + b.double()
        if case["act"] == "relu":
            return z.clamp_min(0)
        if case["act"] == "silu":
            return z * torch.sigmoid(z)
        if case["act"] == "gelu":
            return z * torch.special.ndtr(z)
        if case["act"] == "gelu_tanh":
            return z * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3))
        return z

    if not case["e"]:
        y = layer(x, s["w"], s["b"])
        return y if s["r"] is None else y + s["r"].double()
    off = s["offsets"].tolist()
    return torch.cat([layer(x[lo:hi], s["w"][i], None if s["b"] is None else s["b"][i])
                      for i, (lo, hi) in enumerate(zip(off[:-1], off[1:]))])


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "norm":
        return _exact_norm(s, case)
    if case["op"] == "gate":
        return _exact_gate(s, case)
    if case["op"] == "balance":
        return _exact_balance(s, case)
    if case["op"] == "quantize":
        return _exact_blocks(s["w"].transpose(-1, -2)).transpose(-1, -2)
    return _exact_mx(s, case)
