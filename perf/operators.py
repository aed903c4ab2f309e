"""Workloads of the layer operators that feed the Muon step: fused linear layers, routed experts, dropout.

Each case is one pass through one operator.  ``run`` computes it in a plain
form (elementary torch operations in float32) or, where ``own`` is true, by
the calls that a training or serving program makes of the package.  Sizes are
those of the framework's own workloads (h = 4096 transformer matrices, the
[64, 1408, 2048] and [32, 24, 10240] expert tensors) or generic.
"""

from __future__ import annotations

import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
ACTS = ("none", "relu", "silu", "gelu", "gelu_tanh")
DEV = "cuda"


# ------------------------------------------------------------------ the cases


def _linear(name, dtype, rows, k, n, act, train, bias=True, residual=False, w_t=False):
    return {"name": name, "op": "linear", "dtype": dtype, "rows": rows, "k": k, "n": n, "act": act, "train": train,
            "bias": bias, "residual": residual, "w_t": w_t}


def _experts(name, dtype, rows, e, k, n, act, train, bias=True):
    return {"name": name, "op": "experts", "dtype": dtype, "rows": rows, "e": e, "k": k, "n": n, "act": act,
            "train": train, "bias": bias}


def _route(name, dtype, tokens, top, e, h, train, drop=0.0):
    return {"name": name, "op": "route", "dtype": dtype, "tokens": tokens, "top": top, "e": e, "h": h,
            "train": train, "drop": drop}


def _dropout(name, dtype, rows, cols, p, residual, train):
    return {"name": name, "op": "dropout", "dtype": dtype, "rows": rows, "cols": cols, "p": p, "residual": residual,
            "train": train}


def listed():
    return [
        # One token through the h = 4096 up-projection [h, 4h]: the weight is read once and latency counts.
        _linear("linear_token", "bf16", 1, 4096, 16384, "gelu_tanh", False),
        # A block's down-projection [4h, h] with the residual stream added, forward only (evaluation).
        _linear("linear_down_residual", "bf16", 2048, 16384, 4096, "none", False, residual=True),
        # The up-projection of one training step: forward, dx, dW, db.
        _linear("linear_up_train", "bf16", 8192, 4096, 16384, "gelu", True),
        # Odd sizes in float32, a weight stored [n, k]: a small probe head trained in full precision.
        _linear("linear_odd_f32_train", "f32", 777, 1001, 1343, "silu", True, residual=True, w_t=True),
        # 32 tokens of decoding over 64 experts of [2048, 1408], 6 experts a token: a few rows an expert.
        _experts("experts_decode", "bf16", 192, 64, 2048, 1408, "silu", False),
        # A training step of the same experts: 8192 tokens, 6 experts a token, skewed loads.
        _experts("experts_train", "bf16", 49152, 64, 2048, 1408, "silu", True),
        # The thin [32, 24, 10240] experts (low-rank adapters): a contraction of 24.
        _experts("experts_thin_train", "bf16", 8192, 32, 24, 10240, "none", True, bias=False),
        # 64 tokens of decoding sorted to 64 experts and back.
        _route("route_decode", "bf16", 64, 6, 64, 2048, False),
        # Odd sizes in float32 with entries over an expert's capacity dropped.
        _route("route_odd_f32_train", "f32", 5003, 3, 24, 1000, True, drop=0.1),
        # A training step's 16384 tokens, 8 experts a token.
        _route("route_train", "bf16", 16384, 8, 64, 2048, True),
        # A short odd activation in float32.
        _dropout("dropout_odd_f32", "f32", 7, 1001, 0.1, False, False),
        # Residual dropout of a training step's activations at h = 4096.
        _dropout("dropout_train", "bf16", 16384, 4096, 0.1, True, True),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _size(rng, lo, hi):
    """A size spread over the logarithm of the range: odd, or a multiple of 8 or of 64."""
    v = _log_int(rng, lo, hi)
    step = rng.choice((1, 8, 64))
    return max(lo, min(hi, v // step * step))


def draw(rng):
    op = rng.choice(("linear", "linear", "experts", "experts", "route", "dropout"))
    dtype = rng.choice(("bf16", "bf16", "f32"))
    train = rng.random() < 0.6
    if op == "linear":
        rows, k, n = _size(rng, 1, 8192), _size(rng, 24, 16384), _size(rng, 24, 16384)
        while rows * k * n > 2 ** 38:  # at most half of the largest listed case
            rows = max(1, rows // 2)
        c = _linear("", dtype, rows, k, n, rng.choice(ACTS), train, rng.random() < 0.7, rng.random() < 0.5,
                    rng.random() < 0.5)
    elif op == "experts":
        e, k, n = _log_int(rng, 2, 64), _size(rng, 24, 2048), _size(rng, 24, 2048)
        c = _experts("", dtype, _size(rng, 1, 32768), e, k, n, rng.choice(ACTS), train, rng.random() < 0.7)
    elif op == "route":
        c = _route("", dtype, _size(rng, 1, 16384), rng.randint(1, 8), _log_int(rng, 8, 256), _size(rng, 24, 2048),
                   train, rng.choice((0.0, 0.1)))
    else:
        c = _dropout("", dtype, _size(rng, 1, 16384), _size(rng, 24, 4096), round(rng.uniform(0.02, 0.5), 3),
                     rng.random() < 0.5, train)
    del c["name"]
    return c


# ------------------------------------------------------------------ inputs


def _normal(gen, shape, dtype, std=1.0):
    return (torch.randn(shape, generator=gen, device=DEV) * std).to(dtype)


def _top_experts(gen, tokens, top, e):
    """A router's choice: the `top` largest of noisy scores with a few favoured experts, and their weights."""
    scores = torch.randn(tokens, e, generator=gen, device=DEV) + torch.randn(e, generator=gen, device=DEV) * 0.5
    val, ids = torch.topk(scores, top, dim=1)
    return ids, torch.softmax(val, 1)


def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    dt = DTYPES[case["dtype"]]
    s = {"case": case}
    if case["op"] == "linear":
        m, k, n = case["rows"], case["k"], case["n"]
        s["x"] = _normal(gen, (m, k), dt)
        w = _normal(gen, (n, k) if case["w_t"] else (k, n), dt, k ** -0.5)
        s["w"] = w.t() if case["w_t"] else w
        s["b"] = _normal(gen, (n,), dt, 0.5) if case["bias"] else None
        s["r"] = _normal(gen, (m, n), dt) if case["residual"] else None
        s["gy"] = _normal(gen, (m, n), dt) if case["train"] else None
        grads = ("x", "w", "b")
    elif case["op"] == "experts":
        p, e, k, n = case["rows"], case["e"], case["k"], case["n"]
        load = torch.softmax(torch.randn(e, generator=gen, device=DEV) * 0.5, 0)
        ids = torch.multinomial(load, p, replacement=True, generator=gen)
        counts = (ids[:, None] == torch.arange(e, device=DEV)).sum(0)
        s["offsets"] = torch.cat([counts.new_zeros(1), counts.cumsum(0)]).to(torch.int32)
        s["cap"] = int(counts.max())  # the plain form's padded rows an expert
        s["x"] = _normal(gen, (p, k), dt)
        s["w"] = _normal(gen, (e, k, n), dt, k ** -0.5)
        s["b"] = _normal(gen, (e, n), dt, 0.5) if case["bias"] else None
        s["gy"] = _normal(gen, (p, n), dt) if case["train"] else None
        grads = ("x", "w", "b")
    elif case["op"] == "route":
        t, top, h = case["tokens"], case["top"], case["h"]
        ids, s["weights"] = _top_experts(gen, t, top, case["e"])
        lost = torch.rand(t, top, generator=gen, device=DEV) < case["drop"]
        s["ids"] = torch.where(lost, torch.full_like(ids, -1), ids)
        s["x"] = _normal(gen, (t, h), dt)
        s["ys"] = _normal(gen, (t * top, h), dt)
        s["gy"] = _normal(gen, (t, h), dt) if case["train"] else None
        s["gxs"] = _normal(gen, (t * top, h), dt) if case["train"] else None
        grads = ("x", "ys", "weights")
    else:
        shape = (case["rows"], case["cols"])
        s["x"] = _normal(gen, shape, dt)
        s["r"] = _normal(gen, shape, dt) if case["residual"] else None
        s["gy"] = _normal(gen, shape, dt) if case["train"] else None
        s["seed"], s["offset"] = seed * 2654435761 % (1 << 62), seed % 1000
        grads = ("x",)
    if case["train"]:  # the leaves of a training step
        for g in grads:
            if s.get(g) is not None:
                s[g].requires_grad_()
    return s


# ------------------------------------------------------------------ the plain forms


def _act(z, act):
    """act(z) and its derivative."""
    if act == "none":
        return z, torch.ones_like(z)
    if act == "relu":
        on = (z > 0).to(z.dtype)
        return z * on, on
    if act == "silu":
        q = 1 / (1 + torch.exp(-z))
        return z * q, q * (1 + z * (1 - q))
    if act == "gelu":
        cdf = 0.5 * (1 + torch.erf(z * 0.5 ** 0.5))
        return z * cdf, cdf + z * torch.exp(-0.5 * z * z) * (2 * math.pi) ** -0.5
    c = (2 / math.pi) ** 0.5
    th = torch.tanh(c * (z + 0.044715 * z * z * z))
    return 0.5 * z * (1 + th), 0.5 * (1 + th) + 0.5 * z * (1 - th * th) * c * (1 + 3 * 0.044715 * z * z)


def _plain_linear(s, case):
    dt = DTYPES[case["dtype"]]
    x, w = s["x"].detach().float(), s["w"].detach().float()
    z = x @ w
    if s["b"] is not None:
        z = z + s["b"].detach().float()
    y, slope = _act(z, case["act"])
    if s["r"] is not None:
        y = y + s["r"].float()
    out = {"y": y.to(dt)}
    if case["train"]:
        dz = s["gy"].float() * slope
        out["dx"], out["dw"] = (dz @ w.t()).to(dt), (x.t() @ dz).to(dt)
        if s["b"] is not None:
            out["db"] = dz.sum(0).to(dt)
    return out


def _plain_experts(s, case):
    dt = DTYPES[case["dtype"]]
    p, e, k, n = case["rows"], case["e"], case["k"], case["n"]
    x, w, off = s["x"].detach().float(), s["w"].detach().float(), s["offsets"].long()
    rows = torch.arange(p, device=x.device)
    of = torch.searchsorted(off[1:], rows, right=True)
    rank = rows - off[of]
    xp = x.new_zeros(e, s["cap"], k)
    xp[of, rank] = x
    z = torch.bmm(xp, w)
    if s["b"] is not None:
        z = z + s["b"].detach().float()[:, None]
    y, slope = _act(z, case["act"])
    out = {"y": y[of, rank].to(dt)}
    if case["train"]:
        dz = torch.zeros_like(z)
        dz[of, rank] = s["gy"].float()
        dz = dz * slope
        out["dx"] = torch.bmm(dz, w.transpose(1, 2))[of, rank].to(dt)
        out["dw"] = torch.bmm(xp.transpose(1, 2), dz).to(dt)
        if s["b"] is not None:
            out["db"] = dz.sum(1).to(dt)
    return out


def _plain_route(s, case):
    dt = DTYPES[case["dtype"]]
    t, top, e, h = case["tokens"], case["top"], case["e"], case["h"]
    ids = s["ids"].reshape(-1)
    routed = ids >= 0
    key = torch.where(routed, ids, torch.full_like(ids, e))
    order = torch.sort(key, stable=True)[1]
    counts = (key[:, None] == torch.arange(e, device=key.device)).sum(0)
    offsets = torch.cat([counts.new_zeros(1), counts.cumsum(0)])
    position = torch.empty_like(order)
    position[order] = torch.arange(t * top, device=order.device)
    used = routed[order][:, None]
    token = torch.div(order, top, rounding_mode="floor")
    x, ys, w = s["x"].detach().float(), s["ys"].detach().float(), s["weights"].detach()
    keep = routed.reshape(t, top, 1)
    back = torch.where(keep, ys[position].reshape(t, top, h), torch.zeros((), device=x.device))
    out = {"offsets": offsets.to(torch.int32),
           "order": torch.where(routed[order], order, torch.full_like(order, -1)).to(torch.int32),
           "position": torch.where(routed, position, torch.full_like(position, -1)).reshape(t, top).to(torch.int32),
           "xs": torch.where(used, x[token], torch.zeros((), device=x.device)).to(dt),
           "y": (w[:, :, None] * back).sum(1).to(dt)}
    if case["train"]:
        gy, gxs = s["gy"].float(), s["gxs"].float()
        out["dx"] = torch.where(keep, gxs[position].reshape(t, top, h), torch.zeros((), device=x.device)).sum(1).to(dt)
        flat = w.reshape(-1)[order][:, None]
        out["dys"] = torch.where(used, flat * gy[token], torch.zeros((), device=x.device)).to(dt)
        out["dweights"] = (gy[:, None] * back).sum(2)
    return out


M32 = 0xFFFFFFFF


def _philox(seed, offset, blocks, device):
    """Philox4x32 with 10 rounds (Salmon et al., "Parallel random numbers: as easy as 1, 2, 3", 2011): one 128-bit
    word a block, counter (block, offset), key `seed`, in 64-bit integers."""
    i = torch.arange(blocks, device=device)
    c0, c1 = i & M32, i >> 32
    c2, c3 = torch.full_like(i, offset & M32), torch.full_like(i, offset >> 32 & M32)
    k0, k1 = seed & M32, seed >> 32 & M32
    for _ in range(10):
        a, b = c0 * 0xD2511F53, c2 * 0xCD9E8D57
        c0, c1, c2, c3 = ((b >> 32) & M32) ^ c1 ^ k0, b & M32, ((a >> 32) & M32) ^ c3 ^ k1, a & M32
        k0, k1 = (k0 + 0x9E3779B9) & M32, (k1 + 0xBB67AE85) & M32
    return torch.stack([c0, c1, c2, c3], 1)


def _plain_dropout(s, case):
    dt = DTYPES[case["dtype"]]
    x = s["x"].detach().float()
    n = x.numel()
    words = _philox(s["seed"], s["offset"], (n + 7) // 8, x.device)
    lanes = torch.stack([words & 0xFFFF, words >> 16], 2).reshape(-1)[:n].reshape(x.shape)
    d = int(round(case["p"] * 65536))
    factor = (lanes >= d).float() * (65536.0 / (65536 - d))
    y = x * factor
    if s["r"] is not None:
        y = y + s["r"].float()
    out = {"y": y.to(dt)}
    if case["train"]:
        out["dx"] = (s["gy"].float() * factor).to(dt)
    return out


PLAIN = {"linear": _plain_linear, "experts": _plain_experts, "route": _plain_route, "dropout": _plain_dropout}


# ------------------------------------------------------------------ the framework's calls


def _own_linear(s, case):
    import muon_newton_schulz_05_amd as muon
    y = muon.linear(s["x"], s["w"], s["b"], activation=case["act"], residual=s["r"])
    return _with_grads(y, s, case, {"dx": s["x"], "dw": s["w"], "db": s["b"]})


def _own_experts(s, case):
    import muon_newton_schulz_05_amd as muon
    y = muon.expert_linear(s["x"], s["w"], s["offsets"], s["b"], activation=case["act"])
    return _with_grads(y, s, case, {"dx": s["x"], "dw": s["w"], "db": s["b"]})


def _own_route(s, case):
    import muon_newton_schulz_05_amd as muon
    r = muon.route(s["ids"], case["e"])
    xs = muon.dispatch(s["x"], r)
    y = muon.combine(s["ys"], r, s["weights"])
    out = {"offsets": r.offsets, "order": r.order, "position": r.position, "xs": xs.detach(), "y": y.detach()}
    if case["train"]:
        out["dx"], out["dys"], out["dweights"] = torch.autograd.grad(
            (xs, y), (s["x"], s["ys"], s["weights"]), (s["gxs"], s["gy"]))
    return out


def _own_dropout(s, case):
    import muon_newton_schulz_05_amd as muon
    y = muon.dropout(s["x"], case["p"], seed=s["seed"], offset=s["offset"], residual=s["r"])
    return _with_grads(y, s, case, {"dx": s["x"]})


def _with_grads(y, s, case, leaves):
    out = {"y": y.detach()}
    if case["train"]:
        leaves = {k: v for k, v in leaves.items() if v is not None}
        out.update(zip(leaves, torch.autograd.grad(y, tuple(leaves.values()), s["gy"])))
    return out


OWN = {"linear": _own_linear, "experts": _own_experts, "route": _own_route, "dropout": _own_dropout}


def run(state):
    case = state["case"]
    return (OWN if own else PLAIN)[case["op"]](state, case)


# ------------------------------------------------------------------ what a pass cannot do without


def work(case):
    b = 2 if case["dtype"] == "bf16" else 4
    train = case["train"]
    if case["op"] in ("linear", "experts"):
        m, k, n, e = case["rows"], case["k"], case["n"], case.get("e", 1)
        if case["op"] == "experts":
            e = min(e, m)  # an expert without rows is not read
        els = m * k + e * k * n + m * n + (e * n if case["bias"] else 0) + (m * n if case.get("residual") else 0)
        if train:
            els += m * n + m * k + e * k * n + (e * n if case["bias"] else 0)
        return {"bytes": b * els, "flops": (6 if train else 2) * m * k * n}
    if case["op"] == "route":
        t, p, h = case["tokens"], case["tokens"] * case["top"], case["h"]
        size = 8 * p + 4 * p + 8 * p + 4 * (case["e"] + 1) + b * (2 * t * h + 2 * p * h)
        if train:
            size += 4 * p + b * (2 * t * h + 2 * p * h)
        return {"bytes": size, "flops": 2 * p * h * (3 if train else 1)}
    n = case["rows"] * case["cols"]
    return {"bytes": b * n * (2 + (1 if case["residual"] else 0) + (2 if train else 0)), "flops": n}


# ------------------------------------------------------------------ 64 bits


def _slope64(z, act):
    """act and its derivative, each from its definition, by the derivative's own formula."""
    if act == "none":
        return z, 1.0
    if act == "relu":
        return z.clamp_min(0), (z > 0).double()
    if act == "silu":
        q = torch.sigmoid(z)
        return z * q, q + z * q * (1 - q)
    if act == "gelu":
        cdf = torch.special.ndtr(z)
        return z * cdf, cdf + z * torch.exp(-z.square() / 2) / math.sqrt(2 * math.pi)
    u = math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)
    du = math.sqrt(2 / math.pi) * (1 + 3 * 0.044715 * z ** 2)
    return z / 2 * (1 + torch.tanh(u)), (1 + torch.tanh(u)) / 2 + z / 2 * du / torch.cosh(u).square()


def _affine64(x, w, b, r, gy, act):
    """The layer on one weight: y and, for gy, (dx, dw, db)."""
    x, w = x.detach().double(), w.detach().double()
    z = torch.mm(x, w)
    if b is not None:
        z += b.detach().double()
    y, slope = _slope64(z, act)
    if r is not None:
        y = y + r.double()
    if gy is None:
        return y, None, None, None
    dz = gy.double() * slope
    return y, torch.mm(dz, w.t()), torch.mm(x.t(), dz), dz.sum(0)


def _philox_python(seed, offset, block):
    """One block by Python's own integers."""
    c = [block & M32, block >> 32, offset & M32, offset >> 32]
    k = [seed & M32, seed >> 32 & M32]
    for _ in range(10):
        a, b = c[0] * 0xD2511F53, c[2] * 0xCD9E8D57
        c = [b >> 32 ^ c[1] ^ k[0], b & M32, a >> 32 ^ c[3] ^ k[1], a & M32]
        k = [k[0] + 0x9E3779B9 & M32, k[1] + 0xBB67AE85 & M32]
    return c


def exact(case, seed):
    s = prepare(case, seed)
    out = {}
    if case["op"] == "linear":
        y, dx, dw, db = _affine64(s["x"], s["w"], s["b"], s["r"], s["gy"], case["act"])
        out["y"] = y
        if case["train"]:
            out["dx"], out["dw"] = dx, dw
            if case["bias"]:
                out["db"] = db
        return out
    if case["op"] == "experts":
        off = s["offsets"].tolist()
        got = [_affine64(s["x"][lo:hi], s["w"][i], s["b"][i] if case["bias"] else None, None,
                         s["gy"][lo:hi] if case["train"] else None, case["act"])
               for i, (lo, hi) in enumerate(zip(off[:-1], off[1:]))]
        out["y"] = torch.cat([g[0] for g in got])
        if case["train"]:
            out["dx"], out["dw"] = torch.cat([g[1] for g in got]), torch.stack([g[2] for g in got])
            if case["bias"]:
                out["db"] = torch.stack([g[3] for g in got])
        return out
    if case["op"] == "route":
        t, top, e, h = case["tokens"], case["top"], case["e"], case["h"]
        flat = s["ids"].reshape(-1).cpu()
        lists = [(flat == i).nonzero()[:, 0] for i in range(e)]
        order = torch.cat(lists)
        n = order.numel()
        ends = torch.tensor([0] + [v.numel() for v in lists]).cumsum(0)
        position = torch.full((t * top,), -1)
        position[order] = torch.arange(n)
        dev = s["x"].device
        order, position = order.to(dev), position.to(dev)
        token, rows = order // top, s["ys"].detach().double()[:n]
        wf = s["weights"].detach().double().reshape(-1)[order][:, None]
        zero = torch.zeros(t, h, dtype=torch.float64, device=dev)
        tail = lambda v: torch.cat([v, v.new_zeros(t * top - n, h)])  # noqa: E731
        out = {"offsets": ends.to(torch.int32).to(dev),
               "order": torch.cat([order, order.new_full((t * top - n,), -1)]).to(torch.int32),
               "position": position.reshape(t, top).to(torch.int32),
               "xs": tail(s["x"].detach().double()[token]), "y": zero.index_add(0, token, wf * rows)}
        if case["train"]:
            gy = s["gy"].double()
            out["dx"] = zero.index_add(0, token, s["gxs"].double()[:n])
            out["dys"] = tail(wf * gy[token])
            dw = torch.zeros(t * top, dtype=torch.float64, device=dev)
            dw[order] = (gy[token] * rows).sum(1)
            out["dweights"] = dw.reshape(t, top)
        return out
    # The masks of up to 2^17 values from Python's integers; longer ones have no second generator that is quick
    # enough, and say nothing.
    n = case["rows"] * case["cols"]
    if n > 1 << 17:
        return None
    words = [v for i in range((n + 7) // 8) for v in _philox_python(s["seed"], s["offset"], i)]
    lanes = [v >> sh & 0xFFFF for v in words for sh in (0, 16)][:n]
    d = round(case["p"] * 65536)
    f = torch.tensor([0.0 if v < d else 65536 / (65536 - d) for v in lanes], dtype=torch.float64, device=s["x"].device)
    f = f.reshape(case["rows"], case["cols"])
    out["y"] = s["x"].detach().double() * f + (0 if s["r"] is None else s["r"].double())
    if case["train"]:
        out["dx"] = s["gy"].double() * f
    return out
