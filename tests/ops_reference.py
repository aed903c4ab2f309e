"""Plain float64 forms of the layer operators and the tolerances of their tests.

A tolerance counts the roundings on the way to a value: u = eps / 2 of the
storage type for each value stored in it, 2^-24 for each float32 operation,
taken over the sum of magnitudes that the value is made of."""

from __future__ import annotations

import math

import torch

U32 = 2.0 ** -24


def unit(dtype):
    return torch.finfo(dtype).eps / 2


def act64(z, act):
    if act == "none":
        return z.clone(), torch.ones_like(z)
    if act == "relu":
        return z.clamp_min(0), (z > 0).double()
    if act == "silu":
        q = torch.sigmoid(z)
        return z * q, q + z * q * (1 - q)
    if act == "gelu":
        cdf = 0.5 * torch.special.erfc(-z / math.sqrt(2))
        return z * cdf, cdf + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    c = math.sqrt(2 / math.pi)
    th = torch.tanh(c * (z + 0.044715 * z ** 3))
    return z * (1 + th) / 2, (1 + th) / 2 + z / 2 * (1 - th * th) * c * (1 + 3 * 0.044715 * z * z)


def linear64(x, w, b, r, dy, act):
    """{name: (value, tolerance)} of y and, for dy, dx, dw, db; inputs on the CPU in their storage type."""
    u = unit(x.dtype)
    x, w = x.double(), w.double()
    rows, k = x.shape
    n = w.shape[1]
    z = x @ w
    size = x.abs() @ w.abs()                    # magnitudes behind z
    if b is not None:
        z = z + b.double()
        size = size + b.double().abs()
    y, slope = act64(z, act)
    # float32 sums of k products in any order, and an activation of slope at
    # most 1.13 evaluated with relative errors of a few 2^-24.
    ez = (k + 2) * U32 * size
    ey = 1.2 * ez + 16 * U32 * z.abs()
    if r is not None:
        y = y + r.double()
        ey = ey + U32 * y.abs()
    out = {"y": (y, ey + u * y.abs() + 1e-37)}
    if dy is not None:
        dy = dy.double()
        dz = dy * slope
        # z is stored in x's type; the slopes' own slopes are at most 1.13.
        # relu's slope jumps where z may round across zero.
        edz = torch.zeros_like(dz) if act == "none" else dy.abs() * (1.2 * (ez + u * z.abs()) + 16 * U32)
        if act == "relu":
            edz = torch.where(z.abs() <= ez, dy.abs(), torch.zeros_like(edz))
        edzs = edz + (0 if act == "none" else u * dz.abs())   # as stored
        out["dx"] = _sum(dz @ w.t(), edzs @ w.abs().t() + (n + 2) * U32 * (dz.abs() + edzs) @ w.abs().t(), u)
        out["dw"] = _sum(x.t() @ dz, x.abs().t() @ edzs + (rows + 2) * U32 * x.abs().t() @ (dz.abs() + edzs), u)
        out["db"] = _sum(dz.sum(0), edz.sum(0) + (rows + 2) * U32 * (dz.abs() + edz).sum(0), u)
    return out


def _sum(v, err, u):
    return v, err + u * (v.abs() + err) + 1e-37


def check(name, got, want, norm=None):
    """got within want = (value, tolerance) everywhere, and its 2-norm error within `norm` of the value's."""
    value, tol = want
    got = got.detach().double().cpu()
    assert got.shape == value.shape, (name, got.shape, value.shape)
    diff = (got - value).abs()
    bad = ~(diff <= tol)
    assert not bad.any(), (name, int(bad.sum()), float(diff[bad].max()),
                           [int(i[0]) for i in bad.nonzero(as_tuple=True)], float((diff / tol).nan_to_num().max()))
    if norm is not None and value.numel() > 64:
        off = float(diff.norm() / value.norm().clamp_min(1e-300))
        assert off <= norm, (name, off)


def route64(ids, experts):
    """offsets, order, position by Python's own sort."""
    tokens, top = ids.shape
    flat = ids.reshape(-1).tolist()
    routed = [i for i, e in enumerate(flat) if 0 <= e < experts]
    routed.sort(key=lambda i: (flat[i], i))
    offsets = [0] * (experts + 1)
    for i in routed:
        offsets[flat[i] + 1] += 1
    for e in range(experts):
        offsets[e + 1] += offsets[e]
    position = [-1] * (tokens * top)
    for p, i in enumerate(routed):
        position[i] = p
    order = routed + [-1] * (tokens * top - len(routed))
    return torch.tensor(offsets), torch.tensor(order, dtype=torch.int64), torch.tensor(position).view(tokens, top)


M32 = 0xFFFFFFFF


def philox(seed, offset, block):
    c = [block & M32, block >> 32, offset & M32, offset >> 32]
    k = [seed & M32, seed >> 32 & M32]
    for _ in range(10):
        a, b = c[0] * 0xD2511F53, c[2] * 0xCD9E8D57
        c = [b >> 32 ^ c[1] ^ k[0], b & M32, a >> 32 ^ c[3] ^ k[1], a & M32]
        k = [k[0] + 0x9E3779B9 & M32, k[1] + 0xBB67AE85 & M32]
    return c


def keep_mask(n, p, seed, offset):
    """Kept elements and the scale of dropout."""
    drop = round(p * 65536)
    lanes = [v >> s & 0xFFFF for i in range((n + 7) // 8) for v in philox(seed, offset, i) for s in (0, 16)][:n]
    return torch.tensor([v >= drop for v in lanes]), 65536 / (65536 - drop)
