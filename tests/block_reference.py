"""Plain float64 forms of the operators around a block's products, and the tolerances of their tests.

A tolerance counts the roundings on the way to a value, as in ops_reference: u for
each value stored in a type, U32 for each float32 operation, taken over the magnitudes it acts on.  Sums of
float32 values count one rounding for each addition on the longest path to the result."""

from __future__ import annotations

import torch

from ops_reference import U32, unit

TINY = 1e-37  # what float32 may flush


def path(n, serial=1):
    """Additions on the way of one value into a sum of n: `serial` times those that one thread makes, a wave's and
    a workgroup's."""
    return serial + 6 + 16 + min(n, 16)


def norm64(x, r, w, b, dy, ds, eps, layer):
    """{name: (value, tolerance)} of y, s, and for dy, dx, dw, db; 2-D inputs on the CPU in their storage type."""
    u = unit(x.dtype)
    rows, cols = x.shape
    h = x.double() if r is None else x.double() + r.double()
    eh = torch.zeros_like(h) if r is None else U32 * h.abs()
    one = torch.ones(cols, dtype=torch.float64)
    w = one if w is None else w.double()
    b = 0 * one if b is None else b.double()
    a = path(cols, 1 + cols // 8192)
    mean = h.mean(1, keepdim=True) if layer else torch.zeros(rows, 1, dtype=torch.float64)
    emean = (a * U32 * h.abs().mean(1, keepdim=True) + eh.mean(1, keepdim=True) + U32 * mean.abs()) if layer else 0 * mean
    c = h - mean
    ec = eh + emean + U32 * c.abs()
    var = (c * c).mean(1, keepdim=True)
    evar = (a + 3) * U32 * var + (2 * c.abs() * ec + ec * ec).mean(1, keepdim=True)
    rstd = (var + eps) ** -0.5
    erstd = rstd * (0.5 * evar / (var + eps) + 4 * U32)      # the sum with eps, the root, the division
    xhat = c * rstd
    ex = rstd * ec + c.abs() * erstd + 2 * U32 * xhat.abs()
    y = xhat * w + b
    out = {"y": (y, ex * w.abs() + 2 * U32 * ((xhat * w).abs() + b.abs()) + u * y.abs() + TINY)}
    if r is not None:
        out["s"] = (h, eh + u * h.abs())
    if dy is None:
        return out
    dy = dy.double()
    g = dy * w
    mg = g.mean(1, keepdim=True) if layer else torch.zeros(rows, 1, dtype=torch.float64)
    mx = (g * xhat).mean(1, keepdim=True)
    emg = (a + 2) * U32 * g.abs().mean(1, keepdim=True) if layer else 0 * mg
    emx = (a + 3) * U32 * (g * xhat).abs().mean(1, keepdim=True) + (g.abs() * ex).mean(1, keepdim=True)
    pre = g - mg - xhat * mx
    epre = 3 * U32 * (g.abs() + mg.abs() + (xhat * mx).abs()) + emg + xhat.abs() * emx + ex * mx.abs()
    dx = rstd * pre
    edx = rstd * epre + erstd * pre.abs() + U32 * dx.abs()
    if ds is not None:
        dx = dx + ds.double()
        edx = edx + U32 * (dx.abs() + ds.double().abs())
    # A thread adds one of 512 row groups (64 stretches of wide rows), 1024 threads join them.
    add = path(rows, 2 + rows // (64 if cols > 8192 else 512) + 32) + 32
    add = min(add, rows + 4)
    dw, db = (dy * xhat).sum(0), dy.sum(0)
    out["dx"] = dx, edx + u * dx.abs() + TINY
    out["dw"] = dw, (dy.abs() * ex).sum(0) + add * U32 * (dy * xhat).abs().sum(0) + u * dw.abs() + TINY
    out["db"] = db, add * U32 * dy.abs().sum(0) + u * db.abs() + TINY
    return out


def _exp_rel(d):
    """The relative error of e^d, d <= 0 a rounded difference: d's rounding, and about four more."""
    return U32 * (d.abs().clamp_max(200) + 4)


def softmax64(z):
    """Probabilities (0 in rows of -inf alone) and their relative errors."""
    z = z.double()
    m = z.amax(1, keepdim=True)
    dead = m == -torch.inf
    d = torch.where(dead, -torch.inf, z - m)
    e = torch.exp(d)
    total = e.sum(1, keepdim=True).clamp_min(1e-300)
    rel = _exp_rel(d)
    part = (e * rel).sum(1, keepdim=True) / total
    return e / total, rel + part + path(z.shape[1], 16) * U32


def choose(z, top, mask):
    """ids by Python's own sort: falling, NaN first, ties to the lower index, -inf never."""
    ids = torch.full((len(z), top), -1, dtype=torch.int64)
    for t, row in enumerate(z.double().tolist()):
        if mask is not None and not mask[t]:
            continue
        key = [(0 if v != v else 1, 0 if v != v else -v, i) for i, v in enumerate(row) if v != -float("inf")]
        for j, (_, _, i) in enumerate(sorted(key)[:top]):
            ids[t, j] = i
    return ids


def gate64(z, top, normalize, mask, dw):
    """ids, (weights, tolerance), and for dw (dz, tolerance)."""
    u = unit(z.dtype)
    ids = choose(z, top, mask)
    on = ids >= 0
    at = ids.clamp_min(0)
    if normalize:
        zs = torch.where(on, z.double().gather(1, at), -torch.inf)
        w, rel = softmax64(zs)
    else:
        p, prel = softmax64(z)
        w, rel = torch.where(on, p.gather(1, at), 0), prel.gather(1, at)
    w = torch.where(on, w, 0.0)
    out = {"ids": ids, "weights": (w, w * rel + TINY)}
    if dw is None:
        return out
    dw = torch.where(on, dw.double(), 0.0)
    mean = (w * dw).sum(1, keepdim=True)
    emean = (w * dw.abs() * (rel + path(top, 16) * U32)).sum(1, keepdim=True)
    dz, edz = torch.zeros(z.shape, dtype=torch.float64), torch.zeros(z.shape, dtype=torch.float64)
    rows = torch.arange(len(z))[:, None].expand_as(ids)
    if normalize:
        v = w * (dw - mean)
        ev = w * ((rel + 2 * U32) * (dw - mean).abs() + U32 * (dw.abs() + mean.abs()) + emean)
    else:
        v, ev = w * dw, w * dw.abs() * (rel + 2 * U32)
        live = on.any(1, keepdim=True)
        dz = torch.where(live, -p * mean, 0.0)
        edz = torch.where(live, p * (emean + mean.abs() * (prel + 2 * U32)), 0.0)
    dz.index_put_((rows[on], ids[on]), v[on], accumulate=True)
    edz.index_put_((rows[on], ids[on]), ev[on] + U32 * v[on].abs(), accumulate=True)
    out["dz"] = dz, edz + u * dz.abs() + TINY
    return out


def balance64(z, ids, mask, dloss):
    """counts, (loss, tolerance) and (dz, tolerance)."""
    u = unit(z.dtype)
    t, e = z.shape
    on = torch.ones(t, dtype=torch.bool) if mask is None else mask
    n, top = int(on.sum()), ids.shape[1]
    counts = torch.zeros(e, dtype=torch.int64)
    for i in ids[on].reshape(-1).tolist():
        if 0 <= i < e:
            counts[i] += 1
    f = counts.double() / max(n * top, 1)
    p, rel = softmax64(torch.where(on[:, None], z, torch.zeros((), dtype=z.dtype)))
    p = torch.where(on[:, None], p, 0.0)
    rel = torch.where(p == 0, 0.0, rel)
    share = p.sum(0) / max(n, 1)
    add = path(t, 2 + t // 1024)
    loss = e * (f * share).sum()
    tol = e * (f * ((p * rel).sum(0) / max(n, 1) + add * U32 * share)).sum() + 2 * U32 * loss.abs() + TINY
    mean = (p * f).sum(1, keepdim=True)
    emean = (p * f * (rel + path(e, 16) * U32)).sum(1, keepdim=True)
    scale = dloss * e / max(n, 1)
    dz = scale * p * (f - mean)
    edz = scale * p * ((rel + 8 * U32) * (f - mean).abs() + 2 * U32 * (f + mean) + emean)
    return {"counts": counts, "loss": (loss, tol), "dz": (dz, edz + u * dz.abs() + TINY)}


LEVELS = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def blocks64(v):
    """Four bits along the last dimension: (the values they stand for, codes, scales + 127), one value at a time."""
    rows, k = v.shape
    nb = -(-k // 32)
    full = torch.zeros(rows, nb * 32, dtype=torch.float64)
    full[:, :k] = v.double()
    values, codes = torch.zeros_like(full), torch.zeros(rows, nb * 32, dtype=torch.int64)
    scales = torch.zeros(rows, nb, dtype=torch.int64)
    for r in range(rows):
        for b in range(nb):
            block = full[r, 32 * b:32 * b + 32].tolist()
            at = slice(32 * b, 32 * b + 32)
            if any(x != x or abs(x) == float("inf") for x in block):
                scales[r, b] = 255
                values[r, at] = float("nan")
                continue
            peak, exponent = max(abs(x) for x in block), -127
            if peak > 0:
                exponent = int(float(peak).hex().split("p")[1]) - 2
            exponent = max(exponent, -127)
            scales[r, b] = exponent + 127
            for i, x in enumerate(block):
                a = abs(x) * 2.0 ** -exponent
                best = min(range(8), key=lambda c: (abs(LEVELS[c] - a), c % 2))
                codes[r, 32 * b + i] = best + (8 if x < 0 or (x == 0 and str(x)[0] == "-") else 0)
                values[r, 32 * b + i] = (-1 if x < 0 else 1) * LEVELS[best] * 2.0 ** exponent
    return values[:, :k], codes, scales


def fast_blocks64(v):
    """The values of ``blocks64`` alone, for larger tensors (finite ones)."""
    rows, k = v.shape
    full = torch.zeros(rows, -(-k // 32) * 32, dtype=torch.float64)
    full[:, :k] = v.double()
    b = full.view(rows, full.shape[1] // 32, 32)
    exponent = (torch.frexp(b.abs().amax(2, keepdim=True))[1] - 3).clamp_min(-127)
    scale = torch.ldexp(torch.ones((), dtype=torch.float64), exponent)
    a = b.abs() / scale
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
    q = (torch.round(a / step) * step).clamp_max(6) * torch.sign(b) * scale
    return q.view(full.shape)[:, :k]
