"""Plain float64 references of the token embedding, the group norm and the token
log probabilities, with their gradients (CPU)."""
import math

import torch

F64 = torch.float64


def embedding(table, ids, scale=1.0):
    ok = (ids >= 0) & (ids < table.shape[0])
    y = table.to(F64)[torch.where(ok, ids, 0).long()] * scale
    return torch.where(ok[..., None], y, 0.0)


def embedding_grad(dy, ids, vocab, scale=1.0):
    """(dtable, the sums of absolute values that its rounding goes by)."""
    n = dy.shape[-1]
    ids, dy = ids.reshape(-1).long(), dy.reshape(-1, n).to(F64)
    ok = (ids >= 0) & (ids < vocab)
    out = [torch.zeros(vocab, n, dtype=F64).index_add_(0, ids[ok], v[ok]) * abs(scale) for v in (dy, dy.abs())]
    return (out[0] if scale >= 0 else -out[0]), out[1]


def _silu(z):
    return z * torch.sigmoid(z)


def _slope(z):
    s = torch.sigmoid(z)
    return s * (1.0 + z * (1.0 - s))


def group_norm(x, groups, w=None, b=None, z=None, gate_first=True, activation="silu", eps=1e-5, center=False):
    """(y, mean or None, rstd) in float64."""
    x = x.to(F64)
    u = x if z is None or not gate_first else x * _silu(z.to(F64))
    u = u.unflatten(-1, (groups, -1))
    mean = u.mean(-1, keepdim=True) if center else torch.zeros_like(u[..., :1])
    rstd = 1.0 / torch.sqrt((u - mean).square().mean(-1, keepdim=True) + eps)
    o = ((u - mean) * rstd).flatten(-2)
    o = o if w is None else o * w.to(F64)
    o = o if b is None else o + b.to(F64)
    if z is not None and not gate_first:
        o = o * _silu(z.to(F64))
    elif z is None and activation == "silu":
        o = _silu(o)
    return o, (mean[..., 0] if center else None), rstd[..., 0]


def group_norm_grads(dy, x, groups, w, b, mean, rstd, z=None, gate_first=True, activation="silu"):
    """(dx, dz or None, dw, db) from the statistics given (mean None: no centering)."""
    x, dy, z = x.to(F64), dy.to(F64), None if z is None else z.to(F64)
    before = z is not None and gate_first
    u = (x * _silu(z) if before else x).unflatten(-1, (groups, -1))
    mu = torch.zeros_like(u[..., :1]) if mean is None else mean.to(F64)[..., None]
    r = rstd.to(F64)[..., None]
    xh = ((u - mu) * r).flatten(-2)
    wide = torch.ones(x.shape[-1], dtype=F64) if w is None else w.to(F64)
    o = xh * wide + (0.0 if b is None else b.to(F64))
    dz, do = None, dy
    if z is not None and not gate_first:
        dz, do = dy * o * _slope(z), dy * _silu(z)
    elif z is None and activation == "silu":
        do = dy * _slope(o)
    t, xg = (do * wide).unflatten(-1, (groups, -1)), xh.unflatten(-1, (groups, -1))
    du = t - xg * (t * xg).mean(-1, keepdim=True)
    if mean is not None:
        du = du - t.mean(-1, keepdim=True)
    du = (du * r).flatten(-2)
    dx = du
    if before:
        dx, dz = du * _silu(z), du * x * _slope(z)
    rows = lambda v: v.reshape(-1, v.shape[-1]).sum(0)  # noqa: E731
    return dx, dz, rows(do * xh), rows(do)


def group_norm_bounds(dy, x, groups, w, b, mean, rstd, z=None, gate_first=True, activation="silu", forward=False):
    """Bounds of what float32 leaves of the results, element by element: dict of dx, dz, dw
    and db for the statistics given (forward: of y for exact ones).  With U = 2^-24, a sum
    of fewer than 100 roundings is off by N = 100 U of the sum of absolute terms, a sigmoid
    by (8 + 4 |z|) U.  (u - mu) r is off by those of u, mu and the difference times r: next
    to (|u| + |mu|) r it may be small, and 0 where a group has one channel."""
    U, N = 2.0**-24, 100 * 2.0**-24
    x, dy, z = x.to(F64), dy.to(F64), None if z is None else z.to(F64)
    cut = lambda v: v.unflatten(-1, (groups, -1))  # noqa: E731
    avg = lambda v: cut(v).mean(-1, keepdim=True).expand_as(cut(v)).flatten(-2)  # noqa: E731
    per = lambda v: v.to(F64)[..., None].expand_as(cut(x)).flatten(-2)  # noqa: E731
    before, after = z is not None and gate_first, z is not None and not gate_first
    wide = torch.ones(x.shape[-1], dtype=F64) if w is None else w.to(F64)
    bias = torch.zeros_like(wide) if b is None else b.to(F64)
    off = 0.0 if z is None else (8 + 4 * z.abs()) * U
    u = x * _silu(z) if before else x
    r, mu = per(rstd), torch.zeros_like(u) if mean is None else per(mean)
    xh = (u - mu) * r
    d = N * (u.abs() + mu.abs()) * r + (off * u.abs() * r if before else 0.0)
    if forward:
        if mean is not None:
            d = d + N * avg(u.abs()) * r + (avg(off * u.abs()) * r if before else 0.0)
        d = d + xh.abs() * (N + 2 * avg(d * d).sqrt())
    o = xh * wide + bias
    eo = d * wide.abs() + 4 * U * ((xh * wide).abs() + bias.abs())
    silu_o = z is None and activation == "silu"
    off_o = (8 + 4 * o.abs()) * U
    if forward:
        ey = eo
        if after:
            ey = eo * _silu(z).abs() + (o.abs() + eo) * _silu(z).abs() * off
        elif silu_o:
            ey = 1.1 * eo + off_o * _silu(o).abs()
        return {"y": ey}
    steep = lambda v, k: k * torch.sigmoid(v) * (1 + v.abs())  # noqa: E731
    do, edo = dy, torch.zeros_like(dy)
    out = {}
    if after:
        do = dy * _silu(z)
        edo = off * do.abs()
        out["dz"] = dy.abs() * (eo * _slope(z).abs() + (o.abs() + eo) * steep(z, off) + 4 * U * (o * _slope(z)).abs())
    elif silu_o:
        do = dy * _slope(o)
        edo = dy.abs() * (0.5 * eo + steep(o, off_o))
    t = do * wide
    et = edo * wide.abs() + 2 * U * t.abs()
    txh = avg((t * xh).abs())
    edu = r * (et + avg(et) + N * (t.abs() + avg(t.abs()) + xh.abs() * txh) + d * txh + (xh.abs() + d) * avg(t.abs() * d + et * (xh.abs() + d)))
    out["dx"] = edu
    if before:
        g = t - xh * avg(t * xh)
        du = r * (g if mean is None else g - avg(t))
        out["dx"] = edu * _silu(z).abs() + (du * _silu(z)).abs() * off
        out["dz"] = edu * (x * _slope(z)).abs() + (du * x).abs() * (steep(z, off) + 4 * U * _slope(z).abs())
    rows = lambda v: v.reshape(-1, v.shape[-1]).sum(0)  # noqa: E731
    out["dw"] = rows(do.abs() * d + edo * (xh.abs() + d)) + N * rows((do * xh).abs())
    out["db"] = rows(edo) + N * rows(do.abs())
    return out


def logprobs(x, ids=None, scale=1.0, top=0):
    """dict of logp, entropy, stats, top_ids, top_logp, and of what their rounding goes by:
    t (the token's exponent), first (sum p |t|) and second (sum p t^2) moments."""
    x = x.to(F64)
    rows, vocab = x.shape
    m = x.max(1).values
    t = (x - m[:, None]) * scale
    e = torch.where(x == -math.inf, torch.where(torch.isnan(m)[:, None] | (m == math.inf)[:, None], math.nan, 0.0), torch.exp(t))
    total = e.sum(1)
    none = m == -math.inf
    total = torch.where(none, 0.0, total)
    L = torch.log(total)
    p = torch.where(none[:, None], 0.0, e / total[:, None])
    tt = torch.where(p == 0, 0.0, t)
    m = torch.where(torch.isnan(L), math.nan, m)   # (of a row with a NaN or an infinity)
    out = {"stats": torch.stack([m, L], 1), "entropy": torch.where(none, 0.0, L - (p * tt).sum(1)), "p": p, "t": t,
           "first": (p * tt.abs()).sum(1), "second": (p * tt * tt).sum(1)}
    if ids is not None:
        ok = (ids >= 0) & (ids < vocab)
        ti = t[torch.arange(rows), torch.where(ok, ids, 0).long()]
        out["logp"] = torch.where(ok, torch.where(none, -math.inf, ti - L), 0.0)
        out["ti"] = ti
    if top:
        lost = torch.isnan(L)
        order = torch.sort(x, dim=1, descending=True, stable=True)
        k = min(top, vocab)
        out["top_ids"] = torch.full((rows, top), -1, dtype=torch.int32)
        out["top_logp"] = torch.full((rows, top), -math.inf, dtype=F64)
        can = order.values[:, :k] > -math.inf
        out["top_ids"][:, :k] = torch.where(can, order.indices[:, :k], -1).int()
        out["top_logp"][:, :k] = torch.where(can, (order.values[:, :k] - m[:, None]) * scale - L[:, None], -math.inf)
        out["top_ids"][lost] = -1
        out["top_logp"][lost] = math.nan
    return out


def logprobs_grad(x, ids, stats, dlogp, scale=1.0, entropy=None, dentropy=None):
    """(dx, the size that its rounding goes by) from the statistics given."""
    x, stats = x.to(F64), stats.to(F64)
    rows, vocab = x.shape
    none = stats[:, 1] == -math.inf
    lp = torch.where(none[:, None], -math.inf, (x - stats[:, :1]) * scale - stats[:, 1:])
    p = torch.exp(lp)
    ok = (ids >= 0) & (ids < vocab) if ids is not None else torch.zeros(rows, dtype=torch.bool)
    dl = torch.where(ok, dlogp.to(F64), 0.0) if dlogp is not None else torch.zeros(rows, dtype=F64)
    dh = torch.zeros(rows, dtype=F64) if dentropy is None else dentropy.to(F64)
    H = torch.zeros(rows, dtype=F64) if entropy is None else entropy.to(F64)
    plp = torch.where(p > 0, p * lp, 0.0)
    d = -dl[:, None] * p - dh[:, None] * (plp + H[:, None] * p)
    size = (dl.abs()[:, None] + dh.abs()[:, None] * H.abs()[:, None]) * p + dh.abs()[:, None] * plp.abs()
    size = size * (1.0 + torch.where(p > 0, lp.abs(), 0.0))
    if ids is not None:
        at = torch.where(ok, ids, 0).long()[:, None]
        d.scatter_add_(1, at, dl[:, None])
        size.scatter_add_(1, at, dl.abs()[:, None])
    quiet = ((dl == 0) & (dh == 0)) | none
    return torch.where(quiet[:, None], 0.0, d * scale), torch.where(quiet[:, None], 0.0, size * scale)
