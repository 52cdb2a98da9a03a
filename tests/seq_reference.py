"""Plain float64 references of the sequence operators, token by token and row
by row (test infrastructure only)."""
import torch

F64 = torch.float64


def scan(v, k, q, g, b=None, S0=None, keep=False):
    """(y, S, states) of S_t = e^{g_t} S_{t-1} + b_t v_t k_t^T, y_t = S_t q_t in
    float64; states (with keep): S_0 and the state after every token."""
    v, k, q = (x.to(F64) for x in (v, k, q))
    B, T, H, P = v.shape
    G, N = k.shape[2:]
    k, q = (x.repeat_interleave(H // G, 2) for x in (k, q))
    a = torch.exp(g.to(F64))
    b = torch.ones(B, T, H, dtype=F64) if b is None else b.to(F64)
    S = torch.zeros(B, H, P, N, dtype=F64) if S0 is None else S0.to(F64)
    y = torch.zeros(B, T, H, P, dtype=F64)
    states = [S]
    for t in range(T):
        S = a[:, t, :, None, None] * S + (b[:, t, :, None] * v[:, t])[..., None] * k[:, t, :, None, :]
        y[:, t] = (S * q[:, t, :, None, :]).sum(-1)
        if keep:
            states.append(S)
    return y, S, states


def scan_grads(v, k, q, g, dy, b=None, S0=None, dS=None):
    """(dv, dk, dq, dg, db, dS0) in float64."""
    _, _, states = scan(v, k, q, g, b, S0, keep=True)
    v, k, q, dy = (x.to(F64) for x in (v, k, q, dy))
    B, T, H, P = v.shape
    G, N = k.shape[2:]
    kh, qh = (x.repeat_interleave(H // G, 2) for x in (k, q))
    a = torch.exp(g.to(F64))
    b = torch.ones(B, T, H, dtype=F64) if b is None else b.to(F64)
    D = torch.zeros(B, H, P, N, dtype=F64) if dS is None else dS.to(F64)
    dv, dk, dq = torch.zeros_like(v), torch.zeros_like(kh), torch.zeros_like(qh)
    dg, db = torch.zeros_like(a), torch.zeros_like(a)
    for t in reversed(range(T)):
        D = D + dy[:, t, :, :, None] * qh[:, t, :, None, :]
        dq[:, t] = (states[t + 1] * dy[:, t, :, :, None]).sum(2)
        z = (D * kh[:, t, :, None, :]).sum(3)
        dv[:, t] = b[:, t, :, None] * z
        db[:, t] = (v[:, t] * z).sum(2)
        dk[:, t] = b[:, t, :, None] * (D * v[:, t, :, :, None]).sum(2)
        D = a[:, t, :, None, None] * D
        dg[:, t] = (D * states[t]).sum((2, 3))
    fold = lambda x: x.unflatten(2, (G, H // G)).sum(3)  # noqa: E731
    return dv, fold(dk), fold(dq), dg, db, D


def norm(x, w=None, bias=None, eps=1e-5, center=True):
    x = x.to(F64)
    mu = x.mean(-1, keepdim=True) if center else torch.zeros_like(x[..., :1])
    r = 1.0 / torch.sqrt(((x - mu) ** 2).mean(-1, keepdim=True) + eps)
    y = (x - mu) * r
    if w is not None:
        y = y * w.to(F64)
    if bias is not None:
        y = y + bias.to(F64)
    return y, mu[..., 0], r[..., 0]


def norm_grads(dy, x, w, mu, r, center=True):
    """(dx, dw, dbias) from the statistics given."""
    x, dy, r = x.to(F64), dy.to(F64), r.to(F64)[..., None]
    xh = (x - mu.to(F64)[..., None]) * r if center else x * r
    t = dy if w is None else dy * w.to(F64)
    dx = t - xh * (t * xh).mean(-1, keepdim=True)
    if center:
        dx = dx - t.mean(-1, keepdim=True)
    n = x.shape[-1]
    return r * dx, (dy * xh).reshape(-1, n).sum(0), dy.reshape(-1, n).sum(0)


def rel(got, want):
    """||got - want|| / ||want|| (0 where both are zero)."""
    got, want = got.detach().cpu().to(F64), want.to(F64)
    assert got.shape == want.shape, (got.shape, want.shape)
    off, size = float((got - want).norm()), float(want.norm())
    return off / size if size else (0.0 if off == 0.0 else float("inf"))
