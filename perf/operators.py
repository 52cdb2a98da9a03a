"""Performance cases of the gated scan and the layer norm.

listed() holds fixed cases, draw() makes more of the same ranges, prepare()
makes a case's inputs and run() does one pass: through the library's entry
points where `own` is true, else in plain torch operations in float32.

Gated scan, for every sequence and head (keys and queries are shared by the
heads of a group):
    S_t = exp(g_t) S_{t-1} + b_t v_t k_t^T        (P x N)
    y_t = S_t q_t
g is the log decay (-inf starts a new sequence at t), b an input gate.  Layer
norm: y = (x - mean) / sqrt(var + eps) * w + bias, or with center false the
same without the mean (a root-mean-square norm).

The shapes are those of Mamba-2 130M (24 layers, d_model 768, 24 heads of 64,
state size 128, one key/query group) and odd ones around them.
"""
import math

import torch

own = False

CHUNK = 64
EPS = 1e-5
HEADS, P, N = 24, 64, 128       # Mamba-2 130M
D_MODEL = 768


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def _scan(name, op, batch, tokens, heads=HEADS, groups=1, p=P, n=N, dtype="bf16", gate=True, state=False,
          packed=0, sliced=False):
    """packed: mean length of the sequences packed into a row (0: one sequence
    a row).  sliced: v, k and q are column ranges of one wider tensor, as a
    projection leaves them."""
    return dict(name=name, op=op, batch=batch, tokens=tokens, heads=heads, groups=groups, p=p, n=n, dtype=dtype,
                gate=gate, state=state, packed=packed, sliced=sliced)


def _norm(name, op, rows, n, dtype="bf16", center=True, affine=True):
    return dict(name=name, op=op, rows=rows, n=n, dtype=dtype, center=center, affine=affine)


def listed():
    return [
        # one token of one sequence: the latency of a decode step
        _scan("step_1", "step", 1, 1),
        # one token each of 160 sequences: a full decode batch, bound by the states' traffic
        _scan("step_160", "step", 160, 1),
        # a short prompt with odd sizes, in float32, continuing a state
        _scan("scan_fwd_short_f32", "fwd", 2, 77, heads=6, groups=2, p=40, n=72, dtype="f32", state=True),
        # a training batch, read from the projection's output
        _scan("scan_fwd_train", "fwd", 8, 2048, sliced=True),
        # one long prompt, states in and out: few heads in all, so the time axis has to be split
        _scan("scan_fwd_long", "fwd", 1, 16384, state=True),
        # the gradients of a training batch
        _scan("scan_bwd_train", "bwd", 8, 2048, sliced=True),
        # the gradients of packed sequences of different lengths, one row
        _scan("scan_bwd_packed", "bwd", 1, 8191, packed=700),
        # ungrouped heads in float32, ragged length, gradient of both states
        _scan("scan_bwd_ragged_f32", "bwd", 3, 333, heads=8, groups=8, p=64, n=64, dtype="f32", state=True),
        # the norm before the projection: a training batch, and its gradients with the weight's
        _norm("norm_fwd_train", "norm_fwd", 8 * 2048, D_MODEL),
        _norm("norm_bwd_train", "norm_bwd", 8 * 2048, D_MODEL),
        # the norm of a decode batch (latency)
        _norm("norm_fwd_decode", "norm_fwd", 32, D_MODEL, center=False),
        # few wide float32 rows of odd length
        _norm("norm_bwd_wide_f32", "norm_bwd", 1031, 4099, dtype="f32"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["step", "fwd", "fwd", "bwd", "bwd", "norm_fwd", "norm_bwd"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op.startswith("norm"):
        n = _log_int(rng, 32, 8192)
        rows = _log_int(rng, 1, max(2, 8 * 2048 * D_MODEL // n))
        c = _norm("", op, rows, n, dtype, center=rng.random() < 0.5, affine=rng.random() < 0.8)
    else:
        groups = rng.choice([1, 1, 2, 4])
        heads = groups * rng.choice([1, 2, 3, 6])
        p, n = rng.choice([16, 40, 64, 64, 64, 80, 128]), rng.choice([16, 64, 72, 128, 128, 128])
        most = 8 * 2048 * HEADS // heads * min(1.0, P * N / (p * n)) // (1 if dtype == "bf16" else 8)
        if op == "step":
            batch, tokens = _log_int(rng, 1, 256), 1
        else:
            tokens = _log_int(rng, 1, min(16384, most))
            batch = _log_int(rng, 1, max(1, min(16, int(most) // tokens)))
        c = _scan("", op, batch, tokens, heads, groups, p, n, dtype, gate=rng.random() < 0.7,
                  state=rng.random() < 0.5, packed=0 if op == "step" else rng.choice([0, 0, 50, 700]),
                  sliced=rng.random() < 0.5)
    del c["name"]
    return c


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _dtype(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


def prepare(case, seed):
    dev = torch.device("cuda" if torch.cuda.is_available() else "cpu")
    gen = torch.Generator(device=dev).manual_seed(seed)
    dt = _dtype(case)

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device=dev)

    def uniform(*shape):
        return torch.rand(*shape, generator=gen, device=dev)

    s = {"case": case}
    if case["op"].startswith("norm"):
        rows, n = case["rows"], case["n"]
        # a residual stream: channels of different size and offset
        s["x"] = (normal(rows, n) * (0.5 + uniform(n)) + 0.3 * normal(n)).to(dt)
        s["w"] = 1.0 + 0.2 * normal(n) if case["affine"] else None
        s["bias"] = 0.1 * normal(n) if case["affine"] and case["center"] else None
        if case["op"] == "norm_bwd":
            s["dy"] = normal(rows, n).to(dt)
            x = s["x"].float()  # the statistics that the forward pass kept
            s["mean"] = x.mean(1) if case["center"] else None
            d = x - s["mean"][:, None] if case["center"] else x
            s["rstd"] = torch.rsqrt((d * d).mean(1) + EPS)
        return s
    b, t, h, g, p, n = (case[k] for k in ("batch", "tokens", "heads", "groups", "p", "n"))
    cols = [h * p, g * n, g * n]
    if case["sliced"]:
        wide = normal(b, t, sum(cols)).to(dt)
        v, k, q = wide.split(cols, dim=2)
    else:
        v, k, q = (normal(b, t, c).to(dt) for c in cols)
    s["v"], s["k"], s["q"] = v.unflatten(2, (h, p)), k.unflatten(2, (g, n)), q.unflatten(2, (g, n))
    # step sizes between 0.001 and 0.1, moved by the token; decay rates between 1 and 16 by head
    step = torch.nn.functional.softplus(torch.log(torch.expm1(0.001 * 100.0 ** uniform(h))) + 0.5 * normal(b, t, h))
    s["g"] = -step * (1.0 + 15.0 * uniform(h))
    s["b"] = step if case["gate"] else None
    if case["packed"]:
        s["g"] = torch.where(uniform(b, t, 1) < 1.0 / case["packed"], -math.inf, s["g"])
    s["S0"] = normal(b, h, p, n) if case["state"] or case["op"] == "step" else None
    if case["op"] == "bwd":
        s["dy"] = normal(b, t, h, p).to(dt)
        s["dS"] = normal(b, h, p, n) if case["state"] else None
    return s


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def run(s):
    op = s["case"]["op"]
    if own:
        import spectral_optimizer_ssm_amd as mu
        if op == "step":
            y = mu.muon_gated_scan_step(s["v"][:, 0], s["k"][:, 0], s["q"][:, 0], s["g"][:, 0], s["S0"],
                                        gate=None if s["b"] is None else s["b"][:, 0], S_out=torch.empty_like(s["S0"]))
            return {"y": y[0], "S": y[1]}
        if op == "fwd":
            y, S = mu.muon_gated_scan(s["v"], s["k"], s["q"], s["g"], gate=s["b"], S0=s["S0"])
            return {"y": y, "S": S}
        if op == "bwd":
            r = mu.muon_gated_scan_backward(s["v"], s["k"], s["q"], s["g"], s["dy"], gate=s["b"], S0=s["S0"],
                                            dS=s["dS"])
            return dict(zip(("dv", "dk", "dq", "dg", "db", "dS0"), r))
        if op == "norm_fwd":
            y, mean, rstd = mu.muon_layer_norm(s["x"], s["w"], s["bias"], eps=EPS, center=s["case"]["center"])
            return {"y": y, "mean": mean, "rstd": rstd}
        r = mu.muon_layer_norm_backward(s["dy"], s["x"], s["w"], s["mean"], s["rstd"], center=s["case"]["center"],
                                        bias_grad=s["bias"] is not None)
        return dict(zip(("dx", "dw", "db"), r))
    if op == "step":
        return _plain_step(s)
    if op == "fwd":
        return _plain_forward(s)
    if op == "bwd":
        return _plain_backward(s)
    return _plain_norm(s) if op == "norm_fwd" else _plain_norm_backward(s)


def _plain_step(s):
    case = s["case"]
    heads = torch.arange(case["heads"], device=s["v"].device) // (case["heads"] // case["groups"])
    v, k, q = s["v"][:, 0].float(), s["k"][:, 0].float()[:, heads], s["q"][:, 0].float()[:, heads]
    if s["b"] is not None:
        v = v * s["b"][:, 0, :, None]
    S = torch.exp(s["g"][:, 0])[..., None, None] * s["S0"] + v[..., :, None] * k[..., None, :]
    y = (S * q[..., None, :]).sum(-1)
    return {"y": y.to(s["v"].dtype), "S": S}


def _chunks(x, fill=0.0):
    """[B, T, H, ...] -> float32 [B, H, T / CHUNK, CHUNK, ...], padded with `fill` tokens."""
    x = x.float()
    pad = -x.shape[1] % CHUNK
    if pad:
        x = torch.cat([x, x.new_full((x.shape[0], pad) + x.shape[2:], fill)], 1)
    return x.unflatten(1, (-1, CHUNK)).movedim(3, 1).contiguous()


def _between(g):
    """exp of the sums of g over (j, i], for i >= j (else 0): [..., n] -> [..., n, n]."""
    n = g.shape[-1]
    low = torch.ones(n, n, dtype=torch.bool, device=g.device).tril(-1)
    sums = torch.where(low, g[..., :, None], 0.0).cumsum(-2)
    keep = low | torch.eye(n, dtype=torch.bool, device=g.device)
    return torch.where(keep, torch.exp(sums), 0.0)


def _plain_parts(s):
    """What both directions need, chunk by chunk: operands by head, decays, the states before each chunk."""
    case = s["case"]
    heads = torch.arange(case["heads"], device=s["v"].device) // (case["heads"] // case["groups"])
    v, g = _chunks(s["v"]), _chunks(s["g"])
    k, q = _chunks(s["k"])[:, heads], _chunks(s["q"])[:, heads]
    b = torch.ones_like(g) if s["b"] is None else _chunks(s["b"])
    if s["b"] is None and case["tokens"] % CHUNK:
        b[:, :, -1, case["tokens"] % CHUNK:] = 0.0
    L = _between(g)                                                          # [B, H, C, i, j]
    first = torch.exp(g.cumsum(-1))                                          # from a chunk's start to i
    last = L[..., -1, :]                                                     # from j to a chunk's end
    own_part = torch.matmul(((last * b)[..., None] * v).transpose(-1, -2).contiguous(), k)   # [B, H, C, P, N]
    S0 = torch.zeros_like(own_part[:, :, 0]) if s["S0"] is None else s["S0"]
    parts = torch.cat([S0[:, :, None], own_part], 2)
    sums = g.sum(-1)
    across = _between(torch.cat([torch.zeros_like(sums[..., :1]), sums], -1))   # [B, H, C + 1, C + 1]
    states = torch.matmul(across, parts.flatten(3)).unflatten(3, parts.shape[3:])
    return v, k, q, g, b, L, first, last, across, states


def _unchunk(x, tokens):
    return x.movedim(1, 3).flatten(1, 2)[:, :tokens]


def _plain_forward(s):
    v, k, q, g, b, L, first, last, across, states = _plain_parts(s)
    scores = torch.matmul(q, k.transpose(-1, -2).contiguous()) * L * b[..., None, :]
    y = torch.matmul(scores, v)
    y = y + first[..., None] * torch.matmul(q, states[:, :, :-1].transpose(-1, -2).contiguous())
    return {"y": _unchunk(y, s["case"]["tokens"]).to(s["v"].dtype).contiguous(), "S": states[:, :, -1].contiguous()}


def _plain_backward(s):
    case, dt = s["case"], s["v"].dtype
    tokens, share = case["tokens"], (case["groups"], case["heads"] // case["groups"])
    v, k, q, g, b, L, first, last, across, states = _plain_parts(s)
    dy = _chunks(s["dy"])
    before = states[:, :, :-1]
    # gradients of the states after each chunk (index 0: of S0), in reversed time
    dpart = torch.matmul((first[..., None] * dy).transpose(-1, -2).contiguous(), q)
    end = torch.zeros_like(dpart[:, :, 0]) if s["dS"] is None else s["dS"]
    dstates = torch.cat([dpart, end[:, :, None]], 2)
    dstates = torch.matmul(across.transpose(-1, -2).contiguous(), dstates.flatten(3)).unflatten(3, dstates.shape[3:])
    after = dstates[:, :, 1:]
    A = torch.matmul(q, k.transpose(-1, -2).contiguous())
    E = torch.matmul(dy, v.transpose(-1, -2).contiguous())
    z = torch.matmul((L * A).transpose(-1, -2).contiguous(), dy)
    z_state = last[..., None] * torch.matmul(k, after.transpose(-1, -2).contiguous())
    z = z + z_state
    dv = b[..., None] * z
    db = (v * z).sum(-1)
    D = L * b[..., None, :] * E
    dq_state = first[..., None] * torch.matmul(dy, before)
    dq = torch.matmul(D, k) + dq_state
    dk = torch.matmul(D.transpose(-1, -2).contiguous(), q) + (last * b)[..., None] * torch.matmul(v, after)
    # the log decay of t scales everything that crosses t: pairs inside the chunk, the state before it read after t,
    # the tokens before t read after the chunk, and the state that passes through the chunk
    W = D * A
    inside = W.sum(-1) - W.sum(-2) + (q * dq_state).sum(-1)
    leaving = b * (v * z_state).sum(-1)
    through = L[..., -1, 0] * torch.exp(g[..., 0]) * (before * after).sum((-1, -2))
    dg = inside.flip(-1).cumsum(-1).flip(-1) + (leaving.cumsum(-1) - leaving) + through[..., None]
    dq = dq.unflatten(1, share).sum(2)
    dk = dk.unflatten(1, share).sum(2)
    return {"dv": _unchunk(dv, tokens).to(dt).contiguous(), "dk": _unchunk(dk, tokens).to(dt).contiguous(),
            "dq": _unchunk(dq, tokens).to(dt).contiguous(), "dg": _unchunk(dg, tokens).contiguous(),
            "db": None if s["b"] is None else _unchunk(db, tokens).contiguous(),
            "dS0": None if s["S0"] is None else dstates[:, :, 0].contiguous()}


def _plain_norm(s):
    x = s["x"].float()
    mean = x.mean(1) if s["case"]["center"] else None
    d = x if mean is None else x - mean[:, None]
    rstd = torch.rsqrt((d * d).mean(1) + EPS)
    y = d * rstd[:, None]
    if s["w"] is not None:
        y = y * s["w"]
    if s["bias"] is not None:
        y = y + s["bias"]
    return {"y": y.to(s["x"].dtype), "mean": mean, "rstd": rstd}


def _plain_norm_backward(s):
    x, dy = s["x"].float(), s["dy"].float()
    xh = (x if s["mean"] is None else x - s["mean"][:, None]) * s["rstd"][:, None]
    t = dy if s["w"] is None else dy * s["w"]
    dx = t - xh * (t * xh).mean(1, keepdim=True)
    if s["mean"] is not None:
        dx = dx - t.mean(1, keepdim=True)
    return {"dx": (dx * s["rstd"][:, None]).to(s["x"].dtype), "dw": None if s["w"] is None else (dy * xh).sum(0),
            "db": None if s["bias"] is None else dy.sum(0)}


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------
def work(case):
    e = 2 if case["dtype"] == "bf16" else 4
    if case["op"].startswith("norm"):
        size = case["rows"] * case["n"]
        tensors = 2 if case["op"] == "norm_fwd" else 3
        stats = 4 * case["rows"] * (2 if case["center"] else 1)
        return {"bytes": tensors * e * size + stats + 16 * case["n"],
                "flops": (8 if case["op"] == "norm_fwd" else 14) * size}
    b, t, h, g, p, n = (case[k] for k in ("batch", "tokens", "heads", "groups", "p", "n"))
    v, kq, gates, state = e * b * t * h * p, 2 * e * b * t * g * n, 4 * b * t * h * (2 if case["gate"] else 1), \
        4 * b * h * p * n
    pair = 2.0 * b * t * h * p * n      # one product of a token's vector with a state
    if case["op"] == "bwd":
        return {"bytes": 3 * v + 2 * kq + 2 * gates + (3 * state if case["state"] else 0), "flops": 5 * pair}
    return {"bytes": 2 * v + kq + gates + state * (2 if case["state"] or case["op"] == "step" else 1),
            "flops": 2 * pair}


# ---------------------------------------------------------------------------
# the definitions, token by token, in 64 bits
# ---------------------------------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    if case["op"].startswith("norm"):
        return _exact_norm(case, s)
    f64 = torch.float64
    b, t, h, g, p, n = (case[k] for k in ("batch", "tokens", "heads", "groups", "p", "n"))
    v, k, q = (s[x].to(f64) for x in ("v", "k", "q"))
    k, q = (x.repeat_interleave(h // g, 2) for x in (k, q))
    decay = torch.exp(s["g"].to(f64))
    gate = torch.ones_like(decay) if s["b"] is None else s["b"].to(f64)
    S = torch.zeros(b, h, p, n, dtype=f64, device=v.device) if s["S0"] is None else s["S0"].to(f64)
    kept, y = [S], []
    for i in range(t):
        S = decay[:, i, :, None, None] * S + (gate[:, i, :, None] * v[:, i])[..., None] * k[:, i, :, None, :]
        if case["op"] == "bwd":
            kept.append(S)
        else:
            y.append(torch.matmul(S, q[:, i, :, :, None])[..., 0])
    if case["op"] == "step":
        return {"y": y[0], "S": S}
    if case["op"] == "fwd":
        return {"y": torch.stack(y, 1), "S": S}
    dy = s["dy"].to(f64)
    dS = torch.zeros_like(S) if s["dS"] is None else s["dS"].to(f64)
    dv, dk, dq, dg, db = (torch.zeros_like(x) for x in (v, k, q, decay, decay))
    for i in reversed(range(t)):
        dS = dS + dy[:, i, :, :, None] * q[:, i, :, None, :]
        dq[:, i] = (kept[i + 1] * dy[:, i, :, :, None]).sum(2)
        read = (dS * k[:, i, :, None, :]).sum(3)
        dv[:, i] = gate[:, i, :, None] * read
        db[:, i] = (v[:, i] * read).sum(2)
        dk[:, i] = gate[:, i, :, None] * (dS * v[:, i, :, :, None]).sum(2)
        dS = decay[:, i, :, None, None] * dS
        dg[:, i] = (dS * kept[i]).sum((2, 3))
        kept.pop()
    return {"dv": dv, "dk": dk.unflatten(2, (g, h // g)).sum(3), "dq": dq.unflatten(2, (g, h // g)).sum(3), "dg": dg,
            "db": None if s["b"] is None else db, "dS0": None if s["S0"] is None else dS}


def _exact_norm(case, s):
    x = s["x"].double()
    mean = x.mean(1, keepdim=True) if case["center"] else torch.zeros_like(x[:, :1])
    rstd = 1.0 / torch.sqrt(((x - mean) ** 2).mean(1, keepdim=True) + EPS)
    w = torch.ones_like(x[0]) if s["w"] is None else s["w"].double()
    if case["op"] == "norm_fwd":
        y = (x - mean) * rstd * w
        return {"y": y if s["bias"] is None else y + s["bias"].double(), "mean": mean[:, 0] if case["center"] else None,
                "rstd": rstd[:, 0]}
    # the statistics are inputs of the backward pass
    mean = s["mean"].double()[:, None] if case["center"] else mean
    rstd = s["rstd"].double()[:, None]
    dy = s["dy"].double()
    xh = (x - mean) * rstd
    dxh = dy * w
    part = dxh - dxh.mean(1, keepdim=True) if case["center"] else dxh
    return {"dx": rstd * (part - xh * (dxh * xh).mean(1, keepdim=True)), "dw": None if s["w"] is None else (dy * xh).sum(0),
            "db": None if s["bias"] is None else dy.sum(0)}
