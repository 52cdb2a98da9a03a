"""Performance cases of the token embedding, the gated group norm and the token
log probabilities: what a Mamba-2 language model has around its scan.

listed() holds fixed cases, draw() makes more of the same ranges, prepare()
makes a case's inputs and run() does one pass: through the library's entry
points where `own` is true, else in plain torch operations in float32.

Embedding: y_t = scale table[id_t]; its gradient dtable[v] = scale times the
sum of dy_t over the tokens with id v.  Ids outside the table (padding) give
zeros and take no gradient.

Group norm of rows whose channels are cut into groups, with a gate z:
    before:  y = norm(x silu(z)) w + bias
    after:   y = (norm(x) w + bias) silu(z)
    none:    y = silu(norm(x) w + bias)
norm takes each group of channels of a row by itself, with or without its mean.

Log probabilities: for each row of logits x and its token t
    log p_t = scale x_t - log sum_j exp(scale x_j),   H = -sum_j p_j log p_j,
and the k likeliest tokens (ties: the lowest index first); the gradient of a
loss by the logits from its gradients by log p_t and H.  Rows whose token is
outside the vocabulary (padding) have log p 0 and no gradient by it.

The shapes are those of Mamba-2 130M (d_model 768, inner width 1536, 24 heads,
vocabulary 50,280) and odd ones around them.
"""
import math

import torch

own = False

EPS = 1e-5
VOCAB, D_MODEL, D_INNER, HEADS = 50280, 768, 1536, 24    # Mamba-2 130M
TRAIN = 8 * 2048                                         # tokens of a training batch


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def _embed(name, op, tokens, vocab=VOCAB, n=D_MODEL, dtype="bf16", table="f32", scale=1.0, padding=0.0):
    """dtype: of the rows looked up and of their gradient; table: of the table
    and of its gradient; padding: the share of tokens that are padding."""
    return dict(name=name, op=op, tokens=tokens, vocab=vocab, n=n, dtype=dtype, table=table, scale=scale, padding=padding)


def _norm(name, op, rows, n=D_INNER, groups=1, dtype="bf16", center=False, affine=True, gate="before"):
    return dict(name=name, op=op, rows=rows, n=n, groups=groups, dtype=dtype, center=center, affine=affine, gate=gate)


def _logp(name, op, rows, vocab=VOCAB, dtype="bf16", scale=1.0, top=0, entropy=True, pad=0, mask="none", padding=0.0):
    """pad: unused columns behind each row; mask: what a quarter of the tokens
    is set to; padding: the share of rows without a token."""
    return dict(name=name, op=op, rows=rows, vocab=vocab, dtype=dtype, scale=scale, top=top, entropy=entropy, pad=pad,
                mask=mask, padding=padding)


def listed():
    return [
        # the tokens of a decode batch: latency
        _embed("embed_fwd_decode", "embed_fwd", 32),
        # a training batch, looked up in the float32 master table
        _embed("embed_fwd_train", "embed_fwd", TRAIN),
        # the table's gradient for a training batch: most of the table is written as zero
        _embed("embed_bwd_train", "embed_bwd", TRAIN, padding=0.02),
        # many tokens of an odd width, some of them thousands of times, with scaled embeddings
        _embed("embed_bwd_long", "embed_bwd", 16 * 8192 - 1, n=515, scale=22.6875),
        # the norm behind the scan: a training batch, and its gradients with the gate's and the weight's
        _norm("group_norm_fwd_train", "norm_fwd", TRAIN),
        _norm("group_norm_bwd_train", "norm_bwd", TRAIN),
        # the same in a decode batch: latency
        _norm("group_norm_fwd_decode", "norm_fwd", 32),
        # a group for each head, centred, odd width, gate behind the norm, float32
        _norm("group_norm_bwd_heads_f32", "norm_bwd", 2 * 1031, n=HEADS * 75, groups=HEADS, dtype="f32", center=True,
              gate="after"),
        # what a decoder answers with: four sequences, the chosen token's log probability and the 20 likeliest
        _logp("logp_fwd_decode", "logp_fwd", 4, top=20, pad=8),
        # scoring of texts with alternatives: float32 logits, a temperature, some tokens forbidden
        _logp("logp_fwd_top_f32", "logp_fwd", 1021, vocab=50277, dtype="f32", scale=1.25, top=20, mask="inf"),
        # the loss of a training batch, and its gradient by the logits
        _logp("logp_fwd_train", "logp_fwd", TRAIN, pad=8, padding=0.02),
        _logp("logp_bwd_train", "logp_bwd", TRAIN, pad=8, padding=0.02),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["embed_fwd", "embed_bwd", "embed_bwd", "norm_fwd", "norm_bwd", "logp_fwd", "logp_fwd", "logp_bwd"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op.startswith("embed"):
        n = rng.choice([D_MODEL, _log_int(rng, 16, 2048)])
        vocab = rng.choice([VOCAB, _log_int(rng, 100, 100000)])
        vocab = min(vocab, VOCAB * D_MODEL // n)
        tokens = _log_int(rng, 1, min(16 * 8192, 16 * 8192 * 515 // n))
        c = _embed("", op, tokens, vocab, n, dtype, rng.choice(["f32", "f32", "bf16"]),
                   scale=rng.choice([1.0, round(math.sqrt(n), 3)]), padding=rng.choice([0.0, 0.1]))
    elif op.startswith("norm"):
        groups = rng.choice([1, 1, 2, 8, HEADS])
        width = rng.choice([D_INNER // groups, _log_int(rng, 16, 4096 // min(groups, 16))])
        n = groups * width
        rows = _log_int(rng, 1, max(2, TRAIN * D_INNER // n // (1 if dtype == "bf16" else 2)))
        c = _norm("", op, rows, n, groups, dtype, center=rng.random() < 0.4, affine=rng.random() < 0.8,
                  gate=rng.choice(["before", "before", "after", "none"]))
    else:
        vocab = rng.choice([VOCAB, _log_int(rng, 250, 150000)])
        rows = _log_int(rng, 1, max(2, min(TRAIN, TRAIN * VOCAB // vocab) // (1 if dtype == "bf16" else 2)))
        top = rng.choice([0, 0, 1, 5, 20, 50]) if op == "logp_fwd" and rows <= 4096 else 0
        c = _logp("", op, rows, vocab, dtype, scale=rng.choice([1.0, 1.0, 1.25, 0.7]), top=top,
                  entropy=rng.random() < 0.7, pad=rng.choice([0, 1, 8]), mask=rng.choice(["none", "none", "inf", "lowest"]),
                  padding=rng.choice([0.0, 0.1]))
    del c["name"]
    return c


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
_TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def prepare(case, seed):
    dev = torch.device("cuda" if torch.cuda.is_available() else "cpu")
    gen = torch.Generator(device=dev).manual_seed(seed)
    dt, op = _TYPES[case["dtype"]], case["op"]

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device=dev)

    def uniform(*shape):
        return torch.rand(*shape, generator=gen, device=dev)

    def token_ids(count, vocab):
        # a token's share goes with one over its rank; ranks are spread over the vocabulary
        rank = (torch.exp(uniform(count).double() * math.log(vocab)) - 1.0).long().clamp_(0, vocab - 1)
        step = 7919 if vocab % 7919 else 7907
        return torch.where(uniform(count) < case["padding"], -1, rank * step % vocab)

    s = {"case": case}
    if op.startswith("embed"):
        s["ids"] = token_ids(case["tokens"], case["vocab"])
        if op == "embed_fwd":
            s["table"] = (0.02 * normal(case["vocab"], case["n"])).to(_TYPES[case["table"]])
        else:
            s["dy"] = normal(case["tokens"], case["n"]).to(dt)
    elif op.startswith("norm"):
        rows, n, groups = case["rows"], case["n"], case["groups"]
        s["x"] = (normal(rows, n) * (0.5 + uniform(n)) + 0.3 * normal(n)).to(dt)
        s["z"] = None
        if case["gate"] != "none":
            # a column range of the projection's output
            s["z"] = normal(rows, n + 8).to(dt)[:, :n]
        s["w"] = 1.0 + 0.2 * normal(n) if case["affine"] else None
        s["bias"] = 0.1 * normal(n) if case["affine"] and case["center"] else None
        if op == "norm_bwd":
            s["dy"] = normal(rows, n).to(dt)
            u = s["x"].float()      # the statistics that the forward pass kept
            if case["gate"] == "before":
                u = u * torch.nn.functional.silu(s["z"].float())
            u = u.unflatten(1, (groups, -1))
            s["mean"] = u.mean(2) if case["center"] else None
            d = u - s["mean"][..., None] if case["center"] else u
            s["rstd"] = torch.rsqrt((d * d).mean(2) + EPS)
    else:
        rows, vocab = case["rows"], case["vocab"]
        s["tokens"] = token_ids(rows, vocab)
        # around the tokens' frequencies
        step = 7919 if vocab % 7919 else 7907
        often = torch.empty(vocab, device=dev)
        ranks = torch.arange(vocab, device=dev)
        often[ranks * step % vocab] = -torch.log1p(ranks.float())
        wide = torch.empty(rows, vocab + case["pad"], dtype=dt, device=dev)
        x = wide[:, :vocab]
        for a in range(0, rows, 2048):
            b = min(rows, a + 2048)
            x[a:b] = (2.0 * normal(b - a, vocab) + often).to(dt)
        if case["mask"] != "none":
            x[:, 3::4] = -math.inf if case["mask"] == "inf" else torch.finfo(dt).min
            s["tokens"] = torch.where(s["tokens"] % 4 == 3, s["tokens"] - 1, s["tokens"])
            s["tokens"] = torch.where(s["tokens"] < 0, -1, s["tokens"])
        s["x"] = x
        if op == "logp_bwd":
            # the mean loss over the batch, and a weight on the entropy
            s["dlogp"] = -(0.5 + uniform(rows)) / rows
            s["dentropy"] = 0.01 * normal(rows) / rows if case["entropy"] else None
            largest, logsum, entropy = [], [], []
            for a in range(0, rows, 2048):      # the statistics that the forward pass kept
                t = x[a:a + 2048].float()
                m = t.max(1).values
                t = (t - m[:, None]) * case["scale"]
                e = torch.exp(t)
                total = e.sum(1)
                largest.append(m)
                logsum.append(torch.log(total))
                entropy.append(logsum[-1] - (e * t.clamp_min(-1e4)).sum(1) / total)
            s["stats"] = torch.stack([torch.cat(largest), torch.cat(logsum)], 1)
            s["entropy"] = torch.cat(entropy)
    return s


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def run(s):
    case = s["case"]
    op = case["op"]
    if own:
        import spectral_optimizer_ssm_amd as mu
        if op == "embed_fwd":
            return {"y": mu.muon_embedding(s["table"], s["ids"], scale=case["scale"], dtype=_TYPES[case["dtype"]])}
        if op == "embed_bwd":
            return {"dtable": mu.muon_embedding_backward(s["dy"], s["ids"], case["vocab"], scale=case["scale"],
                                                         dtype=_TYPES[case["table"]])}
        if op == "norm_fwd":
            y, mean, rstd = mu.muon_group_norm(s["x"], case["groups"], s["w"], s["bias"], gate=s["z"],
                                               gate_first=case["gate"] == "before", eps=EPS, center=case["center"])
            return {"y": y, "mean": mean, "rstd": rstd}
        if op == "norm_bwd":
            r = mu.muon_group_norm_backward(s["dy"], s["x"], case["groups"], s["w"], s["bias"], s["mean"], s["rstd"],
                                            gate=s["z"], gate_first=case["gate"] == "before", center=case["center"])
            return dict(zip(("dx", "dz", "dw", "db"), r))
        if op == "logp_fwd":
            logp, entropy, stats, ids, logps = mu.muon_token_logprobs(s["x"], s["tokens"], scale=case["scale"],
                                                                      entropy=case["entropy"], top=case["top"])
            return {"logp": logp, "entropy": entropy, "stats": stats, "ids": ids, "logps": logps}
        return {"dx": mu.muon_token_logprobs_backward(s["x"], s["tokens"], s["stats"], s["dlogp"], scale=case["scale"],
                                                      entropy=s["entropy"] if case["entropy"] else None,
                                                      dentropy=s["dentropy"])}
    return {"embed_fwd": _plain_embed, "embed_bwd": _plain_embed_backward, "norm_fwd": _plain_norm,
            "norm_bwd": _plain_norm_backward, "logp_fwd": _plain_logp, "logp_bwd": _plain_logp_backward}[op](s)


def _plain_embed(s):
    case = s["case"]
    there = (s["ids"] >= 0) & (s["ids"] < case["vocab"])
    y = s["table"][torch.where(there, s["ids"], 0)].float() * case["scale"]
    return {"y": torch.where(there[:, None], y, 0.0).to(_TYPES[case["dtype"]])}


def _plain_embed_backward(s):
    case = s["case"]
    there = (s["ids"] >= 0) & (s["ids"] < case["vocab"])
    d = torch.zeros(case["vocab"], case["n"], device=s["dy"].device)
    d.index_add_(0, torch.where(there, s["ids"], 0), torch.where(there[:, None], s["dy"].float() * case["scale"], 0.0))
    return {"dtable": d.to(_TYPES[case["table"]])}


def _plain_silu(z):
    return z / (1.0 + torch.exp(-z))


def _plain_silu_slope(z):
    p = 1.0 / (1.0 + torch.exp(-z))
    return p * (1.0 + z * (1.0 - p))


def _plain_norm(s):
    case = s["case"]
    u, z = s["x"].float(), None if s["z"] is None else s["z"].float()
    if case["gate"] == "before":
        u = u * _plain_silu(z)
    u = u.unflatten(1, (case["groups"], -1))
    mean = u.mean(2) if case["center"] else None
    d = u if mean is None else u - mean[..., None]
    rstd = torch.rsqrt((d * d).mean(2) + EPS)
    y = (d * rstd[..., None]).flatten(1)
    if s["w"] is not None:
        y = y * s["w"]
    if s["bias"] is not None:
        y = y + s["bias"]
    if case["gate"] == "after":
        y = y * _plain_silu(z)
    elif case["gate"] == "none":
        y = _plain_silu(y)
    return {"y": y.to(s["x"].dtype), "mean": mean, "rstd": rstd}


def _plain_norm_backward(s):
    case, dt = s["case"], s["x"].dtype
    groups = (case["groups"], -1)
    x, dy, z = s["x"].float(), s["dy"].float(), None if s["z"] is None else s["z"].float()
    u = x * _plain_silu(z) if case["gate"] == "before" else x
    u = u.unflatten(1, groups)
    xh = ((u if s["mean"] is None else u - s["mean"][..., None]) * s["rstd"][..., None]).flatten(1)
    o = xh if s["w"] is None else xh * s["w"]
    if s["bias"] is not None:
        o = o + s["bias"]
    dz = None
    if case["gate"] == "after":
        dz = dy * o * _plain_silu_slope(z)
        dy = dy * _plain_silu(z)
    elif case["gate"] == "none":
        dy = dy * _plain_silu_slope(o)
    t = (dy if s["w"] is None else dy * s["w"]).unflatten(1, groups)
    xg = xh.unflatten(1, groups)
    du = t - xg * (t * xg).mean(2, keepdim=True)
    if s["mean"] is not None:
        du = du - t.mean(2, keepdim=True)
    du = (du * s["rstd"][..., None]).flatten(1)
    if case["gate"] == "before":
        dz = du * x * _plain_silu_slope(z)
        du = du * _plain_silu(z)
    return {"dx": du.to(dt), "dz": None if dz is None else dz.to(dt), "dw": None if s["w"] is None else (dy * xh).sum(0),
            "db": None if s["bias"] is None else dy.sum(0)}


def _plain_logp(s):
    case = s["case"]
    x, vocab = s["x"].float(), case["vocab"]
    there = (s["tokens"] >= 0) & (s["tokens"] < vocab)
    m = x.max(1).values
    t = (x - m[:, None]) * case["scale"]
    e = torch.exp(t)
    total = e.sum(1)
    logsum = torch.log(total)
    rows = torch.arange(x.shape[0], device=x.device)
    chosen = t[rows, torch.where(there, s["tokens"], 0)] - logsum
    entropy = logsum - (e * t.clamp_min(-1e4)).sum(1) / total if case["entropy"] else None
    ids = logps = None
    if case["top"]:
        # one whole number orders by logit, then by the lowest index
        bits = (x + 0.0).view(torch.int32).long()
        order = torch.where(bits < 0, bits ^ 0x7FFFFFFF, bits) * 2 ** 31 + (2 ** 31 - 1 - torch.arange(vocab, device=x.device))
        ids = 2 ** 31 - 1 - torch.topk(order, case["top"], 1).values.remainder(2 ** 31)
        logps = t.gather(1, ids) - logsum[:, None]
        ids = ids.int()
    return {"logp": torch.where(there, chosen, 0.0), "entropy": entropy, "stats": torch.stack([m, logsum], 1), "ids": ids,
            "logps": logps}


def _plain_logp_backward(s):
    case = s["case"]
    t = (s["x"].float() - s["stats"][:, :1]) * case["scale"] - s["stats"][:, 1:]
    p = torch.exp(t)
    there = (s["tokens"] >= 0) & (s["tokens"] < case["vocab"])
    dlogp = torch.where(there, s["dlogp"], 0.0)
    d = -dlogp[:, None] * p
    if s["dentropy"] is not None:
        d = d - s["dentropy"][:, None] * p * (t.clamp_min(-1e4) + s["entropy"][:, None])
    rows = torch.arange(d.shape[0], device=d.device)
    d[rows, torch.where(there, s["tokens"], 0)] += dlogp
    return {"dx": (d * case["scale"]).to(s["x"].dtype)}


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------
def work(case):
    e, op = (2 if case["dtype"] == "bf16" else 4), case["op"]
    if op.startswith("embed"):
        tokens, n = case["tokens"], case["n"]
        et = 2 if case["table"] == "bf16" else 4
        if op == "embed_bwd":
            return {"bytes": tokens * (8 + n * e) + case["vocab"] * n * et, "flops": tokens * n}
        # rows of the table that are read: shares 1 / (rank ln vocab)
        log_vocab = math.log(case["vocab"])
        rows = sum(1.0 - (1.0 - min(1.0, 1.0 / ((r + 0.5) * log_vocab))) ** tokens for r in range(case["vocab"]))
        return {"bytes": tokens * (8 + n * e) + min(rows, tokens) * n * et, "flops": tokens * n}
    if op.startswith("norm"):
        size = case["rows"] * case["n"]
        gate = 0 if case["gate"] == "none" else 1
        stats = 4 * case["rows"] * case["groups"] * (2 if case["center"] else 1)
        params = 4 * case["n"] * ((2 if case["center"] else 1) if case["affine"] else 0)
        if op == "norm_fwd":
            return {"bytes": (2 + gate) * e * size + stats + params, "flops": 14 * size}
        return {"bytes": (3 + 2 * gate) * e * size + stats + 2 * params, "flops": 28 * size}
    size = case["rows"] * case["vocab"]
    small = case["rows"] * (8 + 4 + 8 + (4 if case["entropy"] else 0) + 8 * case["top"])
    if op == "logp_fwd":
        return {"bytes": e * size + small, "flops": 6 * size}
    return {"bytes": 2 * e * size + small, "flops": 8 * size}


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op.startswith("embed"):
        return _exact_embed(case, s)
    if op.startswith("norm"):
        return _exact_norm(case, s)
    out = []
    for a in range(0, case["rows"], 512):
        part = {k: v[a:a + 512] if torch.is_tensor(v) else v for k, v in s.items()}
        out.append(_exact_logp(case, part))
    return {k: None if out[0][k] is None else torch.cat([o[k] for o in out]) for k in out[0]}


def _exact_embed(case, s):
    ids = s["ids"]
    keep = torch.nonzero((ids >= 0) & (ids < case["vocab"]))[:, 0]
    if case["op"] == "embed_fwd":
        y = torch.zeros(case["tokens"], case["n"], dtype=torch.float64, device=ids.device)
        y[keep] = s["table"].double()[ids[keep]] * case["scale"]
        return {"y": y}
    order = keep[torch.sort(ids[keep], stable=True).indices]
    d = torch.zeros(case["vocab"], case["n"], dtype=torch.float64, device=ids.device)
    d.index_put_((ids[order],), s["dy"].double()[order], accumulate=True)
    return {"dtable": d * case["scale"]}


def _exact_norm(case, s):
    f64 = torch.float64
    rows, groups = case["rows"], case["groups"]
    w = torch.ones(case["n"], dtype=f64, device=s["x"].device) if s["w"] is None else s["w"].double()
    bias = torch.zeros_like(w) if s["bias"] is None else s["bias"].double()
    x = s["x"].double()
    z = None if s["z"] is None else s["z"].double()
    a = None if z is None else z * torch.sigmoid(z)
    u = (x * a if case["gate"] == "before" else x).reshape(rows, groups, -1)
    if case["op"] == "norm_fwd":
        mean = u.mean(2, keepdim=True) if case["center"] else torch.zeros_like(u[:, :, :1])
        rstd = 1.0 / torch.sqrt((u - mean).square().mean(2, keepdim=True) + EPS)
    else:   # the statistics are inputs of the backward pass
        mean = s["mean"].double()[..., None] if case["center"] else torch.zeros_like(u[:, :, :1])
        rstd = s["rstd"].double()[..., None]
    xh = ((u - mean) * rstd).reshape(rows, -1)
    o = xh * w + bias
    if case["op"] == "norm_fwd":
        y = o if case["gate"] == "before" else o * a if case["gate"] == "after" else o * torch.sigmoid(o)
        return {"y": y, "mean": mean[..., 0] if case["center"] else None, "rstd": rstd[..., 0]}
    dy = s["dy"].double()

    def slope(v):
        sig = torch.sigmoid(v)
        return sig + v * sig * (1.0 - sig)

    do = dy if case["gate"] == "before" else dy * a if case["gate"] == "after" else dy * slope(o)
    dxh = (do * w).reshape(rows, groups, -1)
    xg = xh.reshape(rows, groups, -1)
    part = dxh - dxh.mean(2, keepdim=True) if case["center"] else dxh
    du = (rstd * (part - xg * (dxh * xg).mean(2, keepdim=True))).reshape(rows, -1)
    dz = None if z is None else (du * x if case["gate"] == "before" else dy * o) * slope(z)
    return {"dx": du * a if case["gate"] == "before" else du, "dz": dz,
            "dw": None if s["w"] is None else (do * xh).sum(0), "db": None if s["bias"] is None else do.sum(0)}


def _exact_logp(case, s):
    raw, tokens = s["x"].double(), s["tokens"]
    x = raw * case["scale"]
    logp = torch.log_softmax(x, 1)
    p = torch.exp(logp)
    there = ((tokens >= 0) & (tokens < case["vocab"])).double()
    at = tokens.clamp(0, case["vocab"] - 1)[:, None]
    plogp = torch.where(p > 0, p * logp, torch.zeros_like(p))
    if case["op"] == "logp_bwd":
        # the statistics are inputs of the backward pass
        logp = (raw - s["stats"][:, :1].double()) * case["scale"] - s["stats"][:, 1:].double()
        p = torch.exp(logp)
        plogp = torch.where(p > 0, p * logp, torch.zeros_like(p))
        dlogp = (s["dlogp"].double() * there)[:, None]
        d = -dlogp * p
        if s["dentropy"] is not None:
            d = d - s["dentropy"].double()[:, None] * (plogp + s["entropy"].double()[:, None] * p)
        return {"dx": case["scale"] * d.scatter_add(1, at, dlogp)}
    chosen = torch.where(there > 0, logp.gather(1, at)[:, 0], torch.zeros_like(there))
    ids = logps = None
    if case["top"]:
        order = torch.sort(raw, dim=1, descending=True, stable=True)
        ids = order.indices[:, :case["top"]].int()
        logps = logp.gather(1, ids.long())
    largest = raw.max(1).values
    return {"logp": chosen, "entropy": -plogp.sum(1) if case["entropy"] else None,
            "stats": torch.stack([largest, torch.logsumexp(x, 1) - largest * case["scale"]], 1), "ids": ids, "logps": logps}
