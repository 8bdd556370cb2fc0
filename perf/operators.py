"""The training operators around the AdamW parameters, as cases to be timed and compared.

The embedding table, the normalisation gains and the logits that the LM head produces: lookup
with its gradient by sorted tokens, that gradient taken straight into the AdamW step, layer
norm in both directions, and the distillation loss on a teacher's top logits.  ``run`` computes
a case in elementary torch operations in 32 bits, or, where ``own`` is true, by the library's
entry points.  Sizes follow workloads/configs.py: vocabularies of 65536 and 128000 and hidden
sizes of 768, 1280, 2048 and 8192.
"""
import math

import numpy as np
import torch

own = False

TYPES = {"fp32": torch.float32, "fp16": torch.float16, "bf16": torch.bfloat16}
BYTES = {"fp32": 4, "fp16": 2, "bf16": 2}
ADAMW = dict(lr=3e-3, beta1=0.9, beta2=0.95, eps=1e-8, weight_decay=0.1)
STEP = 10
LN_EPS = 1e-5


def listed():
    return [
        # one decode step of eight sequences: latency only
        dict(name="lookup_8_tokens", op="lookup", rows=65536, dim=768, tokens=8, pad=0, type="bf16"),
        # a training micro-batch of the 24-layer model, the last sequence padded
        dict(name="lookup_16k_tokens", op="lookup", rows=128000, dim=2048, tokens=16384, pad=517, type="bf16"),
        # one of several micro-batches whose gradients add up before a step; a ragged batch
        dict(name="table_grad_added_8191", op="table_grad", rows=65536, dim=1280, tokens=8191, pad=0, type="bf16", add=True),
        # a whole batch's gradient of the 24-layer model's table, written densely
        dict(name="table_grad_64k_tokens", op="table_grad", rows=128000, dim=2048, tokens=65536, pad=4001, type="bf16", add=False),
        # the smallest table of the workloads
        dict(name="table_step_tiny", op="table_step", rows=512, dim=64, tokens=100, pad=3, type="fp32"),
        # the optimizer's step on the 20-layer model's table from one batch's tokens
        dict(name="table_step_16k_tokens", op="table_step", rows=65536, dim=1280, tokens=16384, pad=0, type="bf16"),
        # a few rows in full precision, as in an evaluation loop: latency only
        dict(name="norm_63_rows", op="norm", n=63, dim=768, type="fp32", bias=True),
        # a training micro-batch of the 24-layer model, gains only
        dict(name="norm_32k_rows", op="norm", n=32768, dim=2048, type="bf16", bias=False),
        # a short ragged batch of the 20-layer model in full precision
        dict(name="norm_grad_1023_rows", op="norm_grad", n=1023, dim=1280, type="fp32", bias=True),
        # a training micro-batch of the widest model
        dict(name="norm_grad_16k_rows", op="norm_grad", n=16384, dim=8192, type="bf16", bias=True),
        # loss, then gradient, as an autograd graph calls them; short teacher lists, empty rows
        dict(name="distill_511_rows", op="distill", n=511, vocab=65536, stride=65536, top=50, type="fp16", temperature=2.0),
        # loss and gradient in one call on the 24-layer model's logits, rows padded to 128256
        dict(name="distill_step_4k_rows", op="distill_step", n=4096, vocab=128000, stride=128256, top=128, type="bf16", temperature=1.0),
    ]


def _spread(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(["lookup", "table_grad", "table_step", "norm", "norm_grad", "distill_loss", "distill", "distill_step"])
    kind = rng.choice(["fp32", "fp16", "bf16", "bf16"])
    if op in ("lookup", "table_grad", "table_step"):
        dim = _spread(rng, 33, 8192)
        dim = dim if rng.random() < 0.3 else (dim + 7) // 8 * 8
        most = 65536 * 1024 if op == "table_step" else 131072 * 1280
        rows = _spread(rng, 500, min(131072, most // dim))
        tokens = _spread(rng, 1, min(65536, most // 2 // dim))
        case = dict(op=op, rows=rows, dim=dim, tokens=tokens, pad=rng.choice([0, tokens // 9]), type=kind)
        return dict(case, add=rng.random() < 0.5) if op == "table_grad" else case
    if op in ("norm", "norm_grad"):
        dim = _spread(rng, 33, 16384)
        dim = dim if rng.random() < 0.3 else (dim + 7) // 8 * 8
        return dict(op=op, n=_spread(rng, 1, min(65536, 65536 * 1024 // dim)), dim=dim, type=kind, bias=rng.random() < 0.5)
    vocab = _spread(rng, 500, 131072)
    return dict(op=op, n=_spread(rng, 1, min(16384, 2048 * 65536 // vocab)), vocab=vocab,
                stride=vocab if rng.random() < 0.5 else (vocab + 127) // 128 * 128,
                top=min(vocab, _spread(rng, 1, 256)), type=kind, temperature=rng.choice([0.7, 1.0, 2.0, 4.0]))


def _normal(g, *shape, scale=1.0, dtype=torch.float32):
    return (torch.randn(*shape, generator=g, device="cuda") * scale).to(dtype)


def _tokens(g, case):
    """Frequent tokens have small ids, as in a vocabulary ordered by frequency: id v with a
    probability near 1 / ((v + 1) ln rows).  The padding at the batch's end is -1."""
    u = torch.rand(case["tokens"], generator=g, device="cuda", dtype=torch.float64)
    t = (torch.exp(u * math.log(case["rows"])).floor().long() - 1).clamp_(0, case["rows"] - 1)
    if case["pad"]:
        t[case["tokens"] - case["pad"]:] = -1
    return t


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    op, dtype = case["op"], TYPES[case["type"]]
    s = {"case": case}
    if op in ("lookup", "table_grad", "table_step"):
        rows, dim = case["rows"], case["dim"]
        s["tokens"] = _tokens(g, case)
        s["scale"] = math.sqrt(dim)
        if op != "lookup":
            s["dout"] = _normal(g, case["tokens"], dim, scale=1e-3, dtype=dtype)
        if op == "lookup":
            s["table"] = _normal(g, rows, dim, scale=0.02)
        elif op == "table_grad":
            if case["add"]:
                s["grad"] = _normal(g, rows, dim, scale=1e-2)
        else:
            s["param"] = _normal(g, rows, dim, scale=0.02)
            s["exp_avg"] = _normal(g, rows, dim, scale=1e-2)
            s["exp_avg_sq"] = _normal(g, rows, dim, scale=1e-2).square_()
    elif op in ("norm", "norm_grad"):
        n, dim = case["n"], case["dim"]
        # a few channels carry most of the energy, as in a residual stream
        channel = 1.0 + 10.0 * (torch.rand(dim, generator=g, device="cuda") < 0.01)
        s["x"] = (_normal(g, n, dim) * channel + 0.25).to(dtype)
        s["weight"] = 1.0 + _normal(g, dim, scale=0.1)
        s["bias"] = _normal(g, dim, scale=0.1) if case["bias"] else None
        if op == "norm_grad":
            s["dy"] = _normal(g, n, dim, scale=1e-2, dtype=dtype)
            # what the forward pass kept
            x = s["x"].float()
            s["mean"] = x.mean(1)
            s["rstd"] = 1.0 / torch.sqrt((x - s["mean"][:, None]).square().mean(1) + LN_EPS)
    else:
        n, vocab, top = case["n"], case["vocab"], case["top"]
        first = torch.randint(0, vocab, (n, 1), generator=g, device="cuda")
        ids = (first + torch.arange(top, device="cuda") * max(1, vocab // top)) % vocab
        teacher = torch.sort(_normal(g, n, top, scale=2.0), dim=1, descending=True).values
        logits = _normal(g, n, case["stride"], scale=2.0)
        logits.scatter_add_(1, ids, teacher + 4.0)
        # every ninth teacher list is short, every 31st row has none (padding)
        row = torch.arange(n, device="cuda")[:, None]
        short = (row % 9 == 4) & (torch.arange(top, device="cuda") >= (top + 1) // 2)
        none = row % 31 == 17
        s["logits"] = logits.to(dtype)[:, :vocab]
        s["ids"] = torch.where(short | none, torch.full_like(ids, -1), ids)
        s["teacher"] = teacher.to(dtype)
        # the mean over the rows; with the usual loss scale where fp16 would lose small gradients
        s["weight"] = torch.where(none[:, 0], 0.0, (65536.0 if case["type"] == "fp16" else 1.0) / n).float()
    return s


def work(case):
    op, b = case["op"], BYTES[case["type"]]
    if op in ("lookup", "table_grad", "table_step"):
        rows, dim, live = case["rows"], case["dim"], case["tokens"] - case["pad"]
        v = np.arange(rows, dtype=np.float64)
        p = np.log1p(1.0 / (v + 1.0)) / math.log(rows)
        distinct = float(np.sum(-np.expm1(live * np.log1p(-np.minimum(p, 0.999)))))
        if op == "lookup":
            return {"bytes": case["tokens"] * (8 + dim * b) + distinct * dim * 4, "flops": live * dim}
        if op == "table_step":
            return {"bytes": case["tokens"] * 8 + live * dim * b + rows * dim * 24, "flops": live * dim + rows * dim * 14}
        grad = distinct * dim * 8 if case["add"] else rows * dim * 4
        return {"bytes": case["tokens"] * 8 + live * dim * b + grad, "flops": live * dim + distinct * dim}
    if op == "norm":
        return {"bytes": case["n"] * (2 * case["dim"] * b + 8) + case["dim"] * 4 * (1 + case["bias"]), "flops": 8 * case["n"] * case["dim"]}
    if op == "norm_grad":
        return {"bytes": case["n"] * (3 * case["dim"] * b + 8) + case["dim"] * 4 * (2 + case["bias"]), "flops": 14 * case["n"] * case["dim"]}
    logits = case["n"] * case["vocab"]
    lists = case["n"] * (case["top"] * (8 + b) + 4)
    if op == "distill_loss":
        return {"bytes": logits * b + lists, "flops": 4 * logits}
    return {"bytes": 2 * logits * b + lists, "flops": 6 * logits}


# ---------------------------------------------------------------- the plain forms
def _table_grad(s, rows):
    case = s["case"]
    live = (s["tokens"] >= 0) & (s["tokens"] < rows)
    at = torch.where(live, s["tokens"], 0)
    d = torch.where(live[:, None], s["dout"].float() * s["scale"], 0.0)
    return torch.zeros(rows, case["dim"], device=d.device).index_add_(0, at, d)


def _table_step(s):
    p, m, v, h = s["param"], s["exp_avg"], s["exp_avg_sq"], ADAMW
    g = _table_grad(s, p.shape[0])
    m.mul_(h["beta1"]).add_(g, alpha=1.0 - h["beta1"])
    v.mul_(h["beta2"]).add_(g * g, alpha=1.0 - h["beta2"])
    update = (m / (1.0 - h["beta1"] ** STEP)) / (torch.sqrt(v / (1.0 - h["beta2"] ** STEP)) + h["eps"])
    p.mul_(1.0 - h["lr"] * h["weight_decay"]).add_(update, alpha=-h["lr"])
    return p, m, v


def _norm(s):
    x = s["x"].float()
    mean = x.mean(1, keepdim=True)
    c = x - mean
    rstd = 1.0 / torch.sqrt((c * c).mean(1, keepdim=True) + LN_EPS)
    y = c * rstd * s["weight"]
    if s["bias"] is not None:
        y = y + s["bias"]
    return y.to(s["x"].dtype), mean[:, 0], rstd[:, 0]


def _norm_grad(s):
    dy, rstd = s["dy"].float(), s["rstd"][:, None]
    xhat = (s["x"].float() - s["mean"][:, None]) * rstd
    g = dy * s["weight"]
    dx = rstd * (g - g.mean(1, keepdim=True) - xhat * (g * xhat).mean(1, keepdim=True))
    return dx.to(s["x"].dtype), (dy * xhat).sum(0), dy.sum(0) if s["bias"] is not None else None


def _distill(s, grad):
    t, vocab = s["case"]["temperature"], s["case"]["vocab"]
    z = s["logits"].float()
    top = z.amax(1, keepdim=True)
    e = torch.exp((z - top) / t)
    total = e.sum(1, keepdim=True)
    live = (s["ids"] >= 0) & (s["ids"] < vocab)
    at = torch.where(live, s["ids"], 0)
    a = torch.where(live, s["teacher"].float(), -math.inf)
    some = live.any(1, keepdim=True)
    a = (a - torch.where(some, a.amax(1, keepdim=True), 0.0)) / t
    norm = torch.exp(a).sum(1, keepdim=True)
    p = torch.where(some, torch.exp(a) / norm, 0.0)
    log_ratio = a - torch.log(norm) - (z.gather(1, at) - top) / t + torch.log(total)
    loss = t * t * torch.where(p > 0, p * log_ratio, 0.0).sum(1)
    if not grad:
        return loss, torch.cat([top, total], 1)
    e = e / total * some
    e.scatter_add_(1, at, -p)
    return loss, (e * (t * s["weight"])[:, None]).to(s["logits"].dtype)


def run(state):
    s, case = state, state["case"]
    op = case["op"]
    if own:
        import adamw_optimizer_step_muon_amd as ma

        if op == "lookup":
            return ma.embedding_forward(s["table"], s["tokens"], scale=s["scale"], out_dtype=TYPES[case["type"]])
        if op == "table_grad":
            if case["add"]:
                return ma.embedding_backward(s["dout"], s["tokens"], case["rows"], scale=s["scale"], grad=s["grad"], accumulate=True)
            return ma.embedding_backward(s["dout"], s["tokens"], case["rows"], scale=s["scale"])
        if op == "table_step":
            ma.adamw_step_embedding(s["param"], s["tokens"], s["dout"], s["exp_avg"], s["exp_avg_sq"], scale=s["scale"], step=STEP, **ADAMW)
            return s["param"], s["exp_avg"], s["exp_avg_sq"]
        if op == "norm":
            return ma.layer_norm_forward(s["x"], s["weight"], s["bias"], eps=LN_EPS)
        if op == "norm_grad":
            return ma.layer_norm_backward(s["dy"], s["x"], s["mean"], s["rstd"], s["weight"], bias_grad=s["bias"] is not None)
        if op == "distill_step":
            return ma.distill_loss_grad(s["logits"], s["teacher"], s["ids"], s["weight"], temperature=case["temperature"])
        loss, stats = ma.distill_forward(s["logits"], s["teacher"], s["ids"], temperature=case["temperature"])
        if op == "distill_loss":
            return loss, stats
        return loss, ma.distill_backward(s["logits"], s["teacher"], s["ids"], stats, s["weight"], temperature=case["temperature"])
    if op == "lookup":
        rows = case["rows"]
        live = (s["tokens"] >= 0) & (s["tokens"] < rows)
        out = s["table"][torch.where(live, s["tokens"], 0)] * s["scale"]
        return torch.where(live[:, None], out, 0.0).to(TYPES[case["type"]])
    if op == "table_grad":
        g = _table_grad(s, case["rows"])
        return s["grad"].add_(g) if case["add"] else g
    if op == "table_step":
        return _table_step(s)
    if op == "norm":
        return _norm(s)
    if op == "norm_grad":
        return _norm_grad(s)
    return _distill(s, grad=op != "distill_loss")


# ---------------------------------------------------------------- 64 bits, from the definitions
def exact(case, seed):
    s = prepare(case, seed)
    op, f64 = case["op"], torch.float64
    if op in ("lookup", "table_grad", "table_step"):
        rows, dim = case["rows"], case["dim"]
        keep = torch.nonzero((s["tokens"] > -1) & (s["tokens"] < rows))[:, 0]
        ids = s["tokens"].index_select(0, keep)
        if op == "lookup":
            out = torch.zeros(case["tokens"], dim, dtype=f64, device="cuda")
            out.index_copy_(0, keep, s["table"].index_select(0, ids).to(f64).mul_(s["scale"]))
            return out
        grad = torch.zeros(rows, dim, dtype=f64, device="cuda")
        grad.index_put_((ids,), s["dout"].index_select(0, keep).to(f64), accumulate=True)
        grad.mul_(s["scale"])
        if op == "table_grad":
            return grad.add_(s["grad"].to(f64)) if case["add"] else grad
        b1, b2 = ADAMW["beta1"], ADAMW["beta2"]
        m = torch.lerp(grad, s["exp_avg"].to(f64), b1)
        v = torch.lerp(grad.square(), s["exp_avg_sq"].to(f64), b2)
        root = (v / (1.0 - b2 ** STEP)).sqrt_().add_(ADAMW["eps"])
        p = s["param"].to(f64)
        return p - ADAMW["lr"] * (ADAMW["weight_decay"] * p + m / (1.0 - b1 ** STEP) / root), m, v
    if op in ("norm", "norm_grad"):
        x = s["x"].to(f64)
        if op == "norm":
            var, mean = torch.var_mean(x, 1, correction=0)
            rstd = (var + LN_EPS).rsqrt()
            y = torch.einsum("nd,n,d->nd", x - mean[:, None], rstd, s["weight"].to(f64))
            return y if s["bias"] is None else y + s["bias"].to(f64), mean, rstd
        # the definition's gradient for the saved mean and 1 / deviation
        dy, rstd = s["dy"].to(f64), s["rstd"].to(f64).unsqueeze(1)
        h = x.sub_(s["mean"].to(f64).unsqueeze(1)).mul_(rstd)
        u = dy * s["weight"].to(f64)
        a, b = u.sum(1, keepdim=True) / case["dim"], (u * h).sum(1, keepdim=True) / case["dim"]
        return (u - a - h * b) * rstd, (dy * h).sum(0), dy.sum(0) if s["bias"] is not None else None
    t, n, vocab = case["temperature"], case["n"], case["vocab"]
    z = s["logits"].to(f64)
    log_q = torch.log_softmax(z / t, 1)
    live = (s["ids"] > -1) & (s["ids"] < vocab)
    a = s["teacher"].to(f64) / t
    p = torch.softmax(a.masked_fill(~live, -1e300), 1) * live
    # the teacher's probabilities spread over the vocabulary
    wide = torch.zeros(n, vocab, dtype=f64, device="cuda")
    wide.scatter_add_(1, s["ids"].clamp(0, vocab - 1), p)
    at = s["ids"].clamp(0, vocab - 1)
    loss = t * t * (torch.special.xlogy(p, p) - p * torch.gather(log_q, 1, at)).sum(1)
    if op == "distill_loss":
        high = z.max(1, keepdim=True).values
        return loss, torch.cat([high, torch.exp(torch.logsumexp(z / t, 1, keepdim=True) - high / t)], 1)
    del z
    return loss, (log_q.exp_().mul_(p.sum(1, keepdim=True)) - wide).mul_((t * s["weight"].to(f64))[:, None])
