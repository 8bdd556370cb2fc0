"""fp64 reference of the training operators: embedding, layer norm, distillation.

Written from the definitions, with explicit loops over rows where that is the plainer form;
shares no code with the GPU path.
"""
from __future__ import annotations

import numpy as np


def _f64(x):
    return np.asarray(x, dtype=np.float64)


def embedding(table, tokens, scale=1.0):
    """scale * table[t] for each token; a token outside the table gives zeros."""
    table, tokens = _f64(table), np.asarray(tokens)
    out = np.zeros(tokens.shape + (table.shape[1],))
    for at, t in np.ndenumerate(tokens):
        if 0 <= t < table.shape[0]:
            out[at] = scale * table[t]
    return out


def embedding_grad(dout, tokens, rows, scale=1.0):
    """(gradient, sum of the magnitudes of its terms, tokens per row)."""
    dout, tokens = _f64(dout), np.asarray(tokens).reshape(-1)
    dout = dout.reshape(tokens.size, dout.shape[-1])
    grad, size = np.zeros((rows, dout.shape[1])), np.zeros((rows, dout.shape[1]))
    count = np.zeros(rows, dtype=np.int64)
    for t, d in zip(tokens, dout):
        if 0 <= t < rows:
            grad[t] += scale * d
            size[t] += abs(scale) * np.abs(d)
            count[t] += 1
    return grad, size, count


def layer_norm(x, weight=None, bias=None, eps=1e-5):
    """(y, mean, rstd) over the last dimension."""
    x = _f64(x)
    mean = x.mean(-1)
    rstd = 1.0 / np.sqrt(((x - mean[..., None]) ** 2).mean(-1) + eps)
    y = (x - mean[..., None]) * rstd[..., None]
    if weight is not None:
        y = y * _f64(weight)
    if bias is not None:
        y = y + _f64(bias)
    return y, mean, rstd


def layer_norm_grad(dy, x, mean, rstd, weight=None):
    """(dx, dweight, dbias) for 2-D dy and x and the given mean and rstd."""
    dy, x = _f64(dy), _f64(x)
    h = (x - _f64(mean)[:, None]) * _f64(rstd)[:, None]
    u = dy if weight is None else dy * _f64(weight)
    dx = _f64(rstd)[:, None] * (u - u.mean(1)[:, None] - h * (u * h).mean(1)[:, None])
    return dx, (dy * h).sum(0), dy.sum(0)


def teacher_probabilities(teacher, ids, vocab, temperature=1.0):
    """softmax(teacher / temperature) over each row's live entries, 0 elsewhere."""
    teacher, ids = _f64(teacher), np.asarray(ids)
    p = np.zeros(teacher.shape)
    for r in range(teacher.shape[0]):
        live = (ids[r] >= 0) & (ids[r] < vocab) & (teacher[r] > -np.inf)
        if live.any():
            a = teacher[r][live] / temperature
            e = np.exp(a - a.max())
            p[r][live] = e / e.sum()
    return p


def distill(logits, teacher, ids, temperature=1.0):
    """(loss, p, q) of 2-D logits (n, vocab) and teacher (n, top)."""
    z, ids = _f64(logits), np.asarray(ids)
    p = teacher_probabilities(teacher, ids, z.shape[1], temperature)
    x = (z - z.max(1, keepdims=True)) / temperature
    log_q = x - np.log(np.exp(x).sum(1, keepdims=True))
    loss = np.zeros(z.shape[0])
    for r, i in zip(*np.nonzero(p)):
        loss[r] += temperature ** 2 * p[r, i] * (np.log(p[r, i]) - log_q[r, ids[r, i]])
    return loss, p, np.exp(log_q)


def distill_grad(logits, teacher, ids, row_weight, temperature=1.0):
    """Gradient of sum row_weight * loss by the logits."""
    _, p, q = distill(logits, teacher, ids, temperature)
    dz = q * p.sum(1, keepdims=True)
    for r, i in zip(*np.nonzero(p)):
        dz[r, np.asarray(ids)[r, i]] -= p[r, i]
    w = _f64(row_weight)[:, None]
    return np.where(w == 0, 0.0, w * temperature * dz)
