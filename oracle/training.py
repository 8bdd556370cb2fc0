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


def head_loss(hidden, weight, labels):
    """(loss, lse) of each row's label under the logits hidden weight^T; 0 without a target."""
    hidden, weight, labels = _f64(hidden), _f64(weight), np.asarray(labels)
    loss, lse = np.zeros(labels.size), np.zeros(labels.size)
    for r, label in enumerate(labels.reshape(-1)):
        if 0 <= label < weight.shape[0]:
            z = weight @ hidden[r]
            lse[r] = z.max() + np.log(np.sum(np.exp(z - z.max())))
            loss[r] = lse[r] - z[label]
    return loss, lse


def head_loss_grad(hidden, weight, labels, row_weight):
    """The gradients of sum row_weight * loss by the hidden states and the weight."""
    hidden, weight, labels = _f64(hidden), _f64(weight), np.asarray(labels).reshape(-1)
    dh, dw = np.zeros_like(hidden), np.zeros_like(weight)
    for r, label in enumerate(labels):
        if 0 <= label < weight.shape[0]:
            z = weight @ hidden[r]
            g = np.exp(z - z.max())
            g /= g.sum()
            g[label] -= 1.0
            g *= row_weight[r]
            dh[r] = g @ weight
            dw += np.outer(g, hidden[r])
    return dh, dw


def _norm(x, center, eps):
    mean = x.mean(1) if center else np.zeros(len(x))
    rstd = 1.0 / np.sqrt(((x - mean[:, None]) ** 2).mean(1) + eps)
    return (x - mean[:, None]) * rstd[:, None], mean, rstd


def residual_norm(x, residual, weight=None, bias=None, post_norm=True, post_weight=None, post_bias=None, gate=None,
                  scale=1.0, center=True, eps=1e-5):
    """(out, y, stats) of the norms around a block."""
    x, residual = _f64(x), _f64(residual)
    zero = np.zeros(len(x))
    b, mean1, rstd1 = _norm(x, center, eps) if post_norm else (x, zero, zero)
    b = b * (1.0 if post_weight is None else _f64(post_weight)) + (0.0 if post_bias is None else _f64(post_bias))
    out = residual + scale * (1.0 if gate is None else _f64(gate)) * b
    h, mean2, rstd2 = _norm(out, center, eps)
    y = h * (1.0 if weight is None else _f64(weight)) + (0.0 if bias is None else _f64(bias))
    return out, y, np.stack([mean1, rstd1, mean2, rstd2])


def residual_norm_grad(dout, dy, x, out, stats, weight=None, post_norm=True, post_weight=None, post_bias=None, gate=None,
                       scale=1.0, center=True):
    """(dx, dresidual, dweight, dbias, dpost_weight, dpost_bias, dgate) for given statistics."""
    dout, dy, x, out = (_f64(t) for t in (dout, dy, x, out))
    mean1, rstd1, mean2, rstd2 = (_f64(t)[:, None] for t in stats)
    one = np.ones(x.shape[1])
    weight, post_weight, gate = (one if t is None else _f64(t) for t in (weight, post_weight, gate))
    post_bias = np.zeros_like(one) if post_bias is None else _f64(post_bias)

    def back(u, h, rstd):
        mean = u.mean(1, keepdims=True) if center else 0.0
        return rstd * (u - mean - h * (u * h).mean(1, keepdims=True))

    h2 = (out - mean2) * rstd2
    d = dout + back(dy * weight, h2, rstd2)
    h1 = (x - mean1) * rstd1 if post_norm else x
    b, db = h1 * post_weight + post_bias, d * scale * gate
    dx = back(db * post_weight, h1, rstd1) if post_norm else db
    return dx, d, (dy * h2).sum(0), dy.sum(0), (db * h1).sum(0), db.sum(0), (d * scale * b).sum(0)
