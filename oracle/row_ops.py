"""Plain fp64 definitions of the row operators: layer norm, embedding, MoE router
and MoE row moves, with their gradients.

Test infrastructure only (see oracle/__init__.py).  Each function is the
operator's formula (include/coc.h) in the plainest form; inputs are the storage
dtypes' values as float64, results are not rounded.
"""
from __future__ import annotations

import numpy as np


def layer_norm(h, gamma, beta, eps):
    """(y, mean, rstd) of the rows of h."""
    h = np.asarray(h, dtype=np.float64)
    mean = h.mean(axis=1)
    rstd = 1.0 / np.sqrt(((h - mean[:, None]) ** 2).mean(axis=1) + eps)
    y = (h - mean[:, None]) * rstd[:, None] * gamma
    return (y if beta is None else y + beta), mean, rstd


def layer_norm_backward(dy, h, gamma, mean, rstd, dsum=None):
    """(dx, dgamma, dbeta) with the forward's statistics."""
    xh = (h - mean[:, None]) * rstd[:, None]
    g = dy * gamma
    n = h.shape[1]
    dx = rstd[:, None] * (g - g.sum(1, keepdims=True) / n - xh * (g * xh).sum(1, keepdims=True) / n)
    if dsum is not None:
        dx = dx + dsum
    return dx, (dy * xh).sum(0), dy.sum(0)


def embedding(ids, table, start, scale):
    y = np.zeros((len(ids), table.shape[1]))
    for t, i in enumerate(ids):
        if start <= int(i) < start + len(table):
            y[t] = scale * table[int(i) - start]
    return y


def embedding_grad(ids, dy, vocab, start, scale):
    g = np.zeros((vocab, dy.shape[1]))
    for t, i in enumerate(ids):
        if start <= int(i) < start + vocab:
            g[int(i) - start] += dy[t]
    return scale * g


def piece_of(t, tokens, pieces):
    """The sequence piece of token t: the q with tokens*q//pieces <= t < tokens*(q+1)//pieces."""
    for q in range(pieces):
        if tokens * q // pieces <= t < tokens * (q + 1) // pieces:
            return q
    raise ValueError(t)


def softmax_rows(logits, mask=None):
    """(p, takes part) by row; rows that take no part have p = 0."""
    x = np.asarray(logits, dtype=np.float64)
    p = np.zeros_like(x)
    live = np.zeros(len(x), dtype=bool)
    for t, row in enumerate(x):
        if (mask is not None and not mask[t]) or np.all(row == -np.inf):
            continue
        live[t] = True
        with np.errstate(invalid="ignore"):
            e = np.exp(row - np.max(row))
            p[t] = e / e.sum()
    return p, live


def moe_router(logits, topk, pieces, world, coef, renormalize, mask=None):
    """dict of ids, gates, positions, counts, prob_sums, loss, valid."""
    x = np.asarray(logits, dtype=np.float64)
    tokens, experts = x.shape
    p, live = softmax_rows(x, mask)
    ids = np.full((tokens, topk), -1, dtype=np.int64)
    gates = np.zeros((tokens, topk))
    counts = np.zeros((pieces, experts), dtype=np.int64)
    for t in range(tokens):
        if not live[t]:
            continue
        order = sorted(range(experts), key=lambda e: (-np.inf if np.isnan(x[t, e]) else -x[t, e], e))
        # a NaN is the largest of all, above +inf
        order = [e for e in order if np.isnan(x[t, e])] + [e for e in order if not np.isnan(x[t, e])]
        for j, e in enumerate(order[:topk]):
            if x[t, e] == -np.inf:
                break
            ids[t, j] = e
            gates[t, j] = p[t, e]
            counts[piece_of(t, tokens, pieces), e] += 1
        if renormalize:
            gates[t] /= gates[t].sum()
    local = experts // world
    rows = sorted((ids[t, j] // local, piece_of(t, tokens, pieces), ids[t, j], t, j)
                  for t in range(tokens) for j in range(topk) if ids[t, j] >= 0)
    positions = np.full((tokens, topk), -1, dtype=np.int64)
    for at, (_, _, _, t, j) in enumerate(rows):
        positions[t, j] = at
    n = int(live.sum())
    sums = p.sum(0)
    loss = coef * experts / (topk * n * n) * float((counts.sum(0) * sums).sum()) if n else 0.0
    return {"ids": ids, "gates": gates, "positions": positions, "counts": counts, "prob_sums": sums, "loss": loss,
            "valid": n}


def moe_router_backward(logits, ids, counts, dgates, dloss, coef, renormalize, mask=None):
    """dlogits, by the chain rule through each token's gates and probabilities."""
    p, live = softmax_rows(logits, mask)
    tokens, experts = p.shape
    topk, n = ids.shape[1], max(1, int(live.sum()))
    out = np.zeros_like(p)
    for t in range(tokens):
        if not live[t]:
            continue
        dp = dloss * coef * experts / (topk * n * n) * counts.sum(0).astype(np.float64)
        sel = [(int(e), float(dgates[t, j])) for j, e in enumerate(ids[t]) if e >= 0]
        s = sum(p[t, e] for e, _ in sel)
        for e, d in sel:
            dp[e] += (d - sum(p[t, f] / s * v for f, v in sel)) / s if renormalize else d
        out[t] = p[t] * (dp - (p[t] * dp).sum())
    return out


def moe_combine(h, positions, gates=None):
    y = np.zeros((len(positions), h.shape[1]))
    for t, row in enumerate(positions):
        for j, r in enumerate(row):
            if 0 <= r < len(h):
                y[t] += (1.0 if gates is None else gates[t, j]) * h[r]
    return y


def moe_combine_backward(dy, h, positions, gates):
    """(dh, dgates); rows of dh that no position names are 0 here."""
    dh, dg = np.zeros_like(h), np.zeros(positions.shape)
    for t, row in enumerate(positions):
        for j, r in enumerate(row):
            if 0 <= r < len(h):
                dh[r] = gates[t, j] * dy[t]
                dg[t, j] = (dy[t] * h[r]).sum()
    return dh, dg
