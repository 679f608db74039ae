"""fp64 oracle of the fine-tuning operators: balance loss, router gradient, low-rank adapters and
their gradients, combine gradient.  Written from the definitions, one token, sequence or adapter at a time."""
from __future__ import annotations

import numpy as np

from .moe_oracle import as_f64

__all__ = ["softmax_rows", "balance_loss", "router_backward", "adapter_plan", "lora", "lora_backward",
           "combine_backward"]


def softmax_rows(logits) -> np.ndarray:
    """Softmax of each row; -inf has probability 0, a row of nothing else is 0."""
    l = as_f64(logits)
    m = np.max(l, axis=1, keepdims=True)
    e = np.exp(l - np.where(np.isneginf(m), 0.0, m))
    z = e.sum(1, keepdims=True)
    return np.divide(e, z, out=np.zeros_like(e), where=z != 0)


def _sequences(T, offsets, mask):
    """The tokens that count, sequence by sequence."""
    offsets = [0, T] if offsets is None else [int(v) for v in offsets]
    keep = np.ones(T, bool) if mask is None else np.asarray(mask) != 0
    return [[t for t in range(a, b) if keep[t]] for a, b in zip(offsets, offsets[1:])]


def balance_loss(logits, topk_idx, alpha, offsets=None, mask=None):
    """(loss, counts [S, E], prob [S, E], coef [S])."""
    l, idx = as_f64(logits), np.asarray(topk_idx)
    (T, E), k = l.shape, idx.shape[1]
    seqs = _sequences(T, offsets, mask)
    live = sum(1 for s in seqs if s)
    counts, prob = np.zeros((len(seqs), E), np.int64), np.zeros((len(seqs), E))
    coef, loss = np.zeros(len(seqs)), 0.0
    for s, tokens in enumerate(seqs):
        if not tokens:
            continue
        prob[s] = softmax_rows(l[tokens]).mean(0)
        for e in idx[tokens].ravel():
            if 0 <= e < E:
                counts[s, e] += 1
        n = len(tokens)
        coef[s] = alpha * E / (k * n * n * live)
        loss += alpha * E / live * float(np.sum(counts[s] / (k * n) * prob[s]))
    return loss, counts, prob, coef


def router_backward(logits, topk_idx, d_topk_w=None, renormalize=False, balance=None):
    """d_logits [T, E]; balance: None or (counts, coef, d_loss, offsets, mask)."""
    l, idx = as_f64(logits), np.asarray(topk_idx)
    T, E = l.shape
    d_p = np.zeros((T, E))
    with np.errstate(invalid="ignore"):
        p = softmax_rows(l)
    reached = np.zeros(T, bool)
    if d_topk_w is not None:
        g = as_f64(d_topk_w)
        for t in range(T):
            slots = [j for j in range(idx.shape[1]) if 0 <= idx[t, j] < E]
            if not np.any(g[t] != 0):
                continue
            reached[t] = True
            z = sum(p[t, idx[t, j]] for j in slots) if renormalize else 1.0
            z = z or 1.0
            mean = sum(g[t, j] * p[t, idx[t, j]] for j in slots) / z if renormalize else 0.0
            for j in slots:
                d_p[t, idx[t, j]] += (g[t, j] - mean) / z
    if balance is not None:
        counts, coef, d_loss, offsets, mask = balance
        for s, tokens in enumerate(_sequences(T, offsets, mask)):
            for t in tokens:
                reached[t] = True
                d_p[t] += coef[s] * d_loss * np.asarray(counts[s], np.float64)
    out = np.zeros((T, E))
    r = reached
    out[r] = p[r] * (d_p[r] - np.sum(p[r] * d_p[r], axis=1, keepdims=True))
    return out


def adapter_plan(row_adapter, n):
    row = np.asarray(row_adapter)
    order = [r for a in range(n) for r in np.nonzero(row == a)[0]]
    counts = [int(np.sum(row == a)) for a in range(n)]
    order += [r for r in range(len(row)) if not 0 <= row[r] < n]
    return np.concatenate([[0], np.cumsum(counts)]).astype(np.int64), np.array(order, np.int64)


def lora(x, A, B, row_adapter, scale=None, base=None):
    """(out [rows, N], h [rows, R])."""
    x, A, B, row = as_f64(x), as_f64(A), as_f64(B), np.asarray(row_adapter)
    out = np.zeros((len(x), B.shape[1])) if base is None else as_f64(base).copy()
    h = np.zeros((len(x), A.shape[1]))
    for a in range(len(A)):
        r = np.nonzero(row == a)[0]
        s = 1.0 if scale is None else float(as_f64(scale)[a])
        h[r] = x[r] @ A[a].T
        out[r] += s * (h[r] @ B[a].T)
    return out, h


def lora_backward(dC, x, h, A, B, row_adapter, scale=None, dx_base=None):
    """(dx, dA, dB)."""
    dC, x, h, A, B = (as_f64(v) for v in (dC, x, h, A, B))
    row = np.asarray(row_adapter)
    dx = np.zeros_like(x) if dx_base is None else as_f64(dx_base).copy()
    dA, dB = np.zeros_like(A), np.zeros_like(B)
    for a in range(len(A)):
        r = np.nonzero(row == a)[0]
        s = 1.0 if scale is None else float(as_f64(scale)[a])
        dh = s * (dC[r] @ B[a])
        dx[r] += dh @ A[a]
        dA[a] = dh.T @ x[r]
        dB[a] = s * (dC[r].T @ h[r])
    return dx, dA, dB


def combine_backward(dout, Y, token_to_row, topk_w, shared_base=None):
    """(dY, d_topk_w); shared_base: the first shared row, None without a shared expert."""
    g, Y, w, t2r = as_f64(dout), as_f64(Y), as_f64(topk_w), np.asarray(token_to_row)
    dY, dw = np.zeros_like(Y), np.zeros_like(w)
    for t in range(len(g)):
        for j in range(w.shape[1]):
            if t2r[t, j] >= 0:
                dY[t2r[t, j]] = w[t, j] * g[t]
                dw[t, j] = Y[t2r[t, j]] @ g[t]
        if shared_base is not None:
            dY[shared_base + t] = g[t]
    return dY, dw
