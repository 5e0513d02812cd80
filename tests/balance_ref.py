"""The balance loss over sequences, its counts, the z term and the gradient,
from their definitions in fp64 (numpy), and the sizes the error bounds need."""
import numpy as np


def _tokens_of(T, seqs, mask):
    seqs = np.asarray([0, T] if seqs is None else seqs, np.int64)
    take = np.ones(T, bool) if mask is None else np.asarray(mask) != 0
    return [np.arange(a, b)[take[a:b]] for a, b in zip(seqs[:-1], seqs[1:])]


def softmax(h):
    """Rows without a finite logit have p = 0 and lse = 0."""
    h = np.asarray(h, np.float64)
    m = h.max(axis=1, keepdims=True)
    m = np.where(np.isneginf(m), 0.0, m)
    e = np.exp(h - m)
    s = e.sum(axis=1, keepdims=True)
    with np.errstate(divide="ignore", invalid="ignore"):
        return np.where(s == 0, 0.0, e / s), np.where(s == 0, 0.0, m + np.log(s))[:, 0]


def loss(h, idx, mask, seqs, alpha, z_coef):
    """(loss [2], counts [S, N], P [S, N], tokens [S + 2])"""
    T, N = h.shape
    p, lse = softmax(h)
    rows = _tokens_of(T, seqs, mask)
    n = [len(r) for r in rows]
    used, total = sum(v > 0 for v in n), sum(n)
    counts = np.zeros((len(rows), N), np.int64)
    P = np.zeros((len(rows), N))
    aux = z = 0.0
    for s, r in enumerate(rows):
        if n[s] == 0:
            continue
        e = np.asarray(idx)[r].ravel()
        counts[s] = np.bincount(e[(e >= 0) & (e < N)], minlength=N)
        P[s] = p[r].sum(axis=0) / n[s]
        aux += alpha * N / used * (counts[s] / (idx.shape[1] * n[s]) * P[s]).sum()
        z += z_coef / total * (lse[r] ** 2).sum()
    return np.array([aux, z]), counts, P, np.array(n + [total, used])


def gradient(h, k, mask, seqs, alpha, z_coef, counts, g=(1.0, 1.0)):
    """dL/dh [T, N], the same with every term's magnitude, and which rows are written."""
    T, N = h.shape
    p, lse = softmax(h)
    rows = _tokens_of(T, seqs, mask)
    used, total = sum(len(r) > 0 for r in rows), sum(len(r) for r in rows)
    d, size, written = np.zeros((T, N)), np.zeros((T, N)), np.zeros(T, bool)
    cuts = np.asarray([0, T] if seqs is None else seqs, np.int64)
    written[cuts[0]:cuts[-1]] = True
    for s, r in enumerate(rows):
        if len(r) == 0:
            continue
        a = g[0] * alpha * N / (used * len(r)) * counts[s] / (k * len(r))
        zg = g[1] * 2 * z_coef * lse[r] / total
        dot = p[r] @ a
        d[r] = p[r] * (a - dot[:, None] + zg[:, None])
        size[r] = p[r] * (np.abs(a) + np.abs(p[r] @ np.abs(a))[:, None] + np.abs(zg)[:, None])
    return d, size, written
