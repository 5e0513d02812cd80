"""How far the 4-bit expert kernels may be off, as a relative RMS of each row of y, and numpy
models of their roundings that show what such a bar lets through.

A row's error is y's own rounding to bf16, which the exact result gives, and beside it what H
(and x) lose.  y_o = sum_i w_oi h_i adds up independent errors, so a relative error of every h_i
with RMS r is one of y with RMS r (weights of random sign).  Rounding to b significant bits has a
half step of 2^-b, an RMS below 2^-b / sqrt 3.
  many rows: x exact, H fp16 (11 bits): 2^-11 covers it and fp32's sums.
  few rows: x and H are integers in blocks, off by at most 2^-16 of a block's largest value and
    by 2^-16 / sqrt 3 RMS.  Values of one size within a block (normal x, SwiGLU's products of
    two) have a largest of at most 8 times their RMS here: 2^-13 / sqrt 3 each, 2^-13 for both.
The two parts add in squares; 1.05 for a row's few hundred samples of them."""
import numpy as np

import w4_ref

MANY, FEW = 2.0 ** -11, 2.0 ** -13


def rms(v):
    return np.sqrt((v ** 2).mean(axis=-1))


def allowed(want, lost):
    """The RMS error of each row that `lost` (relative RMS) and the rounding to bf16 explain."""
    return 1.05 * np.sqrt(rms(w4_ref.bf16(want) - want) ** 2 + (lost * rms(want)) ** 2)


def experts(N, d, dff, group, act, seed):
    """Random codes and scales: {name: (q [N, rows, K], scale [N, groups, rows])}"""
    rng = np.random.default_rng(seed)

    def mat(rows, K):
        s = w4_ref.bf16(rng.uniform(0.5, 2.0, (N, (K + group - 1) // group, rows)) * 0.3 / np.sqrt(K) / 4)
        return rng.integers(-7, 8, (N, rows, K)).astype(np.int8), s

    return dict(w1=mat(dff, d), w3=mat(dff, d) if act == "swiglu" else None, w2=mat(d, dff))


def matrices(W, e, group):
    return [None if W[n] is None else w4_ref.values(W[n][0][e].astype(np.float64), W[n][1][e], group) for n in ("w1", "w3", "w2")]


def rows(R, d, seed):
    return w4_ref.bf16(np.random.default_rng(seed).standard_normal((R, d)))


def to_bits(v, bits):
    m, e = np.frexp(v)
    return np.ldexp(np.rint(m * 2.0 ** bits), e - bits)


def to_blocks(v, block, levels=32512):
    """Integers of 16 bits (levels 32512) in blocks with their own unit."""
    pad = np.pad(v, ((0, 0), (0, -v.shape[1] % block))).reshape(v.shape[0], -1, block)
    unit = np.maximum(np.abs(pad).max(axis=2, keepdims=True), 1e-300) / levels
    return (np.rint(pad / unit) * unit).reshape(v.shape[0], -1)[:, : v.shape[1]]


def ffn(x, w1, w3, w2, act, x_round=None, h_round=None):
    """The exact expert, or with x and H rounded; the model's y is bf16 then."""
    xv = x if x_round is None else x_round(x)
    u = xv @ w1.T
    h = u / (1 + np.exp(-u)) * (xv @ w3.T) if act == "swiglu" else np.maximum(u, 0)
    y = (h if h_round is None else h_round(h)) @ w2.T
    return y if h_round is None else w4_ref.bf16(y)
