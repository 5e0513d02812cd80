"""4-bit weights with group scales from their definition (numpy, fp64): packing,
quantisation in exact arithmetic, and the expert FFN with its error bound."""
import numpy as np


def bf16(v):
    """fp64 -> the nearest bf16 value (ties to even), as fp64; no double rounding (normal range)."""
    m, e = np.frexp(np.asarray(v, np.float64))
    return np.ldexp(np.rint(m * 256), e - 8)


def quantize(w, group):
    """w [rows, K] fp64 -> (q [rows, K] in -7..7, scale [groups, rows])"""
    rows, K = w.shape
    q, scales = np.zeros((rows, K), np.int8), []
    for a in range(0, K, group):
        part = w[:, a:a + group]
        s = bf16(np.abs(part).max(axis=1) / 7)
        with np.errstate(divide="ignore", invalid="ignore"):
            r = np.where(s[:, None] > 0, part / s[:, None], 0.0)
        q[:, a:a + group] = np.clip(np.rint(r), -7, 7)
        scales.append(s)
    return q, np.stack(scales)


def pack(q):
    """q [..., K] in -8..7 -> packed rows, word by word as the layout says."""
    K = q.shape[-1]
    nb = (K + 127) // 128
    words = np.zeros(q.shape[:-1] + (nb * 16,), np.uint32)
    for k in range(nb * 128):
        b, n = divmod(k, 128)
        j, rest = divmod(n, 32)
        t, i2 = divmod(rest, 8)
        i, odd = divmod(i2, 2)
        c = q[..., k].astype(np.int64) + 8 if k < K else np.int64(8)
        words[..., 16 * b + 4 * t + j] |= (c << (4 * i + 16 * odd)).astype(np.uint32) if k < K else np.uint32(c << (4 * i + 16 * odd))
    return words.view(np.uint8)


def values(q, scale, group):
    K = q.shape[-1]
    return q * np.repeat(np.moveaxis(scale, -2, -1), group, axis=-1)[..., :K]


def block_error(v):
    """Few rows enter the products as 16-bit integers per block of 64 or 128 values: off by at most half a
    unit, max / 32512 / 2 (1.1: the unit's and its reciprocal's own rounding)."""
    pad = np.pad(np.abs(v), ((0, 0), (0, -v.shape[1] % 128)))
    top = pad.reshape(v.shape[0], -1, 128).max(axis=2)
    return np.repeat(top, 128, axis=1)[:, : v.shape[1]] * (1.1 / 65024)


def ffn(x, w1, w3, w2, b1, b3, b2, act, h_step):
    """One expert on rows x (fp64): (y, error bound).  w [out, in] fp64.

    A product of K terms accumulated in fp32 is off by at most (K + 16) 2^-23 of
    the sum of its terms' magnitudes (every addition rounds or truncates by 2^-23
    at most; 16: the group scales and the sums over warps); h_step is H's
    rounding where it is kept in bf16 (2^-8), y's is 2^-8.
    |silu'| <= 1.1, |silu(u)| <= |u|, and its own evaluation 2^-20."""
    def product(x, w, b, dx):
        c = (w.shape[1] + 16) * 2.0 ** -23
        v = x @ w.T + (0 if b is None else b)
        size = np.abs(x) @ np.abs(w).T + (0 if b is None else np.abs(b))
        return v, c * size + dx @ np.abs(w).T

    dx = block_error(x)
    u, du = product(x, w1, b1, dx)
    if act == "swiglu":
        v, dv = product(x, w3, b3, dx)
        silu = u / (1 + np.exp(-u))
        h = silu * v
        dh = 1.1 * du * (np.abs(v) + dv) + np.abs(silu) * dv + 2.0 ** -20 * np.abs(h)
    else:
        h, dh = np.maximum(u, 0), du
    dh = dh + h_step * (np.abs(h) + dh)
    dh = dh + block_error(np.abs(h) + dh)
    y, dy = product(h, w2, b2, dh)
    return y, dy + 2.0 ** -8 * (np.abs(y) + dy)
