"""Microscaled values, products with them and attention over a cache, in
float64 on the CPU: definitions only (OCP Microscaling Formats v1.0 for the
formats), used by the tests."""
from __future__ import annotations

import numpy as np

GRID = {
    "fp4": np.array([m / 2 if e == 0 else (1 + m / 2) * 2.0 ** (e - 1) for e in range(4) for m in range(2)]),
    "fp8": np.array([m / 8 * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
                     for e in range(16) for m in range(8)][:127]),
}
TOP = {"fp4": 2, "fp8": 8}


def mx_quantize(X, fmt):
    """(codes, scale bytes) of a 2-D array, padded to 128 columns; fp4 codes two to a byte."""
    X = np.asarray(X, dtype=np.float64)
    n, d = X.shape
    cols = -(-d // 128) * 128
    P = np.zeros((n, cols))
    P[:, :d] = X
    P = P.reshape(n, cols // 32, 32)
    grid = GRID[fmt]
    mid = (grid[1:] + grid[:-1]) / 2
    bad = ~np.isfinite(P).all(-1)
    P = np.where(bad[..., None], 0.0, P)
    a = np.abs(P).max(-1)
    e = np.where(a == 0, -127, np.maximum(-127, np.frexp(a)[1] - 1 - TOP[fmt]))
    y = np.abs(P) * 2.0 ** -e[..., None].astype(np.float64)
    lo, hi = np.searchsorted(mid, y, side="left"), np.searchsorted(mid, y, side="right")
    c = np.where(lo % 2 == 0, lo, hi)                  # they differ on a tie: the even code
    c = np.where(bad[..., None], 0, c + np.signbit(P) * (8 if fmt == "fp4" else 128))
    codes = c.astype(np.uint8).reshape(n, cols)
    scales = np.where(bad, 255, e + 127).astype(np.uint8)
    return (codes[:, 0::2] | codes[:, 1::2] << 4 if fmt == "fp4" else codes), scales


def mx_values(codes, scales, fmt, n_cols=None):
    """float64 values of codes and scale bytes (arrays over the last axis)."""
    c = np.asarray(codes)
    if fmt == "fp4":
        c = np.stack((c & 15, c >> 4), -1).reshape(*c.shape[:-1], -1)
        signed = np.concatenate((GRID["fp4"], -GRID["fp4"]))
    else:
        g = np.concatenate((GRID["fp8"], [np.nan]))
        signed = np.concatenate((g, -g))
    s = np.where(np.asarray(scales) == 255, np.nan, 2.0 ** (np.asarray(scales, dtype=np.float64) - 127))
    v = signed[c] * np.repeat(s, 32, axis=-1)
    return v if n_cols is None else v[..., :n_cols]


def attention(Q, K, V, kv_len, scale, window=0):
    """One sequence: Q tokens x heads x d, K and V positions x kv heads x d
    (at least kv_len positions).  Returns the output, sum_j p_j |v_j| and the
    largest sum_c |q_c k_c| of every (token, head), for error bounds."""
    n, heads, d = Q.shape
    g = heads // K.shape[1]
    out, mag, dot = np.zeros(Q.shape), np.zeros(Q.shape), np.zeros((n, heads, 1))
    pos = kv_len - n + np.arange(n)[:, None] - np.arange(kv_len)       # how far ahead of the key a token is
    see = (pos >= 0) & (pos < window if window else True)
    some = see.any(1)
    for h in range(heads):
        k, v, q = K[:kv_len, h // g], V[:kv_len, h // g], Q[:, h]
        if not some.any():
            continue
        s = np.where(see, scale * (q @ k.T), -np.inf)
        w = np.exp(s - np.where(some, s.max(1), 0.0)[:, None])
        w /= np.where(some, w.sum(1), 1.0)[:, None]
        out[:, h], mag[:, h] = w @ v, w @ np.abs(v)
        dot[:, h, 0] = np.where(see, np.abs(q) @ np.abs(k).T, 0.0).max(1)
    return out, mag, dot
