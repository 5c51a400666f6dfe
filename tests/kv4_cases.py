"""Inputs on which one fp16 term of an attention weight is not enough (host side, no GPU).

Pairs of tokens with scores of exactly 0 (keys of code 0 and zero point 0) have the values
7 d s and -6 d s', s' = 7/6 s but for its rounding to 20 bits, so that the output is
next to nothing while the weights p s, numbers of 20 bits, are not.  With n keys of equal
probability 1/n,

  |err| <= eps/2 |o| + 2^-20 sum_j |V_j| / n + 2^-23 (16 + n/16) 30 sum_j s_j / n

the output's rounding; two fp16 terms of each weight (2^-22) and 2^-22 each for the
exponential and the sum of probabilities; fp32 sums of codes and of zero points (at most 15
times the weights each): one rounding for the products of 16 keys, one to subtract the zero
points, three to join warps, at most four to join splits, two to divide, counted as 16.
"""

import numpy as np

F32 = np.float32


def round20(s):
    return ((np.asarray(s, F32).view(np.uint32) + np.uint32(8)) & np.uint32(0xFFFFFFF0)).view(F32)


def pairs(r, n, D):
    """(scales (n), zero points (n), codes (n, D)) of n values, n even, that cancel in pairs:
    7 d s and -6 d s' with s' = 7/6 s, d = +-1 for each dim."""
    s = np.zeros(n, F32)
    s[0::2] = round20(r.uniform(0.5, 1, n // 2))
    s[1::2] = round20(s[0::2] * F32(7) / F32(6))
    d = np.where(r.random((n // 2, D)) < 0.5, 1, -1)
    c = np.zeros((n, D), np.uint8)
    c[0::2], c[1::2] = 8 + 7 * d, 8 - 6 * d
    return s, np.full(n, 8, np.uint8), c


def exact(s, z, c):
    v = s.astype(np.float64)[:, None] * (c.astype(np.float64) - z.astype(np.float64)[:, None])
    return v.mean(0), v


def bound(o, v, s, eps):
    n = len(s)
    return (eps / 2 * np.abs(o) + 2.0 ** -20 * np.abs(v).mean(0)
            + 2.0 ** -23 * (16 + n / 16) * 30 * s.astype(np.float64).mean())


def with_one_term(s, z, c):
    """What one fp16 term of each weight gives (a mistake to be caught)."""
    w = (s * F32(2.0 ** 9)).astype(np.float16).astype(np.float64) * 2.0 ** -9
    return (w[:, None] * (c.astype(np.float64) - z.astype(np.float64)[:, None])).mean(0)


def key_far_below():
    """(code, scale, zero point) of keys of value -90."""
    return 0, round20(F32(6.0)), 15
