"""The 4-bit key/value cache on the host (TEST INFRASTRUCTURE ONLY, like the
rest of this package).

Decisions that produce integers (the grid's scale, zero point and codes, and
the rotations in front of them) are taken in fp32, one rounding per operation,
in the order the header gives; attention over the cached values is fp64.

Grid of a vector x: lo = min(0, min x), hi = max(0, max x),
s = max((hi - lo) (1/15), 2^-100) rounded half up to 20 significant bits,
r = 1/s, zero = clamp(rint(-lo r), 0, 15), code = clamp(rint(x r) + zero, 0, 15),
value = s (code - zero); a vector with a NaN or an infinity, or whose width
overflows, has s = NaN.
"""

from __future__ import annotations

import numpy as np

F32 = np.float32


def rotate(x, table_row, rot: int, interleaved: bool, signs):
    """Position rotation, then the signed Hadamard transform, of (H, D) in fp32."""
    x = np.array(x, dtype=F32)
    D = x.shape[-1]
    if rot:
        h = rot // 2
        c, s = table_row[:h].astype(F32), table_row[h:rot].astype(F32)
        ia = np.arange(0, rot, 2) if interleaved else np.arange(h)
        ib = ia + (1 if interleaved else h)
        a, b = x[:, ia].copy(), x[:, ib].copy()
        x[:, ia] = a * c - b * s
        x[:, ib] = b * c + a * s
    if signs is not None:
        x = x * np.asarray(signs, dtype=F32)
        h = 1
        while h < D:
            y = x.reshape(-1, D // (2 * h), 2, h)
            u, w = y[:, :, 0], y[:, :, 1]
            x = np.stack([u + w, u - w], axis=2).reshape(-1, D)
            h *= 2
        x = x * F32(D ** -0.5)
    return x


def quantize(x):
    """(codes uint8, scale fp32, zero uint8) of fp32 vectors along the last axis."""
    with np.errstate(all="ignore"):
        x = np.asarray(x, dtype=F32)
        lo = np.minimum(x.min(-1), F32(0))
        hi = np.maximum(x.max(-1), F32(0))
        span = hi - lo
        s = np.maximum(span * F32(1 / 15), F32(2.0 ** -100)).astype(F32)
        s[~(span < np.inf)] = np.inf
        s = ((s.view(np.uint32) + np.uint32(8)) & np.uint32(0xFFFFFFF0)).view(F32)
        bad = ~(s < np.inf)
        s[bad] = 1
        r = (F32(1) / s).astype(F32)
        z = np.clip(np.rint(-lo * r), 0, 15)
        c = np.clip(np.rint(x * r[..., None]) + z[..., None], 0, 15)
        c[bad] = 0
        z[bad] = 0
        s[bad] = np.nan
        return c.astype(np.uint8), s, z.astype(np.uint8)


def words(s, z):
    w = np.ascontiguousarray(s, dtype=F32).view(np.uint32) | z.astype(np.uint32)
    return np.where(np.isnan(s), np.uint32(0x7FC00000), w).astype(np.uint32)


def values(codes, w, dtype=np.float64):
    """Values of codes (..., D) and words (...)."""
    s = (w & np.uint32(0xFFFFFFF0)).view(F32).astype(dtype)
    return s[..., None] * (codes.astype(dtype) - (w & np.uint32(15)).astype(dtype)[..., None])


def split_block(block, P: int, D: int):
    """A cache's bytes (..., P (D + 8)) as key codes and value codes (..., P, D),
    key words and value words (..., P)."""
    h = P * D // 2
    out = []
    for i in (0, 1):
        b = block[..., i * h:(i + 1) * h].reshape(block.shape[:-1] + (P, D // 2))
        c = np.empty(b.shape[:-1] + (D,), dtype=np.uint8)
        c[..., 0::2], c[..., 1::2] = b & 15, b >> 4
        out.append(c)
    w = np.ascontiguousarray(block[..., 2 * h:]).view(np.uint32)
    return out[0], out[1], w[..., :P], w[..., P:]


def put(block, P: int, D: int, slot: int, codes, w, isv: int):
    """Writes one token into a (page, head) block (bytes, in place)."""
    o = isv * P * D // 2 + slot * D // 2
    block[o:o + D // 2] = codes[0::2] | codes[1::2] << 4
    o = P * D + 4 * (isv * P + slot)
    block[o:o + 4] = np.array([w], dtype=np.uint32).view(np.uint8)


def visible(p: int, L: int, causal: bool, window: int, sinks: int):
    """Mask over keys 0 .. L-1 of a query at index p."""
    j = np.arange(L)
    m = (j <= p) if causal else np.ones(L, dtype=bool)
    if window:
        m &= (j > p - window) | (j < sinks)
    return m


def attend(q, k, v, scale: float, mask):
    """fp64 attention of one query (D) over keys, values (L, D); mask (L).
    Returns (out (D), lse, probabilities (L))."""
    out = np.zeros(v.shape[-1])
    p = np.zeros(len(k))
    if not mask.any():
        return out, -np.inf, p
    x = (k[mask].astype(np.float64) @ np.asarray(q, dtype=np.float64)) * scale
    m = x.max()
    e = np.exp(x - m)
    p[mask] = e / e.sum()
    out = p[mask] @ v[mask].astype(np.float64)
    return out, float(m + np.log(e.sum())), p
