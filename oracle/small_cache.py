"""Oracle of the smaller KV cache in plain fp64 numpy: the four-bit form, attention over it, the
accumulated attention weights, and eviction by them.  Shares no code with the library.

The four-bit form of 16 channels: a scale (five exponent bits of bias 15, three mantissa bits) and
per channel a sign and one of 0, .5, 1, 1.5, 2, 3, 4, 6.  The scale is the smallest that is at least
max|x|/6, at most 10240; a value is the nearest code times the scale, ties to the even code."""
from __future__ import annotations

import numpy as np

CODES = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
SCALES = np.array([(m / 8) * 2.0 ** -14 if e == 0 else (1 + m / 8) * 2.0 ** (e - 15)
                   for e in range(32) for m in range(8)])
N_SCALES = 227                  # 0 .. 10240 are given out
STRIP = 32
STRIP_BYTES = 4608


def quantise(x: np.ndarray):
    """fp64 [..., 128] -> (codes uint8 [..., 128] with the sign in bit 3, scale bytes uint8 [..., 8])."""
    g = x.reshape(*x.shape[:-1], 8, 16)
    bad = ~np.isfinite(g).all(-1)
    a = np.where(bad[..., None], 0.0, np.abs(g))
    byte = np.minimum(np.searchsorted(6 * SCALES[:N_SCALES], a.max(-1), side="left"), N_SCALES - 1)
    s = SCALES[byte][..., None]
    a = np.minimum(a, 6 * s)    # past the largest scale: held as its largest value
    best = np.zeros(g.shape, dtype=np.uint8)
    dist = np.full(g.shape, np.inf)
    for parity in (0, 1):       # even codes first: a tie keeps the even one
        for c in range(parity, 8, 2):
            d = np.abs(a - CODES[c] * s)
            near = d < dist
            best, dist = np.where(near, np.uint8(c), best), np.where(near, d, dist)
    best = np.where(s > 0, best, 0).astype(np.uint8)
    sign = np.where(best > 0, np.signbit(g), False).astype(np.uint8)
    return (best | (sign << 3)).reshape(x.shape), np.where(bad, 255, byte).astype(np.uint8)


def values(codes: np.ndarray, scales: np.ndarray) -> np.ndarray:
    """fp64 values of codes [..., 128] and scale bytes [..., 8]."""
    full = SCALES.copy()
    full[248] = np.inf
    full[249:] = np.nan
    with np.errstate(invalid="ignore"):
        v = CODES[codes & 7] * np.repeat(full[scales], 16, -1)
    return np.where(codes & 8, -v, v)


def held(x: np.ndarray) -> np.ndarray:
    """What the four-bit form makes of fp64 rows [..., 128]."""
    return values(*quantise(x))


def pack_tile(k: np.ndarray, v: np.ndarray) -> np.ndarray:
    """Keys and values [b][128] of one (page, head) -> its strips uint8 [b/32][4608]."""
    b = k.shape[0]
    out = np.zeros((b // STRIP, STRIP_BYTES), dtype=np.uint8)
    for i, x in enumerate((k, v)):
        codes, scales = quantise(x)
        by = (codes[:, 0::2] | (codes[:, 1::2] << 4)).reshape(b // STRIP, -1)
        out[:, 2048 * i:2048 * (i + 1)] = by
        out[:, 4096 + 256 * i:4096 + 256 * (i + 1)] = scales.reshape(b // STRIP, -1)
    return out


def unpack_tile(strips: np.ndarray):
    """Strips uint8 [..., b/32][4608] -> keys, values fp64 [..., b][128]."""
    lead = strips.shape[:-2]
    got = []
    for i in range(2):
        by = strips[..., 2048 * i:2048 * (i + 1)].reshape(*lead, -1, 64)
        sc = strips[..., 4096 + 256 * i:4096 + 256 * (i + 1)].reshape(*lead, -1, 8)
        codes = np.stack((by & 15, by >> 4), -1).reshape(*lead, by.shape[-2], 128)
        got.append(values(codes, sc))
    return got


def gather(pages: np.ndarray, table, s: int, max_blocks: int, h: int, length: int) -> np.ndarray:
    """Rows [length][...] of sequence s, head h from per-page rows [pages][H][b][...]."""
    b = pages.shape[2]
    n = -(-length // b)
    idx = table[s, :n] if table is not None else s * max_blocks + np.arange(n)
    return pages[idx, h].reshape(n * b, *pages.shape[3:])[:length]


def tokens_of(length: int, b: int, blocks) -> np.ndarray:
    """Positions of the valid tokens of the listed blocks, in order (all blocks if None)."""
    if blocks is None:
        return np.arange(length)
    t = (np.asarray(blocks, dtype=np.int64)[:, None] * b + np.arange(b)).ravel()
    return t[t < length]


def logits(q: np.ndarray, k: np.ndarray, tok: np.ndarray, length: int, scale: float, bias=None) -> np.ndarray:
    """q [M][G][128], keys [length][128] -> [M][G][len(tok)], -inf where token i does not see."""
    M = q.shape[0]
    x = np.einsum("mgd,td->mgt", q, k[tok]) * scale
    if bias is not None:
        x = x + bias
    hidden = tok[None, :] > (length - M + np.arange(M))[:, None]
    return np.where(hidden[:, None, :], -np.inf, x)


def attend(x: np.ndarray, v: np.ndarray):
    """Softmax of the logits [M][G][T] times values [T][128], and the log-sum-exp (0 and -inf for empty rows)."""
    if x.shape[-1] == 0:
        return np.zeros((*x.shape[:2], 128)), np.full(x.shape[:2], -np.inf)
    m = x.max(-1, keepdims=True)
    with np.errstate(invalid="ignore"):
        p = np.where(x == -np.inf, 0.0, np.exp(x - np.where(m == -np.inf, 0.0, m)))
        z = p.sum(-1, keepdims=True)
        # a masked token takes no part, whatever its value is
        o = np.stack([[(p[i, g] / z[i, g])[p[i, g] != 0] @ v[p[i, g] != 0] if z[i, g] != 0 else np.zeros(128)
                       for g in range(x.shape[1])] for i in range(x.shape[0])])
        lse = np.where(z[..., 0] == 0, -np.inf, m[..., 0] + np.log(np.where(z[..., 0] == 0, 1, z[..., 0])))
    return o, lse


def weights(x: np.ndarray, lse: np.ndarray) -> np.ndarray:
    """Sum over the rows of exp(logit - lse): [T]."""
    with np.errstate(invalid="ignore"):
        return np.where(lse[..., None] == -np.inf, 0.0, np.exp(x - lse[..., None])).sum((0, 1))


def keep(acc: np.ndarray, n_keep: int, n_sink: int, n_recent: int) -> np.ndarray:
    """Kept positions (ascending) of a sequence with weights acc [length]."""
    n = len(acc)
    if n <= n_keep:
        return np.arange(n)
    def rank(t):
        if t < n_sink or t >= n - n_recent:
            return (0, 0.0, t)
        return (2, 0.0, t) if np.isnan(acc[t]) else (1, -float(acc[t]), t)
    return np.array(sorted(sorted(range(n), key=rank)[:n_keep]), dtype=np.int64)
