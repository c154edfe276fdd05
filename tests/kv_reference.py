"""Rotary positions and attention over a 4-bit cache in 64 bits, stated from their formulas (no code shared with the
library): what the codes of a cache stand for, and what a row of q makes of them."""
import numpy as np

E2M1 = np.array([0, .5, 1, 1.5, 2, 3, 4, 6, -0., -.5, -1, -1.5, -2, -3, -4, -6])


def e4m3(b):
    b = b.astype(np.int64)
    e, m = (b >> 3) & 15, b & 7
    v = np.where(e > 0, (1 + m / 8) * 2.0 ** (e - 7), m / 8 * 2.0 ** -6)
    return np.where(b & 128, -v, v)


def values(words, scales, biases, mode, g):
    """Numbers of packed words [..., n] (any integer type) with scales (and biases) [..., 8 n / g] as floats or bytes."""
    w = words.astype(np.int64) & 0xFFFFFFFF
    codes = np.stack([(w >> (4 * i)) & 15 for i in range(8)], -1).reshape(words.shape[:-1] + (-1, g))
    if mode == "affine":
        v = scales[..., None].astype(np.float64) * codes + biases[..., None]
    else:
        s = e4m3(scales) if mode == "nvfp4" else 2.0 ** (scales.astype(np.float64) - 127)
        v = E2M1[codes] * s[..., None]
    return v.reshape(words.shape[:-1] + (-1,))


def rotary(x, positions, freqs, interleaved=False, scale=1.0, backward=False):
    """x [T, H, D] float64, positions [T], freqs [R / 2] (the float32 numbers)."""
    half = len(freqs)
    angle = positions.astype(np.float64)[:, None] * freqs.astype(np.float64)
    c, s = np.cos(angle)[:, None] * scale, np.sin(angle)[:, None] * scale * (-1 if backward else 1)
    i = np.arange(half)
    first, second = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
    y = x.copy()
    y[..., first] = x[..., first] * c - x[..., second] * s
    y[..., second] = x[..., first] * s + x[..., second] * c
    return y


def attention(q, k, v, n_rows, scale, causal=True, window=0, dead=None, steps=None):
    """One sequence: q [n, HQ, D], k and v [L, H, D]; dead [L] marks keys that are not there. Returns the output and, for
    each value of it, the sum of p |v| that error bounds are taken of, and the root of the sum of (p (v - o) e)^2, where e is
    the root of scale^2 sum (q k)^2: what independent errors of the values of k, of one relative size, come to. steps [L, H, D]: instead of |v| in that sum."""
    n, HQ, D = q.shape
    L, H = k.shape[:2]
    out, size, spread = np.zeros((n, HQ, D)), np.zeros((n, HQ, D)), np.zeros((n, HQ, D))
    for i in range(n):
        at = L - n_rows + i
        keys = np.arange(L)
        seen = keys <= at if causal else keys >= 0
        if window:
            seen = seen & (keys > at - window)
        if dead is not None:
            seen = seen & ~dead
        keys = keys[seen]
        if not len(keys):
            continue
        for h in range(HQ):
            kk, vv = k[keys, h // (HQ // H)], v[keys, h // (HQ // H)]
            score = kk @ q[i, h] * scale
            p = np.exp(score - score.max())
            p /= p.sum()
            out[i, h] = p @ vv
            size[i, h] = p @ (np.abs(vv) if steps is None else steps[keys, h // (HQ // H)])
            e = np.sqrt((kk * kk) @ (q[i, h] * q[i, h])) * abs(scale)
            spread[i, h] = np.sqrt((p * e) ** 2 @ (vv - out[i, h]) ** 2)
    return out, size, spread
