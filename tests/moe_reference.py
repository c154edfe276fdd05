"""The mixture-of-experts operators from their definitions, in 64 bits on the
CPU (numpy), sharing no code with the library or the oracle."""
import numpy as np

E2M1 = np.array([0, .5, 1, 1.5, 2, 3, 4, 6, -0., -.5, -1, -1.5, -2, -3, -4, -6])


def scores(x, score):
    """Scores of logits x [T, E] (float64); 0 where a logit is not finite."""
    ok = np.isfinite(x)
    x = np.where(ok, x, 0.0)
    if score == "sigmoid":
        return np.where(ok, 1 / (1 + np.exp(-x)), 0.0)
    top = np.where(ok, x, -np.inf).max(1, keepdims=True)
    e = np.where(ok, np.exp(x - np.where(np.isfinite(top), top, 0.0)), 0.0)
    s = e.sum(1, keepdims=True)
    return np.divide(e, s, out=np.zeros_like(e), where=s > 0)


def route(x, k, score="softmax", bias=None, renormalize=True, scale=1.0, groups=1, groups_kept=1, group_top=1):
    """(weights [T, k], experts [T, k])."""
    T, E = x.shape
    s = scores(x, score)
    w, ids = np.zeros((T, k)), np.full((T, k), -1, np.int32)
    per = E // groups
    for t in range(T):
        free = np.isfinite(x[t])
        key = x[t].copy() if bias is None else s[t] + bias
        free &= ~np.isnan(key) & (key > -np.inf)
        value = s[t] if bias is None else key
        if groups_kept < groups:
            g = []
            for i in range(groups):
                v = sorted([value[e] if free[e] else -np.inf for e in range(i * per, (i + 1) * per)], reverse=True)
                g.append(sum(v[:group_top]) if v[group_top - 1] > -np.inf else -np.inf)
            best = sorted(range(groups), key=lambda i: (-g[i], i))[:groups_kept]
            free &= np.isin(np.arange(E) // per, best)
        order = sorted([e for e in range(E) if free[e]], key=lambda e: (-key[e], e))[:k]
        ids[t, :len(order)] = order
        w[t, :len(order)] = s[t, order]
    if renormalize:
        w = w / (w.sum(1, keepdims=True) + 1e-20)
    return scale * w, ids


def route_weights(x, ids, score, renormalize, scale):
    """The weights as a function of the logits for a fixed choice."""
    s = scores(x, score)
    w = np.where(ids >= 0, np.take_along_axis(s, np.maximum(ids, 0), 1), 0.0)
    return scale * (w / (w.sum(1, keepdims=True) + 1e-20) if renormalize else w)


def route_grad(x, ids, g, score, renormalize, scale):
    s = scores(x, score)
    T, E = x.shape
    out = np.zeros((T, E))
    for t in range(T):
        live = ids[t] >= 0
        c = ids[t][live]
        q, gg = s[t, c], g[t][live]
        if renormalize:
            S = q.sum() + 1e-20
            ds = scale * (gg / S - (gg * q).sum() / S ** 2)
        else:
            ds = scale * gg
        full = np.zeros(E)
        full[c] = ds
        if score == "sigmoid":
            out[t] = full * s[t] * (1 - s[t])
        else:
            out[t] = s[t] * (full - (full * s[t]).sum())
            if renormalize:
                out[t] = np.where(np.isin(np.arange(E), c), out[t], 0.0)
    return np.where(np.isfinite(x), out, 0.0)


def mxfp4_decode(words, scale_bytes):
    """uint32 words [..., K/8] and bytes [..., K/32] -> float64 [..., K]."""
    codes = (words[..., None] >> np.arange(0, 32, 4, dtype=np.uint32)) & 15
    v = E2M1[codes].reshape(scale_bytes.shape + (32,))
    unit = np.where(scale_bytes == 255, np.nan, np.exp2(scale_bytes.astype(np.float64) - 127))
    return (v * unit[..., None]).reshape(words.shape[:-1] + (-1,))


def mxfp4_round(x):
    """x rounded to mxfp4 along its last axis (float64 in, the values out)."""
    v = x.reshape(x.shape[:-1] + (-1, 32))
    bad = ~np.isfinite(v).all(-1, keepdims=True)
    v = np.where(bad, 0.0, v)
    m = np.abs(v).max(-1, keepdims=True)
    e = np.where(m > 0, np.floor(np.log2(np.where(m > 0, m, 1.0))), 0.0)
    e = np.where(np.exp2(e) > np.where(m > 0, m, 1.0), e - 1, e)        # log2 may round up to a power of two
    e = np.where(np.exp2(e + 1) <= np.where(m > 0, m, 1.0), e + 1, e)
    unit = np.exp2(np.clip(e - 2, -127, 127))
    a = np.minimum(np.abs(v) / unit, 6.0)
    step = np.where(a < 2, .5, np.where(a < 4, 1.0, 2.0))
    r = np.sign(v) * np.rint(a / step) * step * unit                     # rint's even multiple is the even code
    r = np.where(m > 0, r, 0.0)
    return np.where(bad, np.nan, r).reshape(x.shape)


def swiglu(x):
    K = x.shape[-1] // 2
    g, u = x[..., :K], x[..., K:]
    return g / (1 + np.exp(-g)) * u


def gather_product(x, w, ids):
    """x [B, K], w [E, N, K], ids [B, k] -> [B, k, N]; rows without an expert are zeros."""
    y = np.zeros(ids.shape + (w.shape[1],))
    for e in np.unique(ids[(ids >= 0) & (ids < len(w))]):
        b, j = np.nonzero(ids == e)
        y[b, j] = x[b] @ w[e].T
    return y


def combine(h, w, ids=None):
    live = np.ones(w.shape, bool) if ids is None else ids >= 0
    return np.where(live[..., None], w[..., None] * h, 0.0).sum(1)


def combine_grad(gy, h, w, ids=None):
    live = np.ones(w.shape, bool) if ids is None else ids >= 0
    gh = np.where(live[..., None], w[..., None] * gy[:, None, :], 0.0)
    gw = np.where(live, np.where(live[..., None], h * gy[:, None, :], 0.0).sum(2), 0.0)
    return gh, gw
