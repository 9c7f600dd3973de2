"""Plain numpy definitions, in 64 bits, of the gate's operators and the dense projection.

Test infrastructure: no code of the package.
"""
import numpy as np


def clean(l):
    """Logits as they count: NaN as -inf, +inf as the largest finite fp32 value."""
    l = np.where(np.isnan(l), -np.inf, l.astype(np.float64))
    return np.minimum(l, float(np.finfo(np.float32).max))


def scores(l, score):
    l = clean(l)
    off = np.isneginf(l)
    if score == "sigmoid":
        with np.errstate(over="ignore"):
            return np.where(off, 0.0, 1.0 / (1.0 + np.exp(-l)))
    mx = l.max(1, keepdims=True)
    e = np.where(off, 0.0, np.exp(l - np.where(np.isneginf(mx), 0.0, mx)))
    z = e.sum(1, keepdims=True)
    return e / np.where(z > 0, z, 1.0)


def ratios(l, score):
    """s / sum s along the rows: from e^(l - m) / (1 + e^l), m the smaller of 0 and the row's
    largest logit, whose common factor e^-m keeps 64 bits from underflowing."""
    l = clean(l)
    off = np.isneginf(l)
    m = l.max(1, keepdims=True)
    m = np.where(np.isneginf(m), 0.0, m)
    if score == "sigmoid":
        m = np.minimum(m, 0.0)
        with np.errstate(over="ignore"):
            e = np.where(l > 0, 1.0 / (1.0 + np.exp(-l)),
                         np.exp(np.minimum(l, 0.0) - m) / (1.0 + np.exp(np.minimum(l, 0.0))))
    else:
        e = np.exp(l - m)
    e = np.where(off, 0.0, e)
    z = e.sum(1, keepdims=True)
    return e / np.where(z > 0, z, 1.0)


def shares(l, score):
    return ratios(l, score)


def weights(l, idx, score, renorm, scale):
    if renorm:
        return ratios(np.take_along_axis(l, idx, axis=1), score) * scale
    return np.take_along_axis(scores(l, score), idx, axis=1) * scale


def route(l, bias, k, score="softmax", renorm=False, scale=1.0, n_groups=0, topk_groups=0,
          group_top=0):
    """(indices, weights, p_mean), token by token."""
    T, N = l.shape
    s = scores(l, score)
    lc = clean(l)
    b = np.zeros(N) if bias is None else np.where(np.isnan(bias), -np.inf, bias.astype(np.float64))
    off = np.isneginf(lc) | np.isneginf(b)[None, :]
    v = np.where(off, -np.inf, s + np.where(np.isneginf(b), 0.0, b))
    rank = v if bias is not None else lc
    nodes = n_groups > 1 and topk_groups < n_groups
    idx = np.empty((T, k), np.int64)
    for t in range(T):
        allowed = np.ones(N, bool)
        if nodes:
            per = N // n_groups
            gs = []
            for g in range(n_groups):
                top = sorted((x for x in v[t, g * per:(g + 1) * per] if x != -np.inf), reverse=True)
                total = 0.0
                for x in top[:group_top]:
                    total += x
                # a node without any expert left is behind every other
                gs.append(total)
            best = sorted(range(n_groups), key=lambda g: (-gs[g], g))[:topk_groups]
            allowed = np.isin(np.arange(N) // per, best)
        order = sorted(np.nonzero(allowed)[0],
                       key=lambda e: (off[t, e], 0.0 if off[t, e] else -rank[t, e], e))
        idx[t] = order[:k]
    return idx, weights(l, idx, score, renorm, scale), shares(l, score).mean(0) if T else np.zeros(N)


def route_loss(l, idx, g, c, score, renorm, scale):
    """sum g w + sum c p_mean, for differences."""
    return float((g * weights(l, idx, score, renorm, scale)).sum() + (c * shares(l, score).mean(0)).sum())


def route_grad(l, idx, g, c, score, renorm, scale):
    """Gradient of route_loss, and the size of its terms (for tolerances)."""
    T, N = l.shape
    s = scores(l, score)
    q = shares(l, score)
    ds_over = np.zeros_like(s)          # s * dL/ds, split by its parts' absolute sizes
    mag = np.zeros_like(s)
    sk = np.take_along_axis(s, idx, axis=1)
    gg = scale * g
    if renorm:
        r = ratios(np.take_along_axis(l, idx, axis=1), score)
        u = r * (gg - (gg * r).sum(1, keepdims=True))
        um = np.abs(r) * (np.abs(gg) + np.abs(gg * r).sum(1, keepdims=True))
    else:
        u = sk * gg
        um = np.abs(u)
    for j in range(idx.shape[1]):
        rows = np.arange(T)
        np.add.at(ds_over, (rows, idx[:, j]), u[:, j])
        np.add.at(mag, (rows, idx[:, j]), um[:, j])
    cc = c[None, :] / T
    ds_over += q * (cc - (cc * q).sum(1, keepdims=True))
    mag += q * (np.abs(cc) + np.abs(cc * q).sum(1, keepdims=True))
    if score == "sigmoid":
        with np.errstate(over="ignore"):
            om = 1.0 / (1.0 + np.exp(clean(l)))
        return om * ds_over, om * mag
    # over a softmax the gradient also loses its mean under s; what is divided by a sum has none
    tot = 0.0 if renorm else u.sum(1, keepdims=True)
    totm = 0.0 if renorm else um.sum(1, keepdims=True)
    return ds_over - s * tot, mag + s * totm


def act(name, z):
    from scipy.special import erf, expit
    if name == "relu":
        return np.where(z < 0, 0.0, z)
    if name == "silu":
        return z * expit(z)
    if name == "gelu":
        return 0.5 * z * (1 + erf(z / np.sqrt(2)))
    if name == "gelu_tanh":
        return 0.5 * z * (1 + np.tanh(np.sqrt(2 / np.pi) * (z + 0.044715 * z ** 3)))
    return z


def act_grad(name, z):
    from scipy.special import erf, expit
    if name == "relu":
        return (z > 0).astype(np.float64)
    if name == "silu":
        s = expit(z)
        return s * (1 + z * (1 - s))
    if name == "gelu":
        return 0.5 * (1 + erf(z / np.sqrt(2))) + z * np.exp(-z * z / 2) / np.sqrt(2 * np.pi)
    if name == "gelu_tanh":
        a = np.sqrt(2 / np.pi)
        t = np.tanh(a * (z + 0.044715 * z ** 3))
        return 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * a * (1 + 3 * 0.044715 * z * z)
    return np.ones_like(z)
