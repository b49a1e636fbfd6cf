"""fp64 oracle of the token operators (numpy): embedding and its gradient, the norm with the
residual's addition and its gradient, the 8-bit product, the log probabilities and their gradient.
Test infrastructure only; written from the definitions, one row or one token at a time where that is
the plainest form."""
import numpy as np


def embed(ids, table, scale):
    V = table.shape[0]
    out = np.zeros((ids.size, table.shape[1]))
    for i, t in enumerate(ids.ravel()):
        if 0 <= t < V:
            out[i] = scale * table[t].astype(np.float64)
    return out


def embed_backward(ids, dout, scale, V, onto=None):
    d = np.zeros((V, dout.shape[1])) if onto is None else onto.astype(np.float64).copy()
    for i, t in enumerate(ids.ravel()):
        if 0 <= t < V:
            d[t] += scale * dout[i].astype(np.float64)
    return d


def e4m3(x):
    """x rounded to the nearest e4m3 value (ties to even, saturating at 448), in float64."""
    x = np.asarray(x, dtype=np.float64)
    a = np.abs(x)
    with np.errstate(divide="ignore", invalid="ignore"):
        step = np.exp2(np.maximum(np.floor(np.log2(np.where(a > 0, a, 1.0))), -6) - 3)
    return np.sign(x) * np.minimum(np.round(a / step) * step, 448.0)


def blocks_of(D):
    return np.arange(D) // 128


def norm(x, residual, weight, eps):
    """r, y and the scales of y's blocks of 128 columns."""
    r = x.astype(np.float64) + (0 if residual is None else residual.astype(np.float64))
    y = r / np.sqrt(np.mean(r * r, axis=1, keepdims=True) + eps) * weight.astype(np.float64)
    n, D = y.shape
    peak = np.zeros((n, -(-D // 128)))
    for b in range(peak.shape[1]):
        peak[:, b] = np.max(np.abs(y[:, 128 * b:128 * b + 128]), axis=1, initial=0.0)
    return r, y, np.maximum(peak / 448.0, 2.0 ** -126)


def norm_backward(r, weight, eps, dy, dsum=None):
    r, w, dy = (np.asarray(a, dtype=np.float64) for a in (r, weight, dy))
    q = 1 / np.sqrt(np.mean(r * r, axis=1, keepdims=True) + eps)
    rh = r * q
    dx = q * (w * dy - rh * np.mean(w * dy * rh, axis=1, keepdims=True))
    return dx + (0 if dsum is None else np.asarray(dsum, dtype=np.float64)), np.sum(dy * rh, axis=0)
