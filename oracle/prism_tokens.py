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


LOWEST = -3.38953139e38  # bfloat16's: a logit at or below it is masked


def z_of(logits, c):
    """c logits; -inf where the logit is a mask's value or the product overflows to -inf in float32."""
    with np.errstate(over="ignore", invalid="ignore"):
        overflows = logits.astype(np.float32) * np.float32(c) == -np.inf
    return np.where((logits <= LOWEST * (1 - 1e-9)) | overflows, -np.inf, c * logits.astype(np.float64))


def token_logprobs(logits, targets, c, k):
    """lse, logprob, entropy, top ids and top log probabilities, row by row."""
    z = z_of(logits, c)
    n, V = z.shape
    out = {"lse": np.zeros(n), "logprob": np.zeros(n), "entropy": np.zeros(n), "top_ids": np.full((n, k), -1, dtype=np.int64),
           "top_logprob": np.full((n, k), -np.inf)}
    for i in range(n):
        row = z[i]
        live = np.nonzero(row != -np.inf)[0]
        with np.errstate(invalid="ignore"):
            m, logs = 0.0, -np.inf
            if live.size == 0:
                h = 0.0
            elif np.isnan(row).any() or np.isposinf(row).any():
                logs, h = np.nan, np.nan
            else:
                m = row[live].max()
                e = np.exp(row[live] - m)
                logs = np.log(e.sum())
                h = logs - np.sum(e * (row[live] - m)) / e.sum()
            out["lse"][i], out["entropy"][i] = m + logs, h
            if targets is not None and 0 <= targets[i] < V:
                out["logprob"][i] = -np.inf if live.size == 0 else (row[targets[i]] - m) - logs
            nan = np.isnan(row[live])
            order = live[np.lexsort((live, np.where(nan, 0.0, -row[live]), ~nan))][:k]
            out["top_ids"][i, :order.size] = order
            out["top_logprob"][i, :order.size] = (row[order] - m) - logs
    return out


def token_logprobs_backward(logits, targets, c, lse, entropy, dlogprob, dentropy):
    z = z_of(logits, c)
    g = np.zeros_like(z)
    for i in range(z.shape[0]):
        if lse[i] == -np.inf:
            continue
        live = z[i] != -np.inf
        lp = z[i][live] - lse[i]
        p = np.exp(lp)
        t = targets[i] if targets is not None and dlogprob is not None and 0 <= targets[i] < z.shape[1] else -1
        d = dlogprob[i] if t >= 0 else 0.0
        row = -d * p
        if dentropy is not None:
            row = row - dentropy[i] * p * (lp + entropy[i])
        g[i][live] = row
        if t >= 0 and live[t]:
            g[i, t] += d
    return c * g
