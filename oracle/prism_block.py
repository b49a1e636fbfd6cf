"""fp64 oracle of the block's operators (numpy): the product with bias, activation and residual and its gradients, the
heads' norm and rotation and its gradient, and the draw of a token.  Test infrastructure only; written from the
definitions, one row at a time where that is the plainest form."""
import math
from decimal import Decimal, getcontext
from fractions import Fraction

import numpy as np

from .prism_tokens import z_of

F = np.float64
_erf = np.vectorize(math.erfc, otypes=[F])


def act_value(act, z):
    if act == "gelu":
        return z * 0.5 * _erf(-z / math.sqrt(2))
    return z / (1 + np.exp(-z)) if act == "silu" else z


def act_slope(act, z):
    if act == "gelu":
        return 0.5 * _erf(-z / math.sqrt(2)) + z * np.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    if act == "silu":
        p = 1 / (1 + np.exp(-z))
        return p + z * p * (1 - p)
    return np.ones_like(z)


def linear(x, W, bias, act, residual):
    """pre and y."""
    pre = x.astype(F) @ W.astype(F).T + (0 if bias is None else bias.astype(F))
    return pre, act_value(act, pre) + (0 if residual is None else residual.astype(F))


def linear_backward(dy, W, act, pre, dsum):
    dx = dy.astype(F) @ W.astype(F)
    if act != "none":
        dx = dx * act_slope(act, pre.astype(F))
    return dx + (0 if dsum is None else dsum.astype(F))


def linear_weight_backward(dy, x):
    return dy.astype(F).T @ x.astype(F), dy.astype(F).sum(0)


getcontext().prec = 50
TWO_PI = 2 * Fraction(Decimal("3.14159265358979323846264338327950288419716939937510"))


def angle(position, inv_freq):
    """position inv_freq less its whole turns, for one pair of numbers of any size."""
    turns = Fraction(int(position)) * Fraction(float(inv_freq)) / TWO_PI
    return float((turns - round(turns)) * TWO_PI)


def _pairs(rot, interleaved):
    i = np.arange(rot // 2)
    return (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)


def _size(x, norm, eps):
    if norm == "none":
        return np.ones(x.shape[:-1] + (1,))
    sq = x * x
    return np.sqrt((sq.mean(-1, keepdims=True) if norm == "rms" else sq.sum(-1, keepdims=True)) + eps)


def _angles(positions, inv_freq):
    return np.array([[angle(p, f) for f in inv_freq] for p in positions.ravel()]).reshape(positions.shape + (len(inv_freq),))


def heads(x, heads_, d, dv, norm, eps, q_weight, k_weight, inv_freq, interleaved, amplitude, positions):
    """q, k, v as [B, H, T, size] of rows x [B, T, >= columns]."""
    B, T, _ = x.shape
    x = x.astype(F)
    Hq, Hk, Hv = heads_
    t = _angles(positions, inv_freq)[:, :, None, :]
    first, second = _pairs(2 * len(inv_freq), interleaved)
    out, at = [], 0
    for H, w in ((Hq, q_weight), (Hk, k_weight)):
        y = x[:, :, at:at + H * d].reshape(B, T, H, d)
        at += H * d
        y = y / _size(y, norm, eps) * (1 if w is None else w.astype(F))
        a, b = y[..., first].copy(), y[..., second].copy()
        y = y.copy()
        y[..., first] = amplitude * (a * np.cos(t) - b * np.sin(t))
        y[..., second] = amplitude * (a * np.sin(t) + b * np.cos(t))
        out.append(y.transpose(0, 2, 1, 3))
    out.append(x[:, :, at:at + Hv * dv].reshape(B, T, Hv, dv).transpose(0, 2, 1, 3))
    return out


def heads_backward(x, grads, heads_, d, dv, norm, eps, q_weight, k_weight, inv_freq, interleaved, amplitude, positions):
    """dx [B, T, columns] and the weights' gradients; grads: dq, dk, dv."""
    B, T, _ = x.shape
    x = x.astype(F)
    t = _angles(positions, inv_freq)[:, :, None, :]
    first, second = _pairs(2 * len(inv_freq), interleaved)
    cols, dws, at = [], [], 0
    for H, w, g in ((heads_[0], q_weight, grads[0]), (heads_[1], k_weight, grads[1])):
        y = x[:, :, at:at + H * d].reshape(B, T, H, d)
        at += H * d
        g = g.astype(F).transpose(0, 2, 1, 3).copy()
        a, b = g[..., first].copy(), g[..., second].copy()
        g[..., first] = amplitude * (a * np.cos(t) + b * np.sin(t))
        g[..., second] = amplitude * (b * np.cos(t) - a * np.sin(t))
        size = _size(y, norm, eps)
        wg = g * (1 if w is None else w.astype(F))
        dws.append((g * y / size).sum((0, 1, 2)))
        along = 0.0  # without a norm there is no term along x, be the sum infinite
        if norm != "none":
            along = y * (1.0 if norm == "unit" else 1.0 / d) * (wg * y).sum(-1, keepdims=True) / size ** 3
        cols.append((wg / size - along).reshape(B, T, H * d))
    cols.append(grads[2].astype(F).transpose(0, 2, 1, 3).reshape(B, T, -1))
    return np.concatenate(cols, 2), dws[0], dws[1]


def sample(logits, u, inv_temperature, top_k, top_p, min_p):
    """ids, log shares and numbers kept; each rule an array over the rows or None."""
    n, V = logits.shape
    ids, logprob, kept = np.full(n, -1, dtype=np.int64), np.full(n, -np.inf), np.zeros(n, dtype=np.int64)
    for i in range(n):
        c = 1.0 if inv_temperature is None else float(inv_temperature[i])
        row = logits[i].astype(F) + 0.0
        if not 2.0 ** -60 <= c <= 2.0 ** 126 or np.isnan(row).any() or np.isposinf(row).any():
            logprob[i] = np.nan
            continue
        z = z_of(logits[i:i + 1], c)[0]
        live = np.nonzero(z != -np.inf)[0]
        if live.size == 0:
            continue
        order = live[np.lexsort((live, -row[live]))]
        with np.errstate(under="ignore"):
            e = np.exp(z[order] - z[order[0]])
        m = order.size
        k = 0 if top_k is None else int(top_k[i])
        if 0 < k < m:
            m = k
        p = 1.0 if top_p is None else float(top_p[i])
        if p < 1:  # the fewest whose mass reaches p of that of the first m
            m = min(m, max(1, int(np.searchsorted(np.cumsum(e[:m]), p * e[:m].sum())) + 1))
        q = 0.0 if min_p is None else float(min_p[i])
        if q > 0:
            m = min(m, max(1, int((z[order] - z[order[0]] >= math.log(q)).sum())))  # e >= q, told where e rounds to q
        chosen = np.zeros(V)
        chosen[order[:m]] = e[:m]
        running = np.cumsum(chosen)
        at = float(u[i]) if u[i] > 0 else 0.0
        ids[i] = np.nonzero(chosen)[0][-1] if at >= 1 else np.searchsorted(running, at * running[-1], side="right")
        logprob[i], kept[i] = math.log(chosen[ids[i]] / running[-1]), m
    return ids, logprob, kept
