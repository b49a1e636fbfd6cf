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
