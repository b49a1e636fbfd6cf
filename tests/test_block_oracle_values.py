"""The heads' oracle on values that are not finite: without a norm, what is not turned stays the affair of its own place."""
import numpy as np

from oracle import prism_block as O


def test_heads_oracle_keeps_infinities_in_their_places():
    rng = np.random.default_rng(0)
    x, g = rng.normal(size=(1, 3, 8)), [rng.normal(size=(1, 1, 3, 8)), np.zeros((1, 0, 3, 8)), np.zeros((1, 0, 3, 1))]
    args = ((1, 0, 0), 8, 1, "none", 0.0, np.ones(8), None, np.array([0.5]), False, 1.0, np.arange(3)[None])
    clean, (dclean, _, _) = O.heads(x, *args)[0], O.heads_backward(x, g, *args)
    x[0, 1, 5], g[0][0, 0, 2, 7] = np.inf, np.nan
    y, (dx, dw, _) = O.heads(x, *args)[0], O.heads_backward(x, g, *args)
    assert y[0, 0, 1, 5] == np.inf and np.isnan(dx[0, 2, 7]) and np.isnan(dw[7])
    y[0, 0, 1, 5], dx[0, 2, 7] = clean[0, 0, 1, 5], dclean[0, 2, 7]
    assert np.array_equal(y, clean) and np.array_equal(dx, dclean)
