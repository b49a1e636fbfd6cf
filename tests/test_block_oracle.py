"""The block operators' fp64 oracle (oracle/prism_block.py) against torch in float64 and its differentiation, against differences,
and against brute force, so that what the kernels are compared with is held by something else."""
import itertools
import math

import numpy as np
import pytest
import torch

from oracle import prism_block as O

T64 = torch.float64


def near(got, ref, tol=1e-11):
    ref = ref.detach().numpy() if isinstance(ref, torch.Tensor) else np.asarray(ref)
    assert got.shape == ref.shape and np.max(np.abs(got - ref), initial=0) <= tol * (1 + np.max(np.abs(ref), initial=0))


@pytest.mark.parametrize("act", ["none", "gelu", "silu"])
def test_linear_and_its_gradients(act):
    g = torch.Generator().manual_seed(1)
    z0 = torch.randn(9, 6, generator=g, dtype=T64)  # the pre-activation that x comes from
    W, b, res, dy = (torch.randn(*s, generator=g, dtype=T64) for s in ((5, 6), (5,), (9, 5), (9, 5)))
    f = {"none": lambda v: v, "gelu": torch.nn.functional.gelu, "silu": torch.nn.functional.silu}[act]
    z, W, b = z0.clone().requires_grad_(), W.requires_grad_(), b.requires_grad_()
    pre = torch.nn.functional.linear(f(z), W, b)
    y = f(pre) + res
    got_pre, got = O.linear(f(z0).numpy(), W.detach().numpy(), b.detach().numpy(), act, res.numpy())
    near(got_pre, pre)
    near(got, y)
    dsum = torch.randn(9, 6, generator=g, dtype=T64)
    (pre * dy).sum().backward()
    near(O.linear_backward(dy.numpy(), W.detach().numpy(), act, z0.numpy(), dsum.numpy()), z.grad + dsum)
    dW, db = O.linear_weight_backward(dy.numpy(), f(z0).numpy())
    near(dW, W.grad)
    near(db, b.grad)


@pytest.mark.parametrize("norm", ["none", "unit", "rms"])
@pytest.mark.parametrize("interleaved", [False, True])
def test_heads_and_their_gradient(norm, interleaved):
    rng = np.random.default_rng(3)
    B, T, heads, d, dv, rot = 2, 3, (2, 1, 2), 6, 5, 4
    x = rng.normal(size=(B, T, 3 * d + 2 * dv))
    w = rng.normal(size=(2, d)) * 0.3 + 1
    freq, pos = np.array([0.7, 0.05]), rng.integers(-50, 50, size=(B, T))
    args = (heads, d, dv, norm, 1e-3, w[0], w[1], freq, interleaved, 1.25, pos)
    q, k, v = O.heads(x, *args)
    # a pair as a complex number times e^(i angle)
    y = x[:, :, 2 * d:3 * d]
    size = {"none": 1.0, "unit": np.sqrt((y ** 2).sum(-1, keepdims=True) + 1e-3), "rms": np.sqrt((y ** 2).mean(-1, keepdims=True) + 1e-3)}[norm]
    y = y / size * w[1]
    first, second = ((0, 2), (1, 3)) if interleaved else ((0, 1), (2, 3))
    z = (y[..., first] + 1j * y[..., second]) * 1.25 * np.exp(1j * pos[..., None] * freq)
    near(k[:, 0][..., first], z.real)
    near(k[:, 0][..., second], z.imag)
    near(k[:, 0, :, 4:], y[..., 4:])
    near(v[:, 1], x[:, :, 3 * d + dv:])
    # the gradient against differences of the forward, along every input
    grads = [rng.normal(size=a.shape) for a in (q, k, v)]
    dx, dqw, dkw = O.heads_backward(x, grads, *args)
    loss = lambda x_, w_: sum((a * g).sum() for a, g in zip(O.heads(x_, heads, d, dv, norm, 1e-3, w_[0], w_[1], freq, interleaved, 1.25, pos), grads))  # noqa: E731
    h = 1e-5
    for at in itertools.product(range(B), range(T), range(0, x.shape[2], 3)):
        e = np.zeros_like(x)
        e[at] = h
        assert abs((loss(x + e, w) - loss(x - e, w)) / (2 * h) - dx[at]) < 1e-7
    for z_, dw in enumerate((dqw, dkw)):
        for j in range(d):
            e = np.zeros_like(w)
            e[z_, j] = h
            assert abs((loss(x, w + e) - loss(x, w - e)) / (2 * h) - dw[j]) < 1e-7


def test_angles_of_far_positions():
    for pos, f in ((0, 1.0), (7, 0.5), (-3, 1.0), (1000, 0.25)):
        assert abs(math.remainder(pos * f, 2 * math.pi) - O.angle(pos, f)) < 1e-12
    # 2^40 turns by a whole number of radians: against the reduction in three parts of 2 pi
    far = (1 << 40) + 12345
    from decimal import Decimal, getcontext
    getcontext().prec = 50
    two_pi = 2 * Decimal("3.14159265358979323846264338327950288419716939937510")
    rest = Decimal(far) - (Decimal(far) / two_pi).to_integral_value() * two_pi
    assert abs(float(rest) - O.angle(far, 1.0)) < 1e-15


def test_draws_by_brute_force():
    """Every rule on a small row: the kept set from the definition's prefixes, the token from the masses' intervals."""
    rng = np.random.default_rng(5)
    row = np.array([1.0, 3.0, -np.inf, 3.0, 0.5, 2.0, -3.4e38, 2.0])
    p = np.exp(row - 3.0)
    order = [1, 3, 5, 7, 0, 4]  # by falling logit, then by rising id
    for k, pp, mp in itertools.product((0, 1, 2, 3, 99), (0.0, 0.3, 0.6, 0.9, 1.0), (0.0, 0.3, 0.4, 1.0, 1.5)):
        first = order[:k] if k else order
        total = sum(p[j] for j in first)
        kept = first
        if pp < 1:
            for m in range(1, len(first) + 1):
                if sum(p[j] for j in first[:m]) >= pp * total:
                    kept = first[:m]
                    break
        if mp > 0:
            kept = [j for j in kept if p[j] >= mp] or order[:1]
        for u in rng.random(5):
            ids, logprob, number = O.sample(row[None], np.array([u]), None, np.array([k]), np.array([pp]), np.array([mp]))
            mass, want = sum(p[j] for j in kept), None
            run = 0.0
            for j in sorted(kept):
                run += p[j]
                if run > u * mass:
                    want = j
                    break
            assert ids[0] == want and number[0] == len(kept)
            assert abs(logprob[0] - math.log(p[want] / mass)) < 1e-12


def test_rows_without_a_token():
    inf, nan = np.inf, np.nan
    ids, logprob, kept = O.sample(np.array([[-inf, -inf], [nan, 1.0], [inf, 0.0], [1.0, 2.0]]), np.full(4, 0.5), np.array([1.0, 1.0, 1.0, 0.0]), None, None, None)
    assert ids.tolist() == [-1] * 4 and kept.tolist() == [0] * 4
    assert logprob[0] == -inf and np.isnan(logprob[1:]).all()
