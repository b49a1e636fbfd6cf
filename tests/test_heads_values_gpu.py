"""Heads with values that are not finite: where nothing is turned an infinity or NaN stays the affair of its own place.

What the oracle makes of them in 64 bits has to come out: the same NaN, the same infinities, and of the finite values those of the tolerance
that tests/test_heads_gpu.py derives."""
import numpy as np
import pytest
import torch

from oracle import prism_block as O
from ssm_sequence_layer_gb300 import binding as B
from ssm_sequence_layer_gb300 import build
from tests.test_heads_gpu import DT, f64, half_ulp, pair_size, setup, u

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    build.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"


# d, rot, interleaved: pairs of whole units, of single values, within a unit whose other pairs are not turned, more units than lanes
SHAPES = [(64, 0, False), (64, 32, False), (64, 6, True), (64, 20, True), (30, 6, False), (30, 6, True), (512, 64, False), (512, 36, True), (511, 20, False)]


def spoil(x, at):
    inf, nan = float("inf"), float("nan")
    for i, j in enumerate(at):
        x[..., j] = (inf, -inf, nan)[i % 3]


def same(got, ref, tol, io):
    special = ~np.isfinite(ref)
    assert np.array_equal(np.isnan(got), np.isnan(ref))
    assert np.array_equal(got[special & ~np.isnan(ref)], ref[special & ~np.isnan(ref)])
    ok = ~special
    got, ref = np.where(ok, got, 0), np.where(ok, ref, 0)
    assert np.all(np.abs(got - ref)[ok] <= (tol + half_ulp(io, np.abs(ref) + tol) * 1.0001)[ok])


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("d,rot,interleaved", SHAPES)
def test_values_that_are_not_finite(io, d, rot, interleaved):
    Bn, T, heads = 2, 5, (3, 2, 1)
    x, width, form, args = setup(io, Bn, T, heads, d, 8, rot, "none", True, interleaved, 1.25, True, 0)
    # places that are not turned: the first, the last, and two whose neighbours are finite; none, then one that is turned
    at = sorted({rot, rot + 1, rot + 5, d - 1})
    clean = x.clone()
    spoil(x[0, 1, :d], at)                       # the first query head of a token
    spoil(x[1, 3, (heads[0] + 1) * d:(heads[0] + 2) * d], at)  # the last key head of another
    if rot:
        x[1, 0, d + 1] = float("inf")            # one that is turned: its partner is NaN or infinite too
    with B.Tokens(Bn * T, 64, 8, io=io) as t:
        out, before = t.heads(x, **form), t.heads(clean, **form)
        torch.cuda.synchronize()
    with np.errstate(invalid="ignore"):
        q, k, v = O.heads(f64(x), *args)
        cq, ck, _ = O.heads(f64(clean), *args)
    for key, ref, finite in (("q", q, cq), ("k", k, ck)):
        tol = ((d / 2 + 16) * u) * pair_size(finite / (1.25 if rot else 1.0), rot, interleaved, 1.25)
        same(f64(out[key]), ref, tol, io)
        assert torch.equal(torch.where(torch.isfinite(out[key]), out[key], before[key]), before[key])
    assert torch.equal(out["v"], before["v"])


@pytest.mark.parametrize("io,grads_io", [("bf16", "f32"), ("bf16", "bf16"), ("f32", "f32")])
@pytest.mark.parametrize("d,rot,interleaved", SHAPES)
def test_cotangents_that_are_not_finite(io, grads_io, d, rot, interleaved):
    """Without a norm each place's cotangent reaches its own place only, beyond the turned ones."""
    Bn, T, heads = 2, 5, (3, 2, 1)
    x, width, form, args = setup(io, Bn, T, heads, d, 8, rot, "none", True, interleaved, 1.25, True, 0)
    g = torch.Generator().manual_seed(9)
    grads = {key: torch.randn(Bn, H, T, size, generator=g).to(DT[grads_io]).cuda() for key, H, size in (("dq", 3, d), ("dk", 2, d), ("dv", 1, 8))}
    clean = {key: t.clone() for key, t in grads.items()}
    at = sorted({rot, rot + 1, rot + 5, d - 1})
    spoil(grads["dq"][0, 2, 1], at)
    spoil(grads["dk"][1, 0, 4], at)
    with B.Tokens(Bn * T, 64, 8, io=io) as t:
        out, before = t.heads_backward(x, grads, **form), t.heads_backward(x, clean, **form)
        torch.cuda.synchronize()
    with np.errstate(invalid="ignore"):
        dx, dqw, dkw = O.heads_backward(f64(x), [f64(grads[key]) for key in ("dq", "dk", "dv")], *args)
    for key, ref in (("dx", dx), ("dq_weight", dqw), ("dk_weight", dkw)):
        got, old = f64(out[key]), f64(before[key])
        assert np.array_equal(np.isnan(got), np.isnan(ref)), key
        special = ~np.isfinite(ref)
        assert special.any() and np.array_equal(got[special & ~np.isnan(ref)], ref[special & ~np.isnan(ref)]), key
        assert np.array_equal(got[~special], old[~special]), key


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("norm", ["unit", "rms"])
def test_an_infinite_value_of_a_normed_row(io, norm):
    """Its square makes the row's scale zero: the row is zero but for the place itself, which is NaN."""
    x = torch.ones(1, 2, 64, dtype=DT[io], device="cuda")
    x[0, 1, 40] = float("inf")
    with B.Tokens(2, 64, 8, io=io) as t:
        y = t.heads(x, (1, 0, 0), 64, norm=norm, inv_freq=torch.ones(8, device="cuda"))["q"][0, 0]
    assert torch.isfinite(y[0]).all() and torch.isnan(y[1, 40])
    rest = torch.arange(64, device="cuda") != 40
    assert not y[1][rest].any()
