"""The rotation's frequencies: the plain ones, each scaling at its ends, and what is refused."""
import math

import pytest
import torch

from ssm_sequence_layer_gb300.rotary import rotary_frequencies


def test_plain_frequencies():
    f, a = rotary_frequencies(8)
    assert f.dtype is torch.float32 and a == 1.0
    assert torch.allclose(f, torch.tensor([1.0, 0.1, 0.01, 0.001]), rtol=2 ** -23, atol=0)
    assert rotary_frequencies(0)[0].shape == (0,)


def test_scalings_at_their_ends():
    plain = rotary_frequencies(64)[0].double()
    linear = rotary_frequencies(64, scaling="linear", factor=8)[0].double()
    assert torch.allclose(linear * 8, plain, rtol=2 ** -22, atol=0)
    base = rotary_frequencies(64, scaling="base", factor=8)[0].double()
    assert base[0] == plain[0] and abs(base[-1] / linear[-1] - 1) < 1e-6 and torch.all(base[1:] < plain[1:])
    parts, amplitude = rotary_frequencies(64, scaling="by parts", factor=8, original_length=4096)
    parts = parts.double()
    turns = 4096 * plain / (2 * math.pi)
    assert torch.allclose(parts[turns >= 32], plain[turns >= 32], rtol=2 ** -22, atol=0)
    assert torch.allclose(parts[turns <= 1] * 8, plain[turns <= 1], rtol=2 ** -22, atol=0)
    between = (turns > 1) & (turns < 32)
    assert between.any() and torch.all(parts[between] < plain[between]) and torch.all(parts[between] > plain[between] / 8)
    assert abs(amplitude - (1 + 0.1 * math.log(8))) < 1e-12
    assert torch.equal(rotary_frequencies(64, scaling="by parts", factor=1, original_length=4096)[0], rotary_frequencies(64)[0])


@pytest.mark.parametrize("kw", [dict(rot=7), dict(rot=-2), dict(rot=8, scaling="cubic"), dict(rot=8, scaling="linear", factor=0.5), dict(rot=2, scaling="base", factor=2),
                                dict(rot=8, scaling="by parts", factor=2), dict(rot=8, scaling="by parts", factor=2, original_length=10, fast=1, slow=1),
                                dict(rot=8, scaling="linear", factor=float("nan"))])
def test_refusals(kw):
    with pytest.raises(ValueError):
        rotary_frequencies(**kw)
