"""The position rotation's frequencies for ``Tokens.heads``, also for contexts longer than a model was trained on.

A pair i of the first ``rot`` values of a head is turned by position * inv_freq[i] and multiplied by an amplitude.

An amplitude other than 1 belongs to attention, where it scales the products of queries and keys.  The recurrent layer's step along a
key is 1 - beta |k|^2: it takes keys of length one, so leave the amplitude out there (with beta = 1 a length above sqrt(2) makes the state grow).
"""
from __future__ import annotations

import math


def rotary_frequencies(rot, base=10000.0, scaling=None, factor=1.0, original_length=None, fast=32.0, slow=1.0, device=None):
    """(inv_freq [rot / 2] float32, amplitude) with inv_freq[i] = base ** (-2 i / rot), scaled for contexts ``factor``
    times as long as trained on:
      None        not scaled
      "linear"    every frequency divided by the factor (positions are squeezed together)
      "base"      a base larger by factor ** (rot / (rot - 2)): the slowest pair as with "linear", the fastest as before
      "by parts"  pairs that turn at least ``fast`` times within original_length as before, those that turn at most
                  ``slow`` times as with "linear", between them a mix in proportion to the turns; the amplitude is
                  1 + 0.1 log(factor) (arXiv 2309.00071), for attention only: the layer's keys stay of length one without it
    """
    import torch
    if rot < 0 or rot % 2 != 0:
        raise ValueError(f"rot must be even and >= 0 (got {rot})")
    if scaling not in (None, "linear", "base", "by parts"):
        raise ValueError(f"scaling must be None, 'linear', 'base' or 'by parts' (got {scaling!r})")
    if scaling is not None and not factor >= 1.0:
        raise ValueError(f"factor must be >= 1 (got {factor})")
    amplitude = 1.0
    if scaling == "base":
        if rot < 4:
            raise ValueError("scaling 'base' needs at least two pairs")
        base = base * factor ** (rot / (rot - 2))
    i = torch.arange(rot // 2, dtype=torch.float64)
    freq = torch.pow(torch.tensor(float(base), dtype=torch.float64), -2.0 * i / max(rot, 1))
    if scaling == "linear":
        freq = freq / factor
    elif scaling == "by parts":
        if original_length is None:
            raise ValueError("scaling 'by parts' needs original_length")
        if not fast > slow:
            raise ValueError("fast must be above slow")
        turns = original_length * freq / (2 * math.pi)
        kept = ((turns - slow) / (fast - slow)).clamp(0.0, 1.0)
        freq = freq * kept + freq / factor * (1.0 - kept)
        amplitude = 1.0 + 0.1 * math.log(factor)
    return freq.to(torch.float32).to(device) if device is not None else freq.to(torch.float32), amplitude
