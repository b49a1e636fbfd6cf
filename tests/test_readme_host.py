"""The README's form of the heads gives the layer keys of length one."""
import os
import re

import numpy as np

from oracle import prism_block as O
from ssm_sequence_layer_gb300.rotary import rotary_frequencies


def test_the_readme_form_keeps_keys_of_length_one():
    with open(os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "README.md")) as f:
        text = f.read()
    lines = re.findall(r"^(?:inv_freq, .*|form = dict\(.*)$", text, re.M)
    assert len(lines) == 2
    T = 5
    names = {"rotary_frequencies": rotary_frequencies, "positions": np.arange(T)[None] * 1000}
    exec("\n".join(lines).replace('"cuda"', '"cpu"'), names)
    form = names["form"]
    Hq, Hk, Hv = form["heads"]
    x = np.random.default_rng(0).normal(size=(1, T, (Hq + Hk + Hv) * form["d"]))
    k = O.heads(x, form["heads"], form["d"], form["d"], form["norm"], 1e-6, None, None, form["inv_freq"].double().numpy(), form.get("interleaved", False),
                form.get("amplitude", 1.0), form["positions"])[1]
    assert np.all(np.abs(np.linalg.norm(k, axis=-1) - 1) < 1e-6)
