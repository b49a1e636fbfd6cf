"""Token operators where a value leaves the range of float32 on its way, and other edges of their contract, against
the fp64 oracle.  Tolerances are those of the operators' own tests; beside them, values below the smallest normal
float32 lie on a grid of 2^-149 (of bfloat16: 2^-133), so that a rounding there costs half a step of the grid."""
import numpy as np
import pytest
import torch

from oracle import prism_tokens as O
from ssm_sequence_layer_gb300 import binding as B
from ssm_sequence_layer_gb300 import build
from tests.gpu_util import bf16_half_ulp

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
u = 2.0 ** -24
EPS = 1e-6
GRID = 2.0 ** -149


@pytest.fixture(scope="module", autouse=True)
def _built():
    build.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"


def f64(t):
    return t.float().cpu().double().numpy()


def half_ulp(io, x):
    return np.maximum(bf16_half_ulp(x), 2.0 ** -134) if io == "bf16" else u * np.abs(x) + GRID / 2


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("D", [768, 517, 9000])
def test_norm_where_row_times_weight_leaves_the_range(io, D):
    """Rows and blocks of weights so small or so large that r w underflows or overflows while y is an ordinary number, or
    nearly so: the norm as at any other size, and no NaN in its 8 bits.  The first block's weights are ordinary, so that
    rows of 1e-36 and 1e-37 meet them too."""
    size = torch.tensor([1.0, 1e15, 1e-12, 1e-30, 1e-36, 1e-37, 3e-38, 1e-40, 0.0])
    g = torch.Generator().manual_seed(D)
    x = (torch.randn(size.numel(), D, generator=g).double() * size[:, None].double()).to(DT[io])
    w = 1 + 0.2 * torch.randn(D, generator=g).double()
    for block, times in enumerate((1.0, 1e-37, 1e-20, 1e25, 0.0)):
        w[128 * block:128 * block + 128] *= times
    w = w.to(DT[io])
    with B.Tokens(size.numel(), D, 8, io=io) as t:
        out = t.norm(x.cuda(), w.cuda(), eps=EPS, want=("sum", "y", "y8"))
        torch.cuda.synchronize()
        t.last_device_status()
    r, y, scale = O.norm(f64(x), None, f64(w), EPS)
    assert np.array_equal(f64(out["sum"]), r)
    ey = (D / 64 + 12) * u * np.abs(y) + GRID
    assert np.all(np.abs(f64(out["y"]) - y) <= ey + half_ulp(io, np.abs(y) + ey))
    got = f64(out["y_scale"])
    assert np.all(np.abs(got - scale) <= (D / 64 + 14) * u * scale + GRID)
    s = got[:, O.blocks_of(D)]
    error = np.abs(f64(out["y8"]) * s - y)
    assert np.all(error <= 2.0 ** -4 * np.abs(y) * 1.0001 + 2.0 ** -10 * s * 1.0001 + 1.125 * (ey + (D / 64 + 14) * u * np.abs(y)))
