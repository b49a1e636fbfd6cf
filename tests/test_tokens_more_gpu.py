"""Properties of the token operators that their other tests leave open: the nearest 8-bit value."""
import numpy as np
import pytest
import torch

from oracle import prism_tokens as O
from ssm_sequence_layer_gb300 import binding as B
from ssm_sequence_layer_gb300 import build

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
u = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def _built():
    build.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"


def f64(t):
    return t.float().cpu().double().numpy()


@pytest.mark.parametrize("D", [768, 765])
def test_norm_8bit_values_are_the_nearest(D):
    """Of 12.6 million values, how many are not the e4m3 value nearest to y / scale = 448 v / max |v|, v = r w: in 64 bits
    this order has exact products and a quotient that is exact in the middle between two neighbours, where some hundred of
    these values lie (and where 1 / rms, rounded, would decide).  Left are two roundings
    of fp32, of the block's scale and of the quotient, each with a mean magnitude of 0.35 u relative to its value.  There are 8
    middles between neighbours in an octave, 8 / ln 2 per unit of the logarithm, and a quotient rounded onto a middle
    goes the wrong way half of the time: 12.6e6 * 11.5 * 0.7 u = 6 values, and 20 are beyond five times their spread.
    Without the product's rounding error and the corrected quotient it is about 70."""
    n = 16384
    g = torch.Generator().manual_seed(D)
    x = torch.randn(n, D, generator=g).bfloat16()
    res = (2 * torch.randn(n, D, generator=g) * torch.exp(0.7 * torch.randn(D, generator=g))).bfloat16()
    w = (1 + 0.2 * torch.randn(D, generator=g)).bfloat16()
    with B.Tokens(n, D, 8, io="bf16") as t:
        got = f64(t.norm(x.cuda(), w.cuda(), residual=res.cuda(), want=("y8",))["y8"])
    v = (f64(x) + f64(res)) * f64(w)
    peak = np.stack([np.abs(v[:, b:b + 128]).max(axis=1) for b in range(0, D, 128)], axis=1)[:, O.blocks_of(D)]
    assert np.count_nonzero(got != O.e4m3(448 * v / peak)) <= 20


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("size", [1.0, 1e-29, 2e-33, 1e-36, 3e33])
def test_weights_are_those_of_a_division(io, size):
    """w8 is the e4m3 value of the fp32 quotient W / w_scale: the reciprocal's product, corrected once by the remainder,
    errs from the exact quotient by less than 2^-46 of it before its only rounding.  That is another fp32 number than the division's
    for one quotient in 2^21, and another e4m3 value only if one of the two is a middle between e4m3 values besides (8 of
    the 2^23 fp32 numbers of an octave): none of the values here."""
    N, K = 300, 784
    g = torch.Generator().manual_seed(7)
    W = (torch.randn(N, K, generator=g).double() * torch.exp(torch.randn(N, 1, generator=g)).double() * size).to(DT[io])
    W[128:256, 128:256] = 0.0
    W[128, 128:132] = torch.tensor([448.0, 17.0, 1.0625, 0.001953125 * 1.5], dtype=torch.float64).mul(size).to(DT[io])
    with B.Tokens(1, 64, 64, io=io) as t:
        w8, scale = (a.cpu() for a in t.matmul8_weights(W.cuda()))
    each = scale.repeat_interleave(128, 0)[:N].repeat_interleave(128, 1)[:, :K]
    assert torch.equal(w8.float(), (W.float() / each).clamp(-448, 448).to(torch.float8_e4m3fn).float())
