"""Properties of the token operators that their other tests leave open: the nearest 8-bit value, infinite scales, an
expired wait where CTAs share a tile, handles on streams of their own, gradients added onto a large table, and the served
example's 8-bit head."""
import importlib.util
import os

import numpy as np
import pytest
import torch

from oracle import prism_tokens as O
from ssm_sequence_layer_gb300 import binding as B
from ssm_sequence_layer_gb300 import build

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
u = 2.0 ** -24
EXAMPLE = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "next_item.py")


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


@pytest.mark.parametrize("rows", [3, 16, 40, 140])
@pytest.mark.parametrize("K", [256, 1664])
def test_product_of_infinite_scales(rows, K):
    """A block whose scale is infinite adds infinities with the sign of its sum, and blocks of opposite signs give NaN."""
    N = 300
    g = torch.Generator().manual_seed(rows + K)
    kb, nb = K // 128, 3
    a8, w8 = ((torch.randn(r, K, generator=g) * 60).clamp_(-448, 448).to(torch.float8_e4m3fn) for r in (rows, N))
    sa, sw = torch.rand(rows, kb, generator=g) + 0.1, torch.rand(nb, kb, generator=g) + 0.1
    sa[1, 0] = float("inf")
    sw[2, 1] = float("inf")
    sa[2, kb - 1] = float("nan")
    with B.Tokens(rows, 64, 64, io="f32") as t:
        got = f64(t.matmul8(a8.cuda(), sa.cuda(), w8.cuda(), sw.cuda()))
        t.last_device_status()
    col = np.arange(N) // 128
    a, w = f64(a8).reshape(rows, kb, 128), f64(w8).reshape(N, kb, 128)
    with np.errstate(invalid="ignore"):
        parts = np.einsum("mbk,nbk->mnb", a, w) * f64(sa)[:, None, :] * f64(sw)[col][None]
        ref = parts.sum(2)
    assert np.isposinf(ref).any() and np.isneginf(ref).any() and np.isnan(ref[2]).all() and np.isnan(ref[1]).any()
    assert np.array_equal(np.isnan(got), np.isnan(ref)) and np.array_equal(np.isinf(got), np.isinf(ref))
    assert np.array_equal(got[np.isinf(ref)], ref[np.isinf(ref)])
    ok = np.isfinite(ref)
    size = np.einsum("mbk,nbk->mnb", np.abs(a), np.abs(w)) * f64(sa)[:, None, :] * f64(sw)[col][None]
    assert np.all(np.abs(got[ok] - ref[ok]) <= (2 * 128 + kb + 5) * u * size.sum(2)[ok])


@pytest.mark.parametrize("M,N,K", [(128, 4096, 4096), (64, 1024, 16384)])
def test_an_expired_wait_of_ctas_that_share_a_tile(M, N, K):
    """With a bound of 1 ns the waits of a cluster's CTAs run out: the status says so and the handle works again after it."""
    g = torch.Generator().manual_seed(0)
    a8, w8 = (torch.randn(r, K, generator=g).to(torch.float8_e4m3fn).cuda() for r in (M, N))
    sa, sw = torch.ones(M, K // 128, device="cuda"), torch.ones(N // 128, K // 128, device="cuda")
    with B.Tokens(M, 64, 64, io="f32") as t:
        ref = t.matmul8(a8, sa, w8, sw)
        torch.empty(1 << 28, device="cuda").zero_()  # operands out of L2, so that loads take longer than the bound
        t.set_option(B.PRISM_OPT_WAIT_NS, 1)
        t.matmul8(a8, sa, w8, sw)
        torch.cuda.synchronize()
        with pytest.raises(B.PrismError) as ei:
            t.last_device_status()
        assert ei.value.status == B.PRISM_ERR_TIMEOUT
        t.set_option(B.PRISM_OPT_WAIT_NS, 0)
        assert torch.equal(t.matmul8(a8, sa, w8, sw), ref)
        t.last_device_status()


def test_two_handles_on_two_streams():
    """Handles share nothing: the workspaces' users of two streams do not disturb each other."""
    n, D, V = 6000, 260, 9000
    g = torch.Generator().manual_seed(4)
    sets = []
    for i in range(2):
        ids = torch.randint(-1, V >> (3 * i), (n,), generator=g).cuda()
        rows, w = torch.randn(n, D, generator=g).cuda(), torch.randn(D, generator=g).cuda()
        sets.append((ids, rows, w))
    streams = [torch.cuda.Stream() for _ in sets]
    with B.Tokens(n, D, V, io="f32") as a, B.Tokens(n, D, V, io="f32") as b:
        def work(t, s, ids, rows, w):
            out = []
            for _ in range(6):
                out.append(t.embed_backward(ids, rows, stream=s))
                out += t.norm_backward(rows, w, rows, stream=s).values()
            return out

        alone = [[x.clone() for x in work(t, None, *v)] for t, v in zip((a, b), sets)]
        torch.cuda.synchronize()
        both = [[], []]
        for _ in range(3):
            for i, t in enumerate((a, b)):
                both[i] = work(t, streams[i], *sets[i])
        torch.cuda.synchronize()
        for x, y in zip(alone[0] + alone[1], both[0] + both[1]):
            assert torch.equal(x, y)
        a.last_device_status()
        b.last_device_status()


@pytest.mark.parametrize("n", [300, 6000, 70000])
def test_gradient_added_onto_a_large_vocabulary(n):
    """Ids of 28 bits onto a table of ones: rows without a token keep their bits, the others get the sum added once."""
    V = 1 << 28
    g = torch.Generator().manual_seed(n)
    ids = torch.randint(0, V, (n,), generator=g)
    ids[: n // 2] = V - 1 - torch.randint(0, 50, (n // 2,), generator=g)
    dout = torch.randn(n, 1, generator=g)
    with B.Tokens(n, 1, V, io="f32") as t:
        d = torch.ones(V, 1, device="cuda")
        t.embed_backward(ids.cuda(), dout.cuda(), scale=0.5, dtable=d, accumulate=True)
        torch.cuda.synchronize()
        t.last_device_status()
    rows, inverse = torch.unique(ids, return_inverse=True)
    ref = torch.ones(rows.numel(), dtype=torch.float64).index_add_(0, inverse, 0.5 * dout[:, 0].double())
    size = torch.ones(rows.numel(), dtype=torch.float64).index_add_(0, inverse, 0.5 * dout[:, 0].double().abs())
    count = torch.bincount(inverse)
    assert torch.all((d[rows.cuda(), 0].cpu().double() - ref).abs() <= u * (count + 3) * size)
    d[rows.cuda()] = 1.0
    assert torch.all(d == 1.0)


def test_served_8bit_head_is_near_the_wide_one():
    """An e4m3 value errs by 2^-4 / sqrt(3) * 0.71 = 0.026 of itself in the mean square, a product of two by 0.036, without a
    direction over D products: a logit by 0.036 rms(y) |w|, where y's mean square is that of the norm's weight.  A log
    probability takes the target's logit and a mean of others: twice that, six times over for the largest of all."""
    spec = importlib.util.spec_from_file_location("next_item_served", EXAMPLE)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    model = m.Model().cuda()
    _, follows = m.train(model, 20)
    _, _, alternatives, reference = m.serve(model, follows)
    with torch.no_grad():
        rms, longest = model.w_out.square().mean().sqrt().item(), model.table.norm(dim=1).max().item()
    assert (alternatives - reference).abs().max().item() <= 12 * 0.036 * rms * longest
