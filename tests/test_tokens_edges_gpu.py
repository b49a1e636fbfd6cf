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


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("n,V,chunk", [(5, 60, 9), (1300, 5000, 97), (5, 50021, 997)])
def test_a_product_that_overflows_is_masked(io, n, V, chunk):
    """Logits of -2e38 at an inverse temperature of 2 are -inf: no probability, no place among the top, logprob -inf as a
    target and no gradient there.  Even rows hold ordinary logits besides, odd ones logits of about -1.6e38, whose z are
    finite (and so far apart that lse is the largest and one p is 1)."""
    c = 2.0
    g = torch.Generator().manual_seed(V)
    x = torch.randn(n, V, generator=g) * 3
    x[1::2] = -1.6e38 + 1e36 * torch.rand(x[1::2].shape, generator=g)
    x[:, ::chunk] = -2e38
    targets = (chunk * torch.randint(0, -(-V // chunk), (n,), generator=g))
    targets[4::5] += 1  # and one that is not masked
    x, targets = x.to(DT[io]).cuda(), targets.cuda()
    with B.Tokens(n, 8, V, io=io) as t:
        out = t.token_logprobs(x, targets, inv_temperature=c, k=8)
        ones = torch.ones(n, device="cuda")
        d = f64(t.token_logprobs_backward(x, targets, out["lse"], None, ones, inv_temperature=c))
        t.last_device_status()
    few = slice(0, 20)
    ref = O.token_logprobs(f64(x[few]), targets[few].cpu().numpy(), c, 8)
    hit = np.arange(n) % 5 != 4
    logprob = f64(out["logprob"])
    assert np.all(np.isneginf(logprob[hit])) and np.all(np.isfinite(logprob[~hit]))
    assert np.all(np.isneginf(ref["logprob"][hit[few]]))
    for key in ("lse", "entropy", "top_logprob"):
        got = f64(out[key][few])
        assert np.all(np.abs(got - ref[key]) <= 1e-5 * (1 + np.abs(ref[key]))), key
    assert np.all(f64(x)[np.arange(n)[:, None], out["top_ids"].cpu().numpy()] > -2e38)
    masked = f64(x) * c < -np.finfo(np.float32).max
    assert masked.sum() == n * -(-V // chunk) and np.all(d[masked] == 0)
    # the rest: p within 2^-24 (|z| + |lse|) of itself and the roundings of a few operations and of the output
    rows = np.arange(0, min(n, 20), 2)
    want = O.token_logprobs_backward(f64(x[rows]), targets[rows].cpu().numpy(), c, ref["lse"][rows], ref["entropy"][rows], np.ones(rows.size), None)
    assert np.all(np.abs(d[rows] - want) <= 1e-4 * np.abs(want) + half_ulp(io, want) * 1.001 + 1e-6)


def test_inverse_temperatures_that_the_sums_cannot_take_are_refused():
    """Beyond 2^126 the scale of the exponentials overflows; below 2^-60 a mask written as the lowest value would not be far
    enough below the other logits.  At the limits the results are those of the formula."""
    x = torch.tensor([[1.0, 1.0, 0.5, torch.finfo(torch.float32).min], [0.0, -2.0 ** 60, -2.0 ** 61, torch.finfo(torch.float32).min]], device="cuda")
    ids = torch.tensor([0, 1], device="cuda")
    with B.Tokens(2, 8, 4, io="f32") as t:
        lse = torch.zeros(2, device="cuda")
        for c in (2.0 ** -61, 1e-40, 2.0 ** 127, 3e38):
            for call in (lambda: t.token_logprobs(x, ids, inv_temperature=c),
                         lambda: t.token_logprobs_backward(x, ids, lse, None, lse, inv_temperature=c)):
                with pytest.raises(B.PrismError) as ei:
                    call()
                assert ei.value.status == B.PRISM_ERR_INVALID_ARG
        out = t.token_logprobs(x[:1].contiguous(), ids[:1], inv_temperature=2.0 ** 126, k=4)
        assert out["top_ids"].tolist() == [[0, 1, 2, -1]]
        assert abs(out["logprob"].item() + np.log(2)) < 1e-6 and abs(out["entropy"].item() - np.log(2)) < 1e-6
        out = t.token_logprobs(x[1:].contiguous(), ids[1:], inv_temperature=2.0 ** -60, k=4)
        z = torch.tensor([0.0, -1.0, -2.0], dtype=torch.float64)
        assert abs(out["lse"].item() - torch.logsumexp(z, 0).item()) < 1e-6 and out["top_ids"].tolist() == [[0, 1, 2, -1]]


@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_gradient_of_padded_logits_takes_their_layout(io):
    """Rows of an odd vocabulary in padded logits: rows of the gradient that the call allocates lie as far from a
    16-byte boundary, so that both go in 16-byte units; contiguous logits give a contiguous gradient."""
    n, V, pad = 6, 5001, 7
    g = torch.Generator().manual_seed(0)
    full = torch.randn(n, V + pad, generator=g).to(DT[io]).cuda()
    targets, dlp = torch.randint(0, V, (n,), generator=g).cuda(), torch.randn(n, generator=g).cuda()
    with B.Tokens(n, 8, V, io=io) as t:
        lse = t.token_logprobs(full[:, :V])["lse"]
        got = t.token_logprobs_backward(full[:, :V], targets, lse, None, dlp)
        dense = full[:, :V].contiguous()
        ref = t.token_logprobs_backward(dense, targets, lse, None, dlp)
    assert got.shape == (n, V) and got.stride(1) == 1 and (V + pad - got.stride(0)) * got.element_size() % 16 == 0 and ref.is_contiguous()
    assert torch.equal(got, ref)


def test_tables_of_one_row_or_one_column():
    """A contiguous table whose axis of one element has any stride."""
    ids = torch.tensor([0, -1, 0], device="cuda")
    row = torch.randn(24, device="cuda").as_strided((1, 24), (1, 1))
    with B.Tokens(3, 24, 1, io="f32") as t:
        assert torch.equal(t.embed(ids, row)[::2], row.expand(2, 24))
    column = torch.randn(1, 9, device="cuda").t()
    ids = torch.tensor([8, -1, 3], device="cuda")
    with B.Tokens(3, 1, 9, io="f32") as t:
        assert torch.equal(t.embed(ids, column)[::2], column[[8, 3]])
