"""The norm with the residual's addition, its 8-bit output and its gradient, against the fp64 oracle.

Tolerances, with u = 2^-24 (fp32) and h = half a unit in the last place of the io type:
  sum      one fp32 addition and one rounding: u |r| + h.
  y        the mean square carries at most D/32 + 8 roundings of positive terms (a lane's share of the
           row, then the join), the root halves them; then the root, two products and the rounding of r:
           (D/64 + 12) u |y| + h.
  y_scale  (D/64 + 14) u relative: y's error and one division.
  y8       half a step of e4m3 at the largest |y| / s, plus y's error: |y8 s - y| <= 2^-4 |y| + 2^-10 s
           (a normal value is within 2^-4 of itself, a subnormal one within half of 2^-9), plus the same share of
           y's error and the scale's.
  dx       each of the two terms within (D/32 + 24) u of its magnitude; the mean's terms may cancel, so
           its magnitude is q |rh| mean |w dy rh|; plus u |dx| and h.
  dweight  a sum of n terms: (n + D/64 + 16) u sum |dy rh|."""
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


@pytest.fixture(scope="module", autouse=True)
def _built():
    build.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"


def half_ulp(io, x):
    return bf16_half_ulp(x) if io == "bf16" else u * np.abs(x)


def draw(n, D, io, seed, spread=1.0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(n, D, generator=g).to(DT[io])
    res = (torch.randn(n, D, generator=g) * 2 * torch.exp(torch.randn(D, generator=g) * spread)).to(DT[io])
    w = (1 + 0.2 * torch.randn(D, generator=g)).to(DT[io])
    return x, res, w


def f64(t):
    return t.float().cpu().double().numpy()


SHAPES = [(1, 64), (16, 768), (5, 1), (7, 129), (33, 256), (3, 1000), (130, 1024), (9, 1032), (4, 2056), (3, 4096), (2, 5000),
          (2, 16384), (1, 20001), (1, 65536)]


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("n,D", SHAPES)
@pytest.mark.parametrize("residual", [True, False])
def test_norm(io, n, D, residual):
    x, res, w = draw(n, D, io, n + D)
    with B.Tokens(n, D, 8, io=io) as t:
        out = t.norm(x.cuda(), w.cuda(), residual=res.cuda() if residual else None, eps=EPS, want=("sum", "y", "y8"))
        only = t.norm(x.cuda(), w.cuda(), residual=res.cuda() if residual else None, eps=EPS, want=("y8",))
        torch.cuda.synchronize()
        t.last_device_status()
    r, y, scale = O.norm(f64(x), f64(res) if residual else None, f64(w), EPS)
    assert np.all(np.abs(f64(out["sum"]) - r) <= u * np.abs(r) + half_ulp(io, r) * 1.0001)
    ey = (D / 64 + 12) * u * np.abs(y)
    assert np.all(np.abs(f64(out["y"]) - y) <= ey + half_ulp(io, np.abs(y) + ey))
    got = f64(out["y_scale"])
    assert np.all(np.abs(got - scale) <= (D / 64 + 14) * u * scale + 2.0 ** -149)
    s = got[:, O.blocks_of(D)]
    slack = 1.0 + 2.0 ** -3
    assert np.all(np.abs(f64(out["y8"]) * s - y) <= 2.0 ** -4 * np.abs(y) * 1.0001 + 2.0 ** -10 * s * 1.0001 + slack * (ey + (D / 64 + 14) * u * np.abs(y)))
    assert torch.equal(only["y8"].view(torch.uint8), out["y8"].view(torch.uint8)) and torch.equal(only["y_scale"], out["y_scale"])


def test_norm_8bit_rounding_is_the_nearest():
    """y8 is the e4m3 value nearest to y / y_scale: where the quotient is not within fp32 noise of the
    middle between two neighbours, it equals the oracle's rounding."""
    x, res, w = draw(64, 768, "f32", 3)
    with B.Tokens(64, 768, 8, io="f32") as t:
        out = t.norm(x.cuda(), w.cuda(), residual=res.cuda(), eps=EPS, want=("y", "y8"))
    quotient = f64(out["y"]) / f64(out["y_scale"])[:, O.blocks_of(768)]
    lo, hi = O.e4m3(quotient * (1 - 2.0 ** -20)), O.e4m3(quotient * (1 + 2.0 ** -20))
    clear = lo == hi
    assert clear.mean() > 0.999
    assert np.array_equal(f64(out["y8"])[clear], lo[clear])


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("D", [768, 200])
def test_norm_in_place(io, D):
    """sum may take the residual's place and y the place of x."""
    x, res, w = (a.cuda() for a in draw(21, D, io, 5))
    with B.Tokens(21, D, 8, io=io) as t:
        ref = t.norm(x, w, residual=res, want=("sum", "y", "y8"))
        x2, res2 = x.clone(), res.clone()
        got = t.norm(x2, w, residual=res2, out={"sum": res2, "y": x2, "y8": torch.empty_like(ref["y8"]),
                                                "y_scale": torch.empty_like(ref["y_scale"])})
        torch.cuda.synchronize()
    for k in ref:
        assert torch.equal(ref[k].view(torch.uint8), got[k].view(torch.uint8)), k


@pytest.mark.parametrize("D", [768, 131])
def test_norm_of_special_rows(D):
    x = torch.randn(5, D)
    x[0] = 0.0
    x[1, 3] = float("nan")
    x[2] *= 1e-25          # squares vanish in fp32: y = r / sqrt(eps)
    x[3, 0:128] = 0.0      # a block of zeros
    x[4, 5] = float("inf")
    w = torch.ones(D)
    with B.Tokens(5, D, 8, io="f32") as t:
        out = {k: v.cpu() for k, v in t.norm(x.cuda(), w.cuda(), eps=EPS, want=("y", "y8")).items()}
    assert torch.all(out["y"][0] == 0) and torch.all(out["y8"][0].float() == 0)
    assert torch.all(out["y_scale"][0] == 2.0 ** -126)
    assert torch.all(torch.isnan(out["y"][1])) and torch.all(torch.isnan(out["y8"][1].float()))
    ref = x[2].double() / EPS ** 0.5
    assert torch.all((out["y"][2].double() - ref).abs() <= 1e-6 * ref.abs())
    assert out["y_scale"][3, 0] == 2.0 ** -126 and torch.all(out["y8"][3, :128].float() == 0)
    assert torch.isnan(out["y"][4, 5]) and torch.all(out["y"][4, :5] == 0)  # inf / inf, finite / inf


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("n,D", SHAPES + [(700, 768), (2500, 96), (1999, 250)])
@pytest.mark.parametrize("stream", [True, False])
def test_norm_backward(io, n, D, stream):
    _, r, w = draw(n, D, io, 7 * n + D, spread=0.5)
    g = torch.Generator().manual_seed(n)
    dy = torch.randn(n, D, generator=g).to(DT[io])
    ds = torch.randn(n, D, generator=g).to(DT[io]) if stream else None
    with B.Tokens(n, D, 8, io=io) as t:
        got = t.norm_backward(r.cuda(), w.cuda(), dy.cuda(), dsum=None if ds is None else ds.cuda(), eps=EPS)
        again = dy.cuda().clone()
        inplace = t.norm_backward(r.cuda(), w.cuda(), again, dsum=None if ds is None else ds.cuda(), eps=EPS,
                                  out={"dx": again, "dweight": torch.empty(D, device="cuda")})
        torch.cuda.synchronize()
    assert torch.equal(got["dx"], inplace["dx"]) and torch.equal(got["dweight"], inplace["dweight"])
    r64, w64, dy64 = f64(r), f64(w), f64(dy)
    dx, dw = O.norm_backward(r64, w64, EPS, dy64, None if ds is None else f64(ds))
    q = 1 / np.sqrt(np.mean(r64 ** 2, axis=1, keepdims=True) + EPS)
    size = q * (np.abs(w64 * dy64) + np.abs(r64 * q) * np.mean(np.abs(w64 * dy64 * r64 * q), axis=1, keepdims=True))
    e = (D / 32 + 24) * u * size + u * np.abs(dx)
    assert np.all(np.abs(f64(got["dx"]) - dx) <= e + half_ulp(io, np.abs(dx) + e))
    assert np.all(np.abs(f64(got["dweight"]) - dw) <= (n + D / 64 + 16) * u * np.sum(np.abs(dy64 * r64 * q), axis=0))


def test_norm_gradient_against_differences():
    """Central differences of the oracle's loss <y, c> + <sum, d> along random directions."""
    n, D = 6, 40
    x, res, w = draw(n, D, "f32", 11, spread=0.3)
    g = torch.Generator().manual_seed(2)
    c, d = torch.randn(n, D, generator=g), torch.randn(n, D, generator=g)
    with B.Tokens(n, D, 8, io="f32") as t:
        s = t.norm(x.cuda(), w.cuda(), residual=res.cuda(), eps=EPS, want=("sum", "y"))["sum"]
        got = t.norm_backward(s, w.cuda(), c.cuda(), dsum=d.cuda(), eps=EPS)

    def loss(a, b, v):
        r, y, _ = O.norm(a, b, v, EPS)
        return np.sum(y * f64(c)) + np.sum(r * f64(d))

    for seed in range(4):
        rng = np.random.RandomState(seed)
        va, vw, h = rng.randn(n, D), rng.randn(D), 1e-5
        for which, slope in ((0, np.sum(f64(got["dx"]) * va)), (1, np.sum(f64(got["dx"]) * va)), (2, np.sum(f64(got["dweight"]) * vw))):
            args = [f64(x), f64(res), f64(w)]
            step = vw if which == 2 else va
            up, down = list(args), list(args)
            up[which], down[which] = args[which] + h * step, args[which] - h * step
            diff = (loss(*up) - loss(*down)) / (2 * h)
            assert abs(diff - slope) <= 1e-5 * (1 + abs(diff)) * np.sqrt(n * D)


def test_norm_of_no_rows():
    with B.Tokens(3, 16, 8, io="f32") as t:
        e, w = torch.empty(0, 16, device="cuda"), torch.ones(16, device="cuda")
        assert t.norm(e, w)["y"].shape == (0, 16)
        assert torch.all(t.norm_backward(e, w, e)["dweight"] == 0)


def test_norm_refusals():
    with B.Tokens(4, 16, 9, io="bf16") as t:
        x = torch.zeros(4, 16, dtype=torch.bfloat16, device="cuda")
        w = torch.zeros(16, dtype=torch.bfloat16, device="cuda")
        for bad in (lambda: t.norm(x.float(), w), lambda: t.norm(x, w[:8]), lambda: t.norm(x, w, residual=x[:3]), lambda: t.norm(x.t(), w),
                    lambda: t.norm(x, w, want=("z",)), lambda: t.norm_backward(x, w, x[:2]), lambda: t.norm(x.cpu(), w)):
            with pytest.raises(ValueError):
                bad()
        for status, bad in (
                (B.PRISM_ERR_INVALID_ARG, lambda: t.norm(torch.zeros(5, 16, dtype=torch.bfloat16, device="cuda"), w)),
                (B.PRISM_ERR_INVALID_ARG, lambda: t.norm(x, w, eps=-1.0)),
                (B.PRISM_ERR_INVALID_ARG, lambda: t.norm(x, w, eps=float("nan"))),
                (B.PRISM_ERR_INVALID_ARG, lambda: B.prism_norm(t.handle, 4, x, None, w, EPS, x, None, None, None)),
                (B.PRISM_ERR_INVALID_ARG, lambda: B.prism_norm(t.handle, 4, x, None, w, EPS, None, None, x, None)),
                (B.PRISM_ERR_MISALIGNED, lambda: B.prism_norm(t.handle, 4, x.data_ptr() + 8, None, w, EPS, None, x, None, None)),
                (B.PRISM_ERR_INVALID_ARG, lambda: B.prism_norm_backward(t.handle, 4, x, w, EPS, None, None, x, w.data_ptr()))):
            with pytest.raises(B.PrismError) as ei:
                bad()
            assert ei.value.status == status
