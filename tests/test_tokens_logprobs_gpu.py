"""Log probabilities, entropy, top alternatives and their gradient, against the fp64 oracle.

Tolerances, with u = 2^-24 and zmax = max |z| over a row's finite z:
  z          one product: u |z|.
  exp        2 u for the function and 2 u |d| for its argument d = z - m, so a term exp(d) is within
             (2 + 4 |d|) u of itself; |d| exp(d) < 1, so the sum is within (6 + A) u of itself relatively, with A additions
             in a chain (a thread's share of the row and the joins: at most V/512 + 64) and the joins'
             factors (another 8 u each, at most 24 of them).
  lse        u (2 zmax) + that relative error of the sum + u |lse|:  E = u (3 zmax + V/512 + 300).
  logprob, top_logprob   E + u (2 |z| + |result|).
  entropy    terms p |log p| with the same relative errors, and p and log p each within E:
             2 E (1 + H).
  dlogits    p within E + (4 |log p| + 4) u of itself, the entropy's factor within 2 E (1 + H) + E;
             the result one rounding of the io type more."""
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
INF = float("inf")


@pytest.fixture(scope="module", autouse=True)
def _built():
    build.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"


def f64(t):
    return t.float().cpu().double().numpy()


def draw(n, V, io, seed, pad=0, masked=0.0, std=3.0):
    g = torch.Generator().manual_seed(seed)
    full = (torch.randn(n, V + pad, generator=g) * std).to(DT[io])
    full[torch.rand(n, V + pad, generator=g) < masked] = -INF
    targets = torch.randint(0, V, (n,), generator=g)
    targets[torch.rand(n, generator=g) < 0.2] = -1
    return full.cuda()[:, :V], targets.cuda()


def bound(logits, c, V):
    z = np.abs(c * np.where(np.isfinite(logits) & (logits > O.LOWEST * (1 - 1e-9)), logits, 0.0))
    return u * (3 * z.max(axis=1, initial=0.0) + V / 512 + 300)


def same(got, ref, tol):
    """Equal infinities and NaN, and finite values within tol."""
    ok = np.isfinite(ref)
    assert np.array_equal(np.isnan(got), np.isnan(ref))
    inf = ~ok & ~np.isnan(ref)
    assert np.array_equal(got[inf], ref[inf])
    assert np.all(np.abs(got - ref)[ok] <= np.broadcast_to(tol, ref.shape)[ok])


def check_forward(out, x, targets, c, k):
    V = x.shape[1]
    ref = O.token_logprobs(x, targets, c, k)
    E = bound(x, c, V)
    with np.errstate(invalid="ignore"):
        same(f64(out["lse"]), ref["lse"], E)
        same(f64(out["entropy"]), ref["entropy"], 2 * E * (1 + np.nan_to_num(ref["entropy"])))
        if targets is not None:
            t = np.take_along_axis(x, np.clip(targets, 0, V - 1)[:, None], 1)[:, 0] * c
            same(f64(out["logprob"]), ref["logprob"], E + u * (2 * np.abs(t) + np.abs(ref["logprob"])))
        if k:
            assert np.array_equal(out["top_ids"].cpu().numpy(), ref["top_ids"])
            top = ref["top_logprob"]
            same(f64(out["top_logprob"]), top, E[:, None] + u * (3 * np.abs(top) + 2 * np.abs(ref["lse"])[:, None]))


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("n,V,pad,k,masked,c", [
    (1, 1, 0, 1, 0, 1.0), (3, 2, 0, 32, 0, 0.7), (5, 33, 0, 5, 0.3, 1.3), (7, 100, 3, 32, 0.9, 1.0), (4, 1000, 0, 8, 0, 1.0),
    (300, 511, 1, 3, 0.1, 1.0), (16, 4099, 0, 20, 0.2, 2.0), (3, 50021, 27, 20, 0.1, 1.25), (2, 131072, 0, 32, 0, 1.0),
    (1, 300007, 0, 8, 0, 1.0), (640, 20000, 0, 4, 0, 1.0), (2, 262144, 5, 0, 0, 1.0), (400, 8193, 0, 0, 0.5, 1.0),
    (2, 700001, 0, 16, 0, 1.0), (143, 415, 0, 32, 0, 1.0), (55, 5381, 64, 32, 0, 1.0), (14, 5112, 3, 32, 0.4, 1.0), (9, 260, 0, 32, 0.5, 1.0),
    (1300, 1001, 0, 32, 0.2, 1.0), (1300, 7999, 2, 5, 0, 0.8), (2000, 515, 0, 0, 0.9, 1.0)])
def test_token_logprobs(io, n, V, pad, k, masked, c):
    x, targets = draw(n, V, io, n + V, pad, masked)
    with B.Tokens(n, 8, V, io=io) as t:
        out = t.token_logprobs(x, targets, inv_temperature=c, k=k)
        bare = t.token_logprobs(x, inv_temperature=c)
        again = t.token_logprobs(x, targets, inv_temperature=c, k=k)
        torch.cuda.synchronize()
        t.last_device_status()
    assert sorted(bare) == ["entropy", "lse"]
    for key in out:
        assert torch.equal(out[key], again[key]), "equal inputs give equal bits"
    check_forward(out, f64(x), targets.cpu().numpy(), float(np.float32(c)), k)


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("V", [40, 5000, 50021])
@pytest.mark.parametrize("kind", ["equal", "falling", "rising", "steps", "few", "block", "lowest", "zeros"])
def test_top_of_ordered_rows(io, V, kind):
    """Rows whose order defeats a selection by samples: ties (lowest id first), runs, few live tokens."""
    at = torch.arange(V)
    row = {"equal": torch.full((V,), 1.5), "falling": -0.01 * at, "rising": 0.01 * at, "steps": (at % 7).float(),
           "few": torch.where(at % 997 == 5, 2.0 + 0.0 * at, torch.full((V,), -INF)),
           "block": torch.where((at >= V // 2) & (at < V // 2 + 37), at * 0.001, torch.full((V,), -INF)),
           "lowest": torch.where(at % 5 == 0, at * 0.001, torch.full((V,), torch.finfo(DT[io]).min)),
           "zeros": torch.where(at % 2 == 0, torch.tensor(0.0), torch.tensor(-0.0))}[kind]
    rows = 1300 if V == 5000 else 3  # a warp per row, or a block or cluster per row
    x = row.to(DT[io]).cuda().expand(rows, V).contiguous()
    targets = torch.tensor([0, V - 1, V // 2], device="cuda")
    if rows > 3:
        with B.Tokens(rows, 8, V, io=io) as t:
            many = t.token_logprobs(x, k=32)
            assert torch.equal(many["top_ids"], many["top_ids"][:1].expand(rows, 32))
            check_forward({key: v[:3] for key, v in many.items()}, f64(x[:3]), None, 1.0, 32)
        x = x[:3].contiguous()
    with B.Tokens(3, 8, V, io=io) as t:
        for k in (1, 7, 32):
            out = t.token_logprobs(x, targets, k=k)
            check_forward(out, f64(x), targets.cpu().numpy(), 1.0, k)


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("V", [70, 50021])
def test_rows_without_a_value(io, V):
    x, _ = draw(6, V, io, 1)
    x[0] = -INF
    x[1, 5] = float("nan")
    x[2, V - 1] = INF
    x[3] = torch.finfo(DT[io]).min
    x[4, :] = -INF
    x[4, V // 3] = -2.0
    targets = torch.tensor([1, 1, 1, 1, V // 3, -5], device="cuda")
    with B.Tokens(6, 8, V, io=io) as t:
        out = t.token_logprobs(x, targets, k=4)
        ref = O.token_logprobs(f64(x), targets.cpu().numpy(), 1.0, 4)
        check_forward(out, f64(x), targets.cpu().numpy(), 1.0, 4)
        g = t.token_logprobs_backward(x, targets, out["lse"], out["entropy"], torch.ones(6, device="cuda"), torch.ones(6, device="cuda"))
    assert np.isneginf(ref["lse"][0]) and ref["entropy"][4] == 0
    g = g.float().cpu()
    assert torch.all(g[0] == 0) and torch.all(g[3] == 0) and torch.all(torch.isnan(g[1])) and torch.all(g[4, : V // 3] == 0) and abs(g[4, V // 3]) < 1e-5


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("n,V,pad,masked,c,which", [
    (1, 1, 0, 0, 1.0, "both"), (5, 33, 0, 0.3, 1.3, "both"), (7, 100, 3, 0.9, 1.0, "logprob"), (300, 511, 1, 0.1, 1.0, "both"),
    (16, 4099, 0, 0.2, 2.0, "entropy"), (3, 50021, 27, 0.1, 1.25, "both"), (2, 300007, 0, 0, 1.0, "both"), (700, 2000, 0, 0, 1.0, "logprob")])
def test_token_logprobs_backward(io, n, V, pad, masked, c, which):
    x, targets = draw(n, V, io, 2 * n + V, pad, masked)
    g = torch.Generator().manual_seed(1)
    dlp = torch.randn(n, generator=g).cuda() if which != "entropy" else None
    dh = torch.randn(n, generator=g).cuda() if which != "logprob" else None
    with B.Tokens(n, 8, V, io=io) as t:
        f = t.token_logprobs(x, targets, inv_temperature=c)
        got = t.token_logprobs_backward(x, targets, f["lse"], f["entropy"], dlp, dh, inv_temperature=c)
        shifted = torch.full((n, V + 9), 7.0, dtype=DT[io], device="cuda")  # another row stride than the logits'
        t.token_logprobs_backward(x, targets, f["lse"], f["entropy"], dlp, dh, inv_temperature=c, dlogits=shifted[:, :V])
        copy = x.clone()  # contiguous
        t.token_logprobs_backward(copy, targets, f["lse"], f["entropy"], dlp, dh, inv_temperature=c, dlogits=copy)
        torch.cuda.synchronize()
        t.last_device_status()
    assert torch.equal(got, copy) and torch.equal(got, shifted[:, :V]) and torch.all(shifted[:, V:] == 7.0)
    c = float(np.float32(c))
    x64, t64 = f64(x), targets.cpu().numpy()
    exact = O.token_logprobs(x64, t64, c, 0)
    dlp64, dh64 = (None if a is None else f64(a) for a in (dlp, dh))
    ref = O.token_logprobs_backward(x64, t64, c, exact["lse"], exact["entropy"], dlp64, dh64)
    E = bound(x64, c, V)[:, None]
    with np.errstate(invalid="ignore"):
        lp = c * x64 - exact["lse"][:, None]
        p = np.where(x64 == -np.inf, 0.0, np.exp(lp))
        lp = np.where(x64 == -np.inf, 0.0, lp)
    H = exact["entropy"][:, None]
    rel = E + (4 * np.abs(lp) + 8) * u
    a = 0 if dlp64 is None else np.abs(dlp64)[:, None]
    b = 0 if dh64 is None else np.abs(dh64)[:, None]
    tol = c * (a * (p * rel + 2 * u) + b * p * (rel * (np.abs(lp) + H) + 3 * E * (1 + H) + 8 * u)) + 2.0 ** -126
    same(f64(got), ref, tol + (bf16_half_ulp(np.abs(ref) + tol) if io == "bf16" else u * np.abs(ref)))


def test_gradient_against_differences():
    """Central differences of the oracle's <logprob, a> + <entropy, b> along random directions."""
    n, V, c = 4, 60, 1.3
    x, targets = draw(n, V, "f32", 8, masked=0.2)
    g = torch.Generator().manual_seed(3)
    a, b = torch.randn(n, generator=g), torch.randn(n, generator=g)
    with B.Tokens(n, 8, V, io="f32") as t:
        f = t.token_logprobs(x, targets, inv_temperature=c)
        got = f64(t.token_logprobs_backward(x, targets, f["lse"], f["entropy"], a.cuda(), b.cuda(), inv_temperature=c))
    t64, x64 = targets.cpu().numpy(), f64(x)
    t64 = np.where(np.isinf(x64[np.arange(n), t64]), -1, t64)  # a masked target has no slope to compare

    def loss(y):
        out = O.token_logprobs(y, t64, float(np.float32(c)), 0)
        return np.sum(out["logprob"] * f64(a)) + np.sum(out["entropy"] * f64(b))

    # the gradient of the rows whose target is masked keeps its softmax part: take those rows out of the direction
    rows = (t64 == targets.cpu().numpy())[:, None]
    for seed in range(4):
        v = np.random.RandomState(seed).randn(n, V) * rows
        h = 1e-5
        diff = (loss(x64 + h * v) - loss(x64 - h * v)) / (2 * h)
        assert abs(diff - np.sum(got * v)) <= 1e-5 * (1 + abs(diff)) * np.sqrt(n * V)


def test_targets_beyond_the_vocabulary_are_recorded():
    x = torch.zeros(2, 9, device="cuda")
    with B.Tokens(2, 8, 9, io="f32") as t:
        out = t.token_logprobs(x, torch.tensor([3, 9], device="cuda"))
        torch.cuda.synchronize()
        with pytest.raises(B.PrismError) as ei:
            t.last_device_status()
        assert ei.value.status == B.PRISM_ERR_DEVICE and out["logprob"][1] == 0
        t.token_logprobs_backward(x, torch.tensor([3, 9], device="cuda"), out["lse"], None, torch.ones(2, device="cuda"))
        torch.cuda.synchronize()
        with pytest.raises(B.PrismError):
            t.last_device_status()


def test_logits_type_is_an_option_and_streams():
    x, targets = draw(5, 3000, "f32", 4)
    s = torch.cuda.Stream()
    with B.Tokens(5, 8, 3000, io="bf16", logits="f32") as t:
        ref = t.token_logprobs(x, targets, k=3)
        torch.cuda.synchronize()
        with torch.cuda.stream(s):
            got = t.token_logprobs(x, targets, k=3)
        s.synchronize()
        other = t.token_logprobs(x, targets, k=3, stream=s)
        s.synchronize()
    for key in ref:
        assert torch.equal(ref[key], got[key]) and torch.equal(ref[key], other[key])


def test_logprobs_refusals():
    with B.Tokens(4, 8, 9, io="f32") as t:
        x = torch.zeros(4, 9, device="cuda")
        ids = torch.zeros(4, dtype=torch.int64, device="cuda")
        lse = torch.zeros(4, device="cuda")
        for bad in (lambda: t.token_logprobs(x.bfloat16(), ids), lambda: t.token_logprobs(x[:, :8], ids), lambda: t.token_logprobs(x, ids[:3]),
                    lambda: t.token_logprobs(x, ids, k=2, out={"top_ids": ids}), lambda: t.token_logprobs(x, ids, out={"p": lse}),
                    lambda: t.token_logprobs_backward(x, ids, lse[:2], None, lse), lambda: t.token_logprobs(x.cpu(), ids)):
            with pytest.raises(ValueError):
                bad()
        for status, bad in (
                (B.PRISM_ERR_INVALID_ARG, lambda: t.token_logprobs(torch.zeros(5, 9, device="cuda"))),
                (B.PRISM_ERR_INVALID_ARG, lambda: t.token_logprobs(x, ids, k=33)),
                (B.PRISM_ERR_INVALID_ARG, lambda: t.token_logprobs(x, ids, inv_temperature=0.0)),
                (B.PRISM_ERR_INVALID_ARG, lambda: t.token_logprobs(x, ids, inv_temperature=INF)),
                (B.PRISM_ERR_INVALID_ARG, lambda: t.token_logprobs(x, None, out={"logprob": lse})),
                (B.PRISM_ERR_INVALID_ARG, lambda: t.token_logprobs_backward(x, ids, lse, None, None)),
                (B.PRISM_ERR_INVALID_ARG, lambda: t.token_logprobs_backward(x, ids, lse, None, None, lse)),
                (B.PRISM_ERR_INVALID_ARG, lambda: t.token_logprobs_backward(x, None, lse, None, lse)),
                (B.PRISM_ERR_INVALID_ARG, lambda: B.prism_token_logprobs(t.handle, 4, x, 8, None, 1.0, 0, lse, None, None, None, None)),
                (B.PRISM_ERR_MISALIGNED, lambda: B.prism_token_logprobs(t.handle, 3, x.data_ptr() + 4, 9, None, 1.0, 0, lse, None, None, None, None)),
                (B.PRISM_ERR_INVALID_ARG, lambda: B.prism_token_logprobs_backward(t.handle, 2, x, 9, ids, 1.0, lse, None, lse, None, x, 18))):
            with pytest.raises(B.PrismError) as ei:
                bad()
            assert ei.value.status == status
