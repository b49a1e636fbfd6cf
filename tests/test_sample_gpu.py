"""The draw of a token against the fp64 oracle.  ids and the number kept are whole numbers and have to be equal: the kernel's
masses are within 2^-42 of the first token's and the oracle's within 2^-50 of themselves, and no number here is drawn that near to a border.
logprob = (l - max) c - log(mass): both parts in 64 bits from the logits and masses within 2^-21 of themselves, rounded to fp32:
2^-20 + 2^-23 |logprob|."""
import numpy as np
import pytest
import torch

from oracle import prism_block as O
from ssm_sequence_layer_gb300 import binding as B
from ssm_sequence_layer_gb300 import build

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(scope="module", autouse=True)
def _built():
    build.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"


def f64(t):
    return None if t is None else t.float().cpu().double().numpy()


def check(logits, u, c=None, k=None, p=None, m=None, io=None, V=None):
    """The call's outputs against the oracle's, the rules as [n] tensors; returns what was kept."""
    n, V = logits.shape
    io = "bf16" if logits.dtype is torch.bfloat16 else "f32"
    dev = lambda t: None if t is None else t.cuda()  # noqa: E731
    with B.Tokens(n, 64, V, io=io) as t:
        out = t.sample(logits.cuda() if not logits.is_cuda else logits, dev(u), dev(c), dev(k), dev(p), dev(m))
        torch.cuda.synchronize()
        t.last_device_status()
    ids, logprob, kept = O.sample(f64(logits), f64(u), f64(c), None if k is None else k.cpu().numpy(), f64(p), f64(m))
    assert np.array_equal(out["kept"].cpu().numpy(), kept)
    assert np.array_equal(out["ids"].cpu().numpy(), ids)
    got = f64(out["logprob"])
    same = (got == logprob) | (np.isnan(got) & np.isnan(logprob))
    with np.errstate(invalid="ignore"):
        assert np.all(same | (np.abs(got - logprob) <= 2.0 ** -20 + 2.0 ** -23 * np.abs(logprob)))
    return kept


def rows(n, V, io, seed, std=2.5, masked=False):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(n, V, generator=g) * std
    x[:, torch.randint(0, V, (4,), generator=g)] += 6 * torch.rand(n, 4, generator=g)
    if masked:
        x[torch.rand(n, V, generator=g) < 0.2] = -float("inf")
        x[torch.rand(n, V, generator=g) < 0.1] = -3.3895313892515355e38
    return x.to(DT[io]), torch.rand(n, generator=g), 0.5 + torch.rand(n, generator=g), g


SIZES = [(1, 1), (3, 2), (4, 7), (5, 100), (64, 1000), (9, 2047), (7, 8193), (6, 50021), (2, 131072)]


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("n,V", SIZES)
@pytest.mark.parametrize("masked", [False, True])
def test_rules_one_by_one_and_together(io, n, V, masked):
    x, u, c, g = rows(n, V, io, n + V, masked=masked and V > 20)
    k = torch.randint(0, min(V, 300) + 2, (n,), generator=g).int()
    p = torch.rand(n, generator=g) * 1.05
    m = torch.rand(n, generator=g) * 0.2
    check(x, u)
    check(x, u, c)
    for rules in ((k, None, None), (None, p, None), (None, None, m), (k, p, None), (k, p, m), (None, p, m)):
        check(x, u, c, *rules)


@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_numbers_next_to_a_border(io):
    """u as the float32 nearest to a running mass: nearer than quick masses can tell apart."""
    n, V = 200, 3000
    x, _, c, g = rows(n, V, io, 3)
    z = f64(x) * f64(c)[:, None]
    e = np.exp(z - z.max(1, keepdims=True))
    at = np.cumsum(e, 1) / e.sum(1, keepdims=True)
    u = torch.from_numpy(at[np.arange(n), np.random.default_rng(0).integers(0, V - 1, n)]).float().clamp_max(1 - 2.0 ** -24)
    check(x, u, c)
    # ... and top-p as the float32 nearest to the mass of a prefix
    s = -np.sort(-e, 1)
    p = torch.from_numpy((np.cumsum(s, 1) / s.sum(1, keepdims=True))[np.arange(n), np.arange(n) * 7]).float().clamp_max(1 - 2.0 ** -24)
    kept = check(x, u, c, None, p)
    assert len(set(kept)) > 100


@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_flat_rows(io):
    """Hardly any difference between the tokens: each border lies among thousands of nearly equal or equal masses."""
    g = torch.Generator().manual_seed(1)
    n, V = 40, 20000
    u, p = torch.rand(n, generator=g), torch.rand(n, generator=g)
    k = torch.randint(1, V, (n,), generator=g).int()
    for x in (torch.rand(n, V, generator=g) * 1e-3, torch.rand(n, V, generator=g).round() * 0.5, 5 + torch.rand(n, V, generator=g) * 0.01):
        x = x.to(DT[io])
        check(x, u)
        check(x, u, None, k)
        check(x, u, None, None, p)
        check(x, u, None, k, p)
    equal = torch.full((n, V), -2.5).to(DT[io])
    kept = check(equal, u, None, k)
    assert np.array_equal(kept, k.numpy())
    # equal masses make every running mass a whole number of them: u times their number is no whole number here
    check(equal, (torch.floor(u * V) + 0.5) / V, None, None, None)
    halves = torch.zeros(1, 4)
    check(halves, torch.tensor([0.5]))  # exactly on a border: the token behind it
    check(halves, torch.tensor([0.25]), None, None, torch.tensor([0.5]))  # two tokens reach half of the mass exactly


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("V", [300, 5003, 50021])
def test_orders_and_ties_around_the_kth(io, V):
    """The kth largest among sorted logits, in a crowd of equal ones, and where only a handful of neighbours is above the mask, for k on both
    sides of the sizes at which the kernel's ways part; min-p that many tokens, and all of them, reach."""
    x, u, c, g = rows(12, V, io, 3 * V)
    x[0] = torch.sort(x[0].float(), descending=True)[0].to(x.dtype)
    x[1] = torch.sort(x[1].float())[0].to(x.dtype)
    x[2, 100:] = x[2, 100:].clamp(max=0.5)  # many equal ones below few
    x[3, 10:] = -float("inf")
    x[4] = 0.25
    x[5] = torch.linspace(4, -60, V).to(x.dtype)
    for k in (1, 2, 10, 11, 191, 192, 193, 256, 257, 383, 384, 385, 767, 768, 769, 1024, 1025):
        kk = torch.full((12,), k, dtype=torch.int32)
        check(x, u, c, kk)
        check(x, u, c, kk, torch.full((12,), 0.9))
        check(x, u, c, kk, None, torch.full((12,), 0.02))
    for m in (1e-30, 1e-6, 0.3):
        check(x, u, c, None, None, torch.full((12,), m))
        check(x, u, c, None, torch.full((12,), 0.8), torch.full((12,), m))


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("V,std", [(20011, 1.0), (50021, 1.0), (50021, 6.0)])
def test_borders_among_many_tokens(io, V, std):
    """Rules that end within thousands of tokens, each of them first once, where nothing is short enough to be sorted from its first token on;
    and in rows with little mass beside a few tokens."""
    x, u, c, g = rows(8, V, io, 5 * V, std=std)
    full = lambda v, t=torch.float32: torch.full((8,), v, dtype=t)  # noqa: E731
    for k in (None, 3000, 15000):
        kk = None if k is None else full(k, torch.int32)
        for p in (None, 0.3, 0.9, 0.99, 0.9999):
            for m in (None, 0.2, 0.05, 0.003):
                check(x, u, c, kk, None if p is None else full(p), None if m is None else full(m))


@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_ends_of_the_rules(io):
    n, V = 12, 500
    x, u, c, _ = rows(n, V, io, 8)
    u[0], u[1], u[2], u[3], u[4] = 0.0, 1 - 2.0 ** -24, 1.0, -1.0, float("nan")
    c[5], c[6] = 2.0 ** -60, 2.0 ** 126
    ones = lambda v: torch.full((n,), v)  # noqa: E731
    assert check(x, u, c)[0] == V
    assert (check(x, u, c, ones(1).int()) == 1).all()
    assert (check(x, u, c, ones(V + 5).int())[7:] == V).all() and (check(x, u, c, ones(-3).int())[7:] == V).all()
    assert (check(x, u, c, None, ones(0.0)) == 1).all() and (check(x, u, c, None, ones(-1.0)) == 1).all()
    assert (check(x, u, c, None, ones(2.0))[7:] == V).all()
    assert (check(x, u, c, None, None, ones(3.0)) == 1).all()
    check(x, u, c, None, None, ones(1.0))
    check(x, u, c, None, None, ones(-1.0))
    nan = ones(float("nan"))
    with B.Tokens(n, 64, V, io=io) as t:
        a, b = t.sample(x.cuda(), u.cuda(), c.cuda()), t.sample(x.cuda(), u.cuda(), c.cuda(), None, nan.cuda(), nan.cuda())
        assert all(torch.equal(a[key], b[key]) for key in a)
        s = t.sample(x.cuda(), u.cuda(), 0.5, 7, 0.9, 0.01)
        r = t.sample(x.cuda(), u.cuda(), ones(0.5).cuda(), ones(7).int().cuda(), ones(0.9).cuda(), ones(0.01).cuda())
        assert all(torch.equal(s[key], r[key]) for key in s)


@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_rows_without_a_token(io):
    inf, nan = float("inf"), float("nan")
    x = torch.zeros(6, 300)
    x[0] = -inf
    x[1] = -3.4e38 if io == "f32" else -3.3895313892515355e38
    x[2, 7] = nan
    x[3, 9] = inf
    x[4, 11] = -inf
    x[5, :299] = -inf  # one token alone
    k, p, m = torch.full((6,), 5).int(), torch.full((6,), 0.9), torch.full((6,), 0.1)
    check(x.to(DT[io]), torch.full((6,), 0.5), None, k, p, m)
    check(x.to(DT[io]), torch.full((6,), 0.5))
    c = torch.tensor([1.0, nan, 0.0, -1.0, inf, 1.0])
    with B.Tokens(6, 64, 300, io=io) as t:
        out = t.sample(torch.zeros(6, 300, dtype=DT[io], device="cuda"), torch.full((6,), 0.5, device="cuda"), c.cuda())
        torch.cuda.synchronize()
        with pytest.raises(B.PrismError) as e:
            t.last_device_status()
        assert e.value.status == B.PRISM_ERR_DEVICE and "inv_temperature" in str(e.value)
        t.last_device_status()
    assert out["ids"].tolist() == [150, -1, -1, -1, -1, 150] and out["kept"].tolist() == [300, 0, 0, 0, 0, 300]
    assert torch.isnan(out["logprob"][1:5]).all()


def test_signed_zeros_are_equal():
    x = torch.tensor([[-0.0, 0.0, -0.0, 0.0, -1.0]])
    assert check(x, torch.tensor([0.6]), None, torch.tensor([2]).int()) == [2]
    ids = []
    with B.Tokens(1, 64, 5, io="f32") as t:
        for v in (0.25, 0.75):
            ids.append(t.sample(x.cuda(), torch.tensor([v]).cuda(), None, 2)["ids"].item())
    assert ids == [0, 1]


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("pad", [1, 3, 8])
def test_padded_rows_are_not_read(io, pad):
    n, V = 9, 1235
    x, u, c, _ = rows(n, V, io, 4)
    full = torch.full((n, V + pad), float("nan"), dtype=DT[io], device="cuda")
    full[:, :V] = x.cuda()
    k, p = torch.full((n,), 30).int(), torch.full((n,), 0.8)
    check(full[:, :V], u, c, k, p)
    check(full[:, :V], u, c)
    with B.Tokens(n, 64, V, io=io) as t:
        few = t.sample(full[:, :V], u.cuda(), out={"ids": torch.empty(n, dtype=torch.int64, device="cuda")})
        assert torch.equal(few["ids"], t.sample(x.cuda(), u.cuda())["ids"]) and list(few) == ["ids"]
        assert t.sample(torch.empty(0, V, dtype=DT[io], device="cuda"), torch.empty(0, device="cuda"))["ids"].shape == (0,)


def test_shares_of_many_draws():
    """A grid of u over [0, 1): each kept token gets as many of them as its share says, within one."""
    n = 4096
    g = torch.Generator().manual_seed(0)
    row = torch.randn(50, generator=g) * 1.5
    u = (torch.arange(n) + 0.5) / n
    with B.Tokens(n, 64, 50, io="f32") as t:
        ids = t.sample(row.repeat(n, 1).cuda(), u.cuda(), None, 20)["ids"].cpu().numpy()
    keep = np.argsort(-row.numpy(), kind="stable")[:20]
    e = np.zeros(50)
    e[keep] = np.exp(row.double().numpy())[keep]
    assert np.all(np.abs(np.bincount(ids, minlength=50) - n * e / e.sum()) <= 1) and np.all(np.diff(ids) >= 0)


def test_refusals():
    x, u = torch.zeros(4, 40, dtype=torch.bfloat16, device="cuda"), torch.zeros(4, device="cuda")
    ids = torch.zeros(4, dtype=torch.int64, device="cuda")
    bad, misaligned = B.PRISM_ERR_INVALID_ARG, B.PRISM_ERR_MISALIGNED
    none = (None,) * 4
    with B.Tokens(4, 64, 40) as t:
        for call, status in [(lambda: B.prism_sample(t.handle, 5, x, 40, u, *none, ids, None, None), bad), (lambda: B.prism_sample(t.handle, 4, x, 39, u, *none, ids, None, None), bad),
                             (lambda: B.prism_sample(t.handle, 4, None, 40, u, *none, ids, None, None), bad), (lambda: B.prism_sample(t.handle, 4, x, 40, None, *none, ids, None, None), bad),
                             (lambda: B.prism_sample(t.handle, 4, x, 40, u, *none, None, None, None), bad),
                             (lambda: B.prism_sample(t.handle, 4, x, 40, u.data_ptr() + 2, *none, ids, None, None), misaligned),
                             (lambda: B.prism_sample(t.handle, 4, x, 40, u, *none, ids.data_ptr() + 4, None, None), misaligned),
                             (lambda: B.prism_sample(t.handle, 4, x, 40, u, None, u.data_ptr() + 1, None, None, ids, None, None), misaligned)]:
            with pytest.raises(B.PrismError) as e:
                call()
            assert e.value.status == status


def test_streams_graphs_and_equal_bits():
    x, u, c, _ = rows(20, 7000, "f32", 2)
    x, u, c = x.cuda(), u.cuda(), c.cuda()
    with B.Tokens(20, 64, 7000, io="f32") as t:
        call = lambda **kw: t.sample(x, u, c, 100, 0.9, **kw)  # noqa: E731
        first = call()
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        own = call(stream=side)
        torch.cuda.synchronize()
        assert all(torch.equal(own[key], first[key]) for key in first)
        graph = torch.cuda.CUDAGraph()
        rules = [torch.full((20,), v, device="cuda", dtype=d) for v, d in ((100, torch.int32), (0.9, torch.float32))]
        with torch.cuda.graph(graph):
            held = t.sample(x, u, c, *rules)
        u0 = u.clone()
        u.copy_(1 - u)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(held["ids"], call()["ids"]) and not torch.equal(held["ids"], first["ids"])
        u.copy_(u0)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(held[key], first[key]) for key in first)
