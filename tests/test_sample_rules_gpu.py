"""The draw where one rule makes another one idle, and at the far end of u, against the fp64 oracle (tolerances: tests/test_sample_gpu.py).

No row here has a border nearer to a token's edge than the kernel's units can tell; where the seeds are changed that has to be looked at again."""
import numpy as np
import pytest
import torch

from ssm_sequence_layer_gb300 import binding as B
from ssm_sequence_layer_gb300 import build
from tests.test_sample_gpu import DT, check

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    build.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"


def combinations(live, V):
    """Rows of (top_k, top_p, min_p): a top_k around the live tokens' number and far beyond, beside the two others."""
    ks = [live - 1, live, live + 1, V, 2 ** 31 - 1]
    return [(k, p, m) for k in ks for p in (0.3, 0.9, 0.9999) for m in (0.0, 0.01)]


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("V", [1100, 2000, 8193, 50021, 131072])
@pytest.mark.parametrize("std", [1.0, 2.5, 6.0])
@pytest.mark.parametrize("masked", [False, True])
def test_top_k_that_reaches_all_beside_top_p(io, V, std, masked):
    """top_k of the vocabulary's size, or of more tokens than are live, leaves the row to top-p and min-p.  A deviation of 1 has no token
    further than 22 below the largest, 6 has many."""
    g = torch.Generator().manual_seed(V + int(10 * std))
    row = torch.randn(V, generator=g) * std
    if masked:
        row[torch.randperm(V, generator=g)[: V // 3]] = -float("inf")
    live = int((row != -float("inf")).sum())
    rules = combinations(live, V)
    n = len(rules)
    x = torch.stack([row[torch.randperm(V, generator=g)] for _ in range(n)]).to(DT[io])
    u = torch.rand(n, generator=g)
    k, p, m = (torch.tensor([r[i] for r in rules]) for i in range(3))
    k = k.int()
    for c in (None, torch.full((n,), 0.8)):
        with_all = check(x, u, c, k, p, m)
        without = check(x, u, c, None, p, m)
        assert np.array_equal(with_all[k.numpy() >= live], without[k.numpy() >= live])


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("V", [40, 700, 5000, 50021, 200000])
def test_u_of_one_gives_the_last_kept_id(io, V):
    """... where the last ids are the least likely: below what a sum of the others tells, and below what masses tell at all."""
    g = torch.Generator().manual_seed(V)
    lowest = torch.tensor([-16.0, -25.0, -29.0, -40.0, -80.0])
    flat = torch.randn(V, generator=g)
    last = V - V // 10  # of the likely ones
    x = flat.repeat(5, 1)
    x[:, last:] = lowest[:, None] + 0.1 * torch.rand(5, V - last, generator=g)
    x = x.to(DT[io])
    for u in (1.0, 2.0, float("inf")):
        uu = torch.full((5,), u)
        from_oracle = lambda *rules: check(x, uu, None, *rules)  # noqa: E731
        assert (from_oracle() == V).all()
        from_oracle(torch.full((5,), V - 3).int())
        from_oracle(torch.full((5,), min(V, 200)).int())
        from_oracle(None, torch.full((5,), 0.9999))
        from_oracle(None, None, torch.full((5,), 1e-8))
        from_oracle(torch.full((5,), V // 2).int(), torch.full((5,), 0.9), torch.full((5,), 1e-3))
    # a row that falls by one from id to id: all of the first fifty are kept
    steep = -torch.arange(V).float().repeat(1, 1).to(DT[io])
    check(steep, torch.ones(1), None, torch.full((1,), min(V, 50)).int())


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("V,n", [(7, 400), (42, 400), (494, 400), (3000, 200), (22326, 200)])
def test_top_p_next_to_one_beside_a_small_min_p(io, V, n):
    """What top-p leaves out, 2^-24 of the mass, is less than rough masses tell: whether it ends the row before min-p does has to be found with
    closer ones."""
    g = torch.Generator().manual_seed(V)
    x = (torch.randn(n, V, generator=g) * torch.tensor([2.5, 6.0, 4.0, 2.5]).repeat(n // 4)[:, None]).to(DT[io])
    p, m = torch.full((n,), 1 - 2.0 ** -24), torch.tensor([1e-10, 1e-20]).repeat(n // 2)
    # the tokens' masses from the smallest on, against what is left out: only rows in which they are further apart than two units a token
    e = np.exp(x.double().numpy() - x.double().numpy().max(1, keepdims=True))
    tail = np.cumsum(np.sort(e, 1), 1)
    gap = np.abs(tail - ((1 - p.double().numpy()) * tail[:, -1])[:, None]).min(1)
    clear = torch.from_numpy(gap > 2 * V * 2.0 ** -44)
    assert clear.sum() >= 50
    x, p, m, u = x[clear], p[clear], m[clear], torch.rand(n, generator=g)[clear]
    kept = check(x, u, None, None, p, m)
    assert (kept < V).any()
    check(x, u, None, torch.full((x.shape[0],), V).int(), p, m)
    check(x, u, None, None, p, None)


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("V", [2000, 9000, 50021])
@pytest.mark.parametrize("min_p", [None, 1e-9])
def test_every_top_p_next_to_one(io, V, min_p):
    """Every float32 of 1 - 2^-12 .. 1, and as many all over (0, 1), of three rows: wherever the border falls it is found, also between what two
    threads add up."""
    g = torch.Generator().manual_seed(V)
    p = torch.cat([1 - torch.arange(1, 4097) * 2.0 ** -24, torch.rand(4096, generator=g)])
    n = p.numel()
    with B.Tokens(n, 64, V, io=io) as t:
        for _ in range(3):
            row = (torch.randn(V, generator=g) * 2.5).to(DT[io])
            out = t.sample(row.cuda().repeat(n, 1), torch.full((n,), 0.5, device="cuda"), None, None, p.cuda(), min_p)
            torch.cuda.synchronize()
            t.last_device_status()
            z = np.sort(row.double().numpy())[::-1]
            e = np.exp(z - z[0])
            running = np.cumsum(e)
            target = p.double().numpy() * running[-1]
            kept = np.searchsorted(running, target) + 1
            # where a border is within the kernel's units of a token's edge either side will do
            near = np.minimum(np.abs(running[np.minimum(kept, V) - 1] - target), np.abs(running[np.maximum(kept - 2, 0)] - target)) <= 2 * V * 2.0 ** -44
            if min_p is not None:
                kept = np.minimum(kept, int((z - z[0] >= np.log(np.float32(min_p).astype(np.float64))).sum()))
            assert near.mean() < 0.5
            assert np.array_equal(out["kept"].cpu().numpy()[~near], kept[~near])


@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_u_next_to_one_where_one_token_has_nearly_all(io):
    """A row whose other tokens' masses vanish beside the largest one's in float32: u of 1 - 2^-24 falls beyond the largest by half of its distance to
    one, which rough masses do not show although their sum ends with that token."""
    row = torch.tensor([9.140625, -7.578125, -8.0859375, -13.046875, -18.28125, -32.0, -52.5])
    x = row.repeat(4, 1)
    x[1], x[2] = row[[1, 0, 2, 3, 4, 5, 6]], row[[1, 2, 3, 4, 5, 6, 0]]
    x[3, 1:3] = -9.0
    check(x.to(DT[io]), torch.full((4,), 1 - 2.0 ** -24))
    for V in (900, 30000):
        g = torch.Generator().manual_seed(V)
        x = torch.full((50, V), -60.0)
        x.scatter_(1, torch.randint(0, V, (50, 40), generator=g), -17 - 4 * torch.rand(50, 40, generator=g))
        x.scatter_(1, torch.randint(0, V // 2, (50, 1), generator=g), 0.0)
        check(x.to(DT[io]), torch.full((50,), 1 - 2.0 ** -24))
        check(x.to(DT[io]), torch.full((50,), 1 - 2.0 ** -23))
