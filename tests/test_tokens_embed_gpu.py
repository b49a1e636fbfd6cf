"""The embedding and its gradient against the fp64 oracle.

Tolerances.  The lookup multiplies once and rounds once: half a unit in the last place of the io type,
plus half a unit of fp32.  A gradient row is a sum of m terms in fp32: |error| <= m 2^-24 sum |terms|
(any order of additions), plus one rounding for the scale and one for an addition onto the table."""
import numpy as np
import pytest
import torch

from oracle import prism_tokens as O
from ssm_sequence_layer_gb300 import binding as B
from ssm_sequence_layer_gb300 import build
from tests.gpu_util import bf16_half_ulp

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(scope="module", autouse=True)
def _built():
    build.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"


def draw_ids(n, V, seed, kind):
    g = torch.Generator().manual_seed(seed)
    if kind == "one":
        return torch.full((n,), V - 1, dtype=torch.int64)
    if kind == "none":
        return torch.full((n,), -1, dtype=torch.int64)
    if kind == "distinct":
        return torch.randperm(V, generator=g)[:n]
    ids = (torch.exp(torch.rand(n, generator=g, dtype=torch.float64) * np.log(V + 1)) - 1).long().clamp_(0, V - 1)
    ids[torch.rand(n, generator=g) < 0.1] = -1
    return ids


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("n,D,V,pad", [(1, 64, 10, 0), (16, 768, 5003, 0), (333, 257, 1000, 0), (70, 8, 17, 8), (5, 1, 3, 0),
                                       (40, 2048, 100, 3), (0, 32, 10, 0)])
def test_embed(io, n, D, V, pad):
    g = torch.Generator().manual_seed(n + D)
    full = torch.randn(V, D + pad, generator=g).to(DT[io]).cuda()
    table = full[:, :D]
    ids = draw_ids(n, V, 3, "zipf")
    with B.Tokens(max(n, 1), D, V, io=io) as t:
        out = t.embed(ids.cuda(), table, scale=1.7)
        torch.cuda.synchronize()
        t.last_device_status()
    ref = O.embed(ids.numpy(), table.float().cpu().numpy(), float(np.float32(1.7)))
    got = out.double().cpu().numpy()
    assert got.shape == ref.shape
    half_ulp = bf16_half_ulp(ref) if io == "bf16" else 2.0 ** -24 * np.abs(ref)
    assert np.all(np.abs(got - ref) <= half_ulp + 2.0 ** -24 * np.abs(ref))
    assert np.all(got[ids.numpy() < 0] == 0)


def check_gradient(got, ids, dout, scale, V, onto=None):
    ref = O.embed_backward(ids, dout, scale, V, onto)
    size = O.embed_backward(ids, np.abs(dout), abs(scale), V)
    count = np.bincount(ids[ids >= 0], minlength=V)[:, None]
    tol = 2.0 ** -24 * ((count + 2) * size + np.abs(ref) + (0 if onto is None else np.abs(onto)))
    assert np.all(np.abs(got - ref) <= tol)
    if onto is None:
        assert np.all(got[count[:, 0] == 0] == 0)


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("n,D,V,kind", [
    (1, 64, 10, "zipf"), (16, 768, 50, "zipf"), (17, 8, 3, "zipf"), (333, 257, 1000, "zipf"), (2048, 64, 511, "zipf"),
    (2049, 64, 512, "zipf"), (5000, 40, 70001, "zipf"), (5000, 128, 7, "one"), (300, 136, 20, "none"),
    (4000, 72, 4000, "distinct"), (12000, 1032, 300, "zipf"), (3000, 1, 300000, "zipf"), (270000, 16, 90, "zipf"),
    (20000, 24, 40000, "zipf"), (40000, 8, 600000, "zipf"), (65537, 8, 1000, "one"), (70000, 12, 262144, "zipf"), (2500, 520, 9000, "one")])
def test_embed_backward(io, n, D, V, kind):
    g = torch.Generator().manual_seed(n * 3 + D)
    ids = draw_ids(n, V, 5, kind)
    dout = torch.randn(n, D, generator=g).to(DT[io])
    with B.Tokens(n, D, V, io=io) as t:
        dtable = torch.full((V, D), float("nan"), device="cuda")
        t.embed_backward(ids.cuda(), dout.cuda(), scale=0.75, dtable=dtable)
        first = dtable.clone()
        onto = torch.randn(V, D, generator=g).cuda()
        added = onto.clone()
        t.embed_backward(ids.cuda(), dout.cuda(), scale=0.75, dtable=added, accumulate=True)
        t.embed_backward(ids.cuda(), dout.cuda(), scale=0.75, dtable=dtable)
        torch.cuda.synchronize()
        t.last_device_status()
    assert torch.equal(first, dtable), "equal inputs give equal bits"
    d64 = dout.double().numpy()
    check_gradient(first.double().cpu().numpy(), ids.numpy(), d64, 0.75, V)
    check_gradient(added.double().cpu().numpy(), ids.numpy(), d64, 0.75, V, onto.double().cpu().numpy())


def test_ids_of_the_largest_vocabulary():
    """Ids of up to 30 bits, the sort's four passes, on both sides of the cluster sort's capacity; the table
    itself does not fit, so the gradient goes onto ids that are the last rows of nothing: D = 1, 2^28 rows."""
    V = 1 << 28
    for n in (100, 5000, 70000):
        g = torch.Generator().manual_seed(n)
        ids = torch.randint(0, V, (n,), generator=g)
        ids[: n // 2] = V - 1 - torch.randint(0, 50, (n // 2,), generator=g)
        dout = torch.randn(n, 1, generator=g)
        with B.Tokens(n, 1, V, io="f32") as t:
            d = t.embed_backward(ids.cuda(), dout.cuda())
            torch.cuda.synchronize()
            t.last_device_status()
        rows, inverse = torch.unique(ids, return_inverse=True)
        ref = torch.zeros(rows.numel(), dtype=torch.float64).index_add_(0, inverse, dout[:, 0].double())
        size = torch.zeros(rows.numel(), dtype=torch.float64).index_add_(0, inverse, dout[:, 0].double().abs())
        count = torch.bincount(inverse)
        assert torch.all((d[rows.cuda(), 0].cpu().double() - ref).abs() <= 2.0 ** -24 * (count + 2) * size)
        assert torch.count_nonzero(d).item() == torch.count_nonzero(ref.float()).item()
        del d


@pytest.mark.parametrize("n,D", [(300, 131), (5000, 132), (5000, 133), (70000, 134)])
def test_tables_larger_than_the_sort_clears(n, D):
    """160 to 420 MB of table: rows without a token are zero wherever they are cleared, rows at any alignment."""
    V = 300007 if n < 65537 else 800000
    g = torch.Generator().manual_seed(D)
    ids = draw_ids(n, V, D, "zipf")
    ids = torch.where(ids >= 0, torch.randperm(V, generator=g)[ids], ids)
    dout = torch.randn(n, D, generator=g)
    with B.Tokens(n, D, V, io="f32") as t:
        room = torch.full((V * D + 8,), float("nan"), device="cuda")
        dtable = room[4:4 + V * D].view(V, D)
        t.embed_backward(ids.cuda(), dout.cuda(), dtable=dtable)
        torch.cuda.synchronize()
        t.last_device_status()
    assert torch.isnan(room[:4]).all() and torch.isnan(room[4 + V * D:]).all()
    keep = ids >= 0
    rows, inverse = torch.unique(ids[keep], return_inverse=True)
    ref = torch.zeros(rows.numel(), D, dtype=torch.float64).index_add_(0, inverse, dout[keep].double())
    size = torch.zeros(rows.numel(), D, dtype=torch.float64).index_add_(0, inverse, dout[keep].double().abs())
    count = torch.bincount(inverse)[:, None]
    assert torch.all((dtable[rows.cuda()].cpu().double() - ref).abs() <= 2.0 ** -24 * (count + 2) * size)
    dtable[rows.cuda()] = 0
    assert torch.count_nonzero(dtable).item() == 0


def test_embed_gradient_is_the_lookup_transposed():
    """<embed(table), c> = <table, embed_backward(c)> for the linear map that a set of ids defines."""
    n, D, V = 500, 96, 77
    g = torch.Generator().manual_seed(0)
    ids = draw_ids(n, V, 9, "zipf").cuda()
    table, c = torch.randn(V, D, generator=g).cuda(), torch.randn(n, D, generator=g).cuda()
    with B.Tokens(n, D, V, io="f32") as t:
        a = (t.embed(ids, table, scale=2.0).double() * c.double()).sum()
        b = (table.double() * t.embed_backward(ids, c, scale=2.0).double()).sum()
    # both sides sum n D products of size about 2 with fp32 roundings inside
    assert abs(a - b) <= 2.0 ** -20 * n * D


def test_no_tokens_clears_the_gradient():
    with B.Tokens(4, 8, 5, io="f32") as t:
        d = torch.full((5, 8), 3.0, device="cuda")
        t.embed_backward(torch.empty(0, dtype=torch.int64, device="cuda"), torch.empty(0, 8, device="cuda"), dtable=d)
        assert torch.all(d == 0)


def test_ids_beyond_the_vocabulary_are_recorded():
    ids = torch.tensor([1, 9, 2], device="cuda")
    table = torch.ones(9, 16, device="cuda")
    with B.Tokens(3, 16, 9, io="f32") as t:
        out = t.embed(ids, table)
        torch.cuda.synchronize()
        with pytest.raises(B.PrismError) as ei:
            t.last_device_status()
        assert ei.value.status == B.PRISM_ERR_DEVICE
        t.last_device_status()  # read once, then clear
        assert torch.equal(out.cpu(), torch.tensor([1.0, 0.0, 1.0])[:, None].expand(3, 16))
        d = t.embed_backward(ids, out)
        torch.cuda.synchronize()
        with pytest.raises(B.PrismError):
            t.last_device_status()
        assert d.sum().item() == 32.0


def test_embed_runs_on_the_callers_stream_and_in_a_graph():
    n, D, V = 3000, 64, 200
    ids, dout = draw_ids(n, V, 2, "zipf").cuda(), torch.randn(n, D, device="cuda")
    with B.Tokens(n, D, V, io="f32") as t:
        ref = t.embed_backward(ids, dout)
        torch.cuda.synchronize()
        s = torch.cuda.Stream()
        d = torch.empty(V, D, device="cuda")
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            t.embed_backward(ids, dout, dtable=d)
        for _ in range(2):
            d.fill_(float("nan"))
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(d, ref)


def test_embed_refusals():
    with B.Tokens(4, 16, 9, io="bf16") as t:
        ids = torch.zeros(4, dtype=torch.int64, device="cuda")
        table = torch.zeros(9, 16, dtype=torch.bfloat16, device="cuda")
        for bad in (lambda: t.embed(ids.int(), table), lambda: t.embed(ids, table.float()), lambda: t.embed(ids, table[:8]),
                    lambda: t.embed(ids, table, out=torch.zeros(3, 16, dtype=torch.bfloat16, device="cuda")),
                    lambda: t.embed_backward(ids, table[:3]), lambda: t.embed_backward(ids, table[:4], accumulate=True),
                    lambda: t.embed(ids.cpu(), table)):
            with pytest.raises(ValueError):
                bad()
        for status, bad in ((B.PRISM_ERR_INVALID_ARG, lambda: t.embed(torch.zeros(5, dtype=torch.int64, device="cuda"), table)),
                            (B.PRISM_ERR_INVALID_ARG, lambda: B.prism_embed(t.handle, 4, ids, table, 15, 1.0, table)),
                            (B.PRISM_ERR_INVALID_ARG, lambda: B.prism_embed(t.handle, 4, None, table, 16, 1.0, table)),
                            (B.PRISM_ERR_MISALIGNED, lambda: B.prism_embed(t.handle, 4, ids, table.data_ptr() + 2, 16, 1.0, table)),
                            (B.PRISM_ERR_INVALID_ARG, lambda: t.set_option(B.PRISM_OPT_SEGMENTS, 1))):
            with pytest.raises(B.PrismError) as ei:
                bad()
            assert ei.value.status == status


def test_outputs_come_from_the_given_streams_memory():
    """A block that the current stream has just freed may still be read by its pending work, so a call on
    another stream must not get it for its output."""
    n, D, V = 4096, 1024, 64
    g = torch.Generator().manual_seed(1)
    ids, table = draw_ids(n, V, 2, "zipf").cuda(), torch.randn(V, D, generator=g).cuda()
    s = torch.cuda.Stream()
    with B.Tokens(n, D, V, io="f32") as t:
        ref = t.embed(ids, table)
        torch.cuda.synchronize()
        freed = torch.empty(n, D, device="cuda")
        address = freed.data_ptr()
        del freed
        outs = [t.embed(ids, table, stream=s), t.embed(ids, table, stream=s.cuda_stream)]
        assert all(o.data_ptr() != address for o in outs)
        outs.append(t.embed(ids, table, stream=0))
        torch.cuda.synchronize()
    for o in outs:
        assert torch.equal(o, ref)
