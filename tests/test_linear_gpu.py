"""The product with bias, activation and residual, and its gradients, against the fp64 oracle.

Tolerances, with u = 2^-24 (fp32), h = half a unit in the last place of the io type and S = sum |a_k b_k| (+ |bias|):
  pre, and every product before what follows it: K additions in any order, each within u of a partial sum that is at most S, and
    the last few of the epilogue: (K + 8) u S.  fp32 operands enter in three bfloat16 parts; what is dropped of each product
    is two terms of at most 2^-7 2^-15 of it each and one below: 2^-20 S.
  y        the activation's slope is at most 1.13 in magnitude: 1.13 times that, 2^-19 |act(pre)| for the activation itself
    (its approximations are within 2^-20 of the value), 2^-126 where it falls below the normal numbers, u |y| and h.
  dx       |slope| times the product's error plus 2^-19 |product| max(|slope|, |z| phi(z)) for the slope's own
    (a sum of two terms of that size), u |dx| and h.
  dW, dbias  sums of M terms: (M + 8) u S (2^-20 S more for fp32 operands), and u |dW| for the addition onto what is there."""
import numpy as np
import pytest
import torch

from oracle import prism_block as O
from ssm_sequence_layer_gb300 import binding as B
from ssm_sequence_layer_gb300 import build
from tests.gpu_util import bf16_half_ulp

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
u = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def _built():
    build.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"


def half_ulp(io, x):
    return bf16_half_ulp(x) if io == "bf16" else u * np.abs(x)


def f64(t):
    return t.float().cpu().double().numpy()


def tensors(io, seed, *shapes):
    g = torch.Generator().manual_seed(seed)
    return [torch.randn(*s, generator=g).to(DT[io]).cuda() for s in shapes]


def close(got, ref, err, io):
    err = err + u * np.abs(ref)
    bad = np.abs(f64(got) - ref) > err + half_ulp(io, np.abs(ref) + err) * 1.0001
    assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[:4].tolist(), float(np.max(np.abs(f64(got) - ref) / (err + half_ulp(io, ref) + 1e-300))))


def product_error(io, a, b, extra=0.0):
    K = a.shape[1]
    return ((K + 8) * u + (2.0 ** -20 if io == "f32" else 0.0)) * (np.abs(a) @ np.abs(b) + extra)


FEW = [(17, 768, 768), (24, 2304, 72), (32, 7290, 64), (32, 7296, 64), (32, 1024, 8192), (32, 1024, 8200), (33, 100, 520), (47, 1000, 2304), (63, 257, 2312), (64, 2048, 2048),
       (64, 2049, 2048), (65, 768, 768)]
SHAPES = [(1, 1, 1), (1, 64, 64), (2, 130, 72), (5, 7, 3), (16, 2304, 768), (8, 264, 1000), (17, 129, 65), (33, 8, 4096), (64, 96, 128), (128, 256, 64),
          (129, 255, 136), (300, 515, 770), (200, 64, 1041), (1003, 770, 200), (2500, 768, 256), (40, 4096, 48)]


@pytest.mark.parametrize("io,M,N,K", [(io, *shape) for io in ("bf16", "f32") for shape in SHAPES] + [("bf16", *shape) for shape in FEW])
def test_linear(io, M, N, K):
    x, W, b, r = tensors(io, M + N + K, (M, K), (N, K), (N,), (M, N))
    W *= K ** -0.5
    X, WW, bb, rr = (f64(t) for t in (x, W, b, r))
    with B.Tokens(M, 64, 64, io=io) as t:
        runs = {(act, has): t.linear(x, W, bias=b if has else None, activation=act, residual=r if has else None, want=("y", "pre"))
                for act in ("none", "gelu", "silu") for has in (True, False)}
        only = t.linear(x, W, bias=b, activation="gelu", residual=r)
        torch.cuda.synchronize()
        t.last_device_status()
    assert torch.equal(only["y"], runs["gelu", True]["y"]) and list(only) == ["y"]
    for (act, has), out in runs.items():
        pre, y = O.linear(X, WW, bb if has else None, act, rr if has else None)
        e = product_error(io, X, WW.T, np.abs(bb) if has else 0.0)
        close(out["pre"], pre, e, io)
        close(out["y"], y, 1.13 * e + 2.0 ** -19 * np.abs(O.act_value(act, pre)) + 2.0 ** -126, io)


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_linear_backward(io, M, N, K):
    dy, W, pre, ds = tensors(io, M + N + K + 1, (M, N), (N, K), (M, K), (M, K))
    W *= K ** -0.5
    pre *= 2
    D, WW, P, S = (f64(t) for t in (dy, W, pre, ds))
    with B.Tokens(M, 64, 64, io=io) as t:
        runs = {(act, has): t.linear_backward(dy, W, activation=act, pre=pre if act != "none" else None, dsum=ds if has else None)
                for act in ("none", "gelu", "silu") for has in (True, False)}
        torch.cuda.synchronize()
        t.last_device_status()
    for (act, has), dx in runs.items():
        plain = O.linear_backward(D, WW, "none", None, None)
        ref = O.linear_backward(D, WW, act, P, S if has else None)
        slope = np.abs(O.act_slope(act, P)) if act != "none" else 1.0
        e = slope * product_error(io, D, WW)
        if act != "none":
            e = e + 2.0 ** -19 * np.abs(plain) * np.maximum(slope, np.abs(P) * np.exp(-P * P / 2) * 0.4 if act == "gelu" else np.abs(P) * np.exp(-np.abs(P)))
        close(dx, ref, e, io)


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("M,N,K", SHAPES + [(5000, 40, 24), (16384, 8, 8), (9999, 130, 7)])
def test_linear_weight_backward(io, M, N, K):
    dy, x = tensors(io, M + N + K + 2, (M, N), (M, K))
    D, X = f64(dy), f64(x)
    onto = torch.randn(N, K, device="cuda"), torch.randn(N, device="cuda")
    with B.Tokens(M, 64, 64, io=io) as t:
        out = t.linear_weight_backward(dy, x, want=("dW", "dbias"))
        alone = t.linear_weight_backward(dy, x)
        added = t.linear_weight_backward(dy, x, out={"dW": onto[0].clone(), "dbias": onto[1].clone()}, accumulate=True)
        torch.cuda.synchronize()
        t.last_device_status()
    assert torch.equal(alone["dW"], out["dW"])
    dW, db = O.linear_weight_backward(D, X)
    e, eb = product_error(io, D.T, X), product_error(io, D.T, np.ones((M, 1)))[:, 0]
    close(out["dW"], dW, e, "f32")
    close(out["dbias"], db, eb, "f32")
    for got, add, ref, err in ((added["dW"], onto[0], dW, e), (added["dbias"], onto[1], db, eb)):
        close(got, ref + f64(add), err, "f32")


@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_gradients_of_large_sums_keep_their_bits(io):
    """Sums over many tokens, as a training step has them: 2^-20 of the root of the sum of squares is an eighth of what a
    sum of M terms added one to the other in fp32 may lose on average (a walk of M steps of up to 2^-24 of sums that grow
    like their root: 2^-24 root(M / 2) = 2^-17.5 at M = 16384)."""
    M, N, K = 16384, 96, 80
    dy, x = tensors(io, 9, (M, N), (M, K))
    with B.Tokens(M, 64, 64, io=io) as t:
        out = t.linear_weight_backward(dy, x, want=("dW", "dbias"))
    D, X = f64(dy), f64(x)
    dW, db = O.linear_weight_backward(D, X)
    assert np.sqrt(np.mean((f64(out["dW"]) - dW) ** 2)) <= 2.0 ** -20 * np.sqrt(np.mean(dW ** 2))
    assert np.sqrt(np.mean((f64(out["dbias"]) - db) ** 2)) <= 2.0 ** -20 * np.sqrt(np.mean(db ** 2))


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("M,N,K", [(3, 40, 64), (150, 200, 72), (150, 201, 71), (700, 768, 256)])
def test_in_place_and_no_rows(io, M, N, K):
    x, W, r, dy, ds, pre = tensors(io, 4, (M, K), (N, K), (M, N), (M, N), (M, K), (M, K))
    empty = torch.empty(0, K, dtype=DT[io], device="cuda"), torch.empty(0, N, dtype=DT[io], device="cuda")
    with B.Tokens(M, 64, 64, io=io) as t:
        y = t.linear(x, W, activation="silu", residual=r)["y"]
        dx = t.linear_backward(dy, W, activation="gelu", pre=pre, dsum=ds)
        r2, ds2, pre2 = r.clone(), ds.clone(), pre.clone()
        t.linear(x, W, activation="silu", residual=r2, out={"y": r2})
        t.linear_backward(dy, W, activation="gelu", pre=pre, dsum=ds2, dx=ds2)
        t.linear_backward(dy, W, activation="gelu", pre=pre2, dsum=ds, dx=pre2)
        assert torch.equal(r2, y) and torch.equal(ds2, dx) and torch.equal(pre2, dx)
        assert t.linear(empty[0], W)["y"].shape == (0, N) and t.linear_backward(empty[1], W).shape == (0, K)
        out = {"dW": torch.full((N, K), 7.0, device="cuda"), "dbias": torch.full((N,), 7.0, device="cuda")}
        t.linear_weight_backward(empty[1], empty[0], out=out, accumulate=True)
        assert torch.all(out["dW"] == 7) and torch.all(out["dbias"] == 7)
        t.linear_weight_backward(empty[1], empty[0], out=out)
        assert not out["dW"].any() and not out["dbias"].any()
        t.last_device_status()


@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_bounds_are_kept(io):
    """Outputs inside a larger buffer: what lies before and behind them stays as it was; rows behind the last do too."""
    for M, N, K in ((5, 33, 24), (140, 264, 72), (131, 257, 65)):
        x, W, b = tensors(io, 6, (M, K), (N, K), (N,))
        pad = 64
        with B.Tokens(M + 5, 64, 64, io=io) as t:
            for which in ("y", "pre", "dx", "dW"):
                shape = {"y": (M, N), "pre": (M, N), "dx": (M, K), "dW": (N, K)}[which]
                dtype = torch.float32 if which == "dW" else DT[io]
                buf = torch.full((2 * pad + shape[0] * shape[1],), 42.0, dtype=dtype, device="cuda")
                inner = buf[pad:-pad].view(shape)
                if which in ("y", "pre"):
                    other = torch.empty(M, N, dtype=DT[io], device="cuda")
                    t.linear(x, W, bias=b, activation="gelu", out={"y": other, "pre": other.clone(), which: inner})
                elif which == "dx":
                    t.linear_backward(torch.ones(M, N, dtype=DT[io], device="cuda"), W, dx=inner)
                else:
                    t.linear_weight_backward(torch.ones(M, N, dtype=DT[io], device="cuda"), x, out={"dW": inner})
                assert torch.all(buf[:pad] == 42) and torch.all(buf[-pad:] == 42) and not torch.all(inner == 42), which


def test_far_ends_of_the_activations():
    """Where the exponentials leave float32: gelu and silu go to 0 and z, their slopes to 0 and 1, NaN stays NaN."""
    z = torch.tensor([0.0, -0.0, 1e-30, -1e-30, 5.0, -5.0, -9.0, -12.0, -14.0, 30.0, -30.0, -87.0, -89.0, -104.0, 1e30, -1e30, float("inf"), -float("inf"), float("nan")])
    n = z.numel()
    one = torch.ones(n, 1, device="cuda")
    for act in ("gelu", "silu"):
        with B.Tokens(n, 64, 64, io="f32") as t:
            y = f64(t.linear(one, torch.zeros(1, 1, device="cuda"), activation=act, bias=None)["y"])[:, 0]
            assert not y.any()
            # the pre-activation as a bias, one product a value
            got = np.array([f64(t.linear(torch.zeros(1, 1, device="cuda"), torch.zeros(1, 1, device="cuda"), bias=v.view(1).cuda(), activation=act)["y"])[0, 0] for v in z])
            slope = f64(t.linear_backward(one, torch.ones(1, 1, device="cuda"), activation=act, pre=z.view(n, 1).cuda()))[:, 0]
        v = z.double().numpy()
        finite = np.clip(np.nan_to_num(v, nan=0.0, posinf=1e30, neginf=-700), -700, 1e30)
        with np.errstate(under="ignore", over="ignore", invalid="ignore"):
            ref, sref = O.act_value(act, finite), O.act_slope(act, np.clip(finite, -700, 700))
        ref[v == np.inf] = np.inf
        ok = ~np.isnan(v) & np.isfinite(ref)
        assert np.all(np.abs(got - ref)[ok] <= 2.0 ** -19 * np.abs(ref[ok]) + 2.0 ** -126) and np.isnan(got[-1]) and got[v == np.inf] == np.inf
        assert np.all(np.abs(slope - sref)[~np.isnan(v)] <= 2.0 ** -19) and np.isnan(slope[-1])


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("M,N,K", [(4, 64, 128), (150, 136, 72), (150, 135, 71)])
def test_nan_stays_in_its_row(io, M, N, K):
    x, W = tensors(io, 11, (M, K), (N, K))
    with B.Tokens(M, 64, 64, io=io) as t:
        ref = t.linear(x, W)["y"]
        x[M // 2, K // 3] = float("nan")
        y = t.linear(x, W)["y"]
    assert torch.isnan(y[M // 2]).all()
    rest = torch.arange(M, device="cuda") != M // 2
    assert torch.equal(y[rest], ref[rest])


def test_refusals():
    x, W = tensors("bf16", 2, (8, 64), (32, 64))
    out = torch.empty(8, 32, dtype=torch.bfloat16, device="cuda")
    with B.Tokens(8, 64, 64) as t:
        h = t.handle
        for call, status in [
                (lambda: B.prism_linear(h, 9, 32, 64, x, W, None, 0, None, out, None), B.PRISM_ERR_INVALID_ARG),
                (lambda: B.prism_linear(h, -1, 32, 64, x, W, None, 0, None, out, None), B.PRISM_ERR_INVALID_ARG),
                (lambda: B.prism_linear(h, 8, 0, 64, x, W, None, 0, None, out, None), B.PRISM_ERR_INVALID_ARG),
                (lambda: B.prism_linear(h, 8, 32, 0, x, W, None, 0, None, out, None), B.PRISM_ERR_INVALID_ARG),
                (lambda: B.prism_linear(h, 8, 32, (1 << 20) + 1, x, W, None, 0, None, out, None), B.PRISM_ERR_UNSUPPORTED),
                (lambda: B.prism_linear(h, 8, 32, 64, x, W, None, 3, None, out, None), B.PRISM_ERR_INVALID_ARG),
                (lambda: B.prism_linear(h, 8, 32, 64, None, W, None, 0, None, out, None), B.PRISM_ERR_INVALID_ARG),
                (lambda: B.prism_linear(h, 8, 32, 64, x, None, None, 0, None, out, None), B.PRISM_ERR_INVALID_ARG),
                (lambda: B.prism_linear(h, 8, 32, 64, x, W, None, 0, None, None, None), B.PRISM_ERR_INVALID_ARG),
                (lambda: B.prism_linear(h, 8, 32, 64, x, W, None, 0, None, out, out), B.PRISM_ERR_INVALID_ARG),
                (lambda: B.prism_linear(h, 8, 32, 64, x.data_ptr() + 2, W, None, 0, None, out, None), B.PRISM_ERR_MISALIGNED),
                (lambda: B.prism_linear(h, 8, 32, 64, x, W, W.data_ptr() + 4, 0, None, out, None), B.PRISM_ERR_MISALIGNED),
                (lambda: B.prism_linear_backward(h, 8, 32, 64, out, W, 1, None, None, x), B.PRISM_ERR_INVALID_ARG),
                (lambda: B.prism_linear_backward(h, 8, 32, 64, out, W, 0, None, x.data_ptr() + 8, x), B.PRISM_ERR_MISALIGNED),
                (lambda: B.prism_linear_weight_backward(h, 8, 32, 64, out, x, 0, None, None), B.PRISM_ERR_INVALID_ARG),
                (lambda: B.prism_linear_weight_backward(h, 8, 32, 64, out, None, 0, W, None), B.PRISM_ERR_INVALID_ARG)]:
            with pytest.raises(B.PrismError) as e:
                call()
            assert e.value.status == status


@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_streams_graphs_and_equal_bits(io):
    """On a stream of its own, captured and replayed with new inputs, and again: the same bits every time."""
    M, N, K = 333, 264, 136
    x, W, b, dy = tensors(io, 13, (M, K), (N, K), (N,), (M, N))
    with B.Tokens(M, 64, 64, io=io) as t:
        def call():
            out = t.linear(x, W, bias=b, activation="gelu", want=("y", "pre"))
            grads = t.linear_weight_backward(dy, x, want=("dW", "dbias"))
            return [*out.values(), t.linear_backward(dy, W, activation="none", dsum=x), *grads.values()]
        first = call()
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        own = t.linear(x, W, bias=b, activation="gelu", want=("y", "pre"), stream=side)
        torch.cuda.synchronize()
        assert torch.equal(own["y"], first[0]) and torch.equal(own["pre"], first[1])
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            held = call()
        x0 = x.clone()
        x.mul_(-0.5)
        graph.replay()
        torch.cuda.synchronize()
        changed = [h.clone() for h in held]
        for a, c in zip(call(), changed):
            assert torch.equal(a, c)
        x.copy_(x0)
        for _ in range(3):
            graph.replay()
        torch.cuda.synchronize()
        for a, c in zip(first, held):
            assert torch.equal(a, c)
        t.last_device_status()


@pytest.mark.parametrize("M,N,K", [(5000, 2056, 136), (4608, 2304, 64), (9000, 1000, 520)])
def test_many_tiles(M, N, K):
    """Tiles that two SMs share and CTAs that finish several, with last rows and columns that fill a tile in part."""
    x, W, b, r, pre, dy, ds = tensors("bf16", 17, (M, K), (N, K), (N,), (M, N), (M, N), (M, K), (M, N))
    W *= K ** -0.5
    X, WW, bb, rr, P, D, S = (f64(t) for t in (x, W, b, r, pre, dy, ds))
    with B.Tokens(M, 64, 64) as t:
        out = t.linear(x, W, bias=b, activation="gelu", residual=r, want=("y", "pre"))
        # the same sizes for the gradient: its output is [M, N] too, its sum runs over K
        dx = t.linear_backward(x, W.t().contiguous(), activation="silu", pre=pre, dsum=ds)
        g = t.linear_weight_backward(ds, x, want=("dW", "dbias"))
        torch.cuda.synchronize()
        t.last_device_status()
    z, y = O.linear(X, WW, bb, "gelu", rr)
    e = product_error("bf16", X, WW.T, np.abs(bb))
    close(out["pre"], z, e, "bf16")
    close(out["y"], y, 1.13 * e + 2.0 ** -19 * np.abs(O.act_value("gelu", z)) + 2.0 ** -126, "bf16")
    plain, ref = O.linear_backward(X, WW.T, "none", None, None), O.linear_backward(X, WW.T, "silu", P, S)
    slope = np.abs(O.act_slope("silu", P))
    close(dx, ref, slope * product_error("bf16", X, WW.T) + 2.0 ** -19 * np.abs(plain) * np.maximum(slope, np.abs(P) * np.exp(-np.abs(P))), "bf16")
    dW, db = O.linear_weight_backward(S, X)
    close(g["dW"], dW, product_error("bf16", S.T, X), "f32")
    close(g["dbias"], db, product_error("bf16", S.T, np.ones((M, 1)))[:, 0], "f32")


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("M,N,K", [(8, 64, 64), (100, 136, 1024), (2500, 2304, 256), (300, 257, 65)])
def test_an_expired_wait_is_reported(io, M, N, K):
    """A bound of one nanosecond lets the waits of the tile kernels run out: the call returns, the status says so, and the next
    call with the bound as it was is right."""
    x, W, dy, ds = tensors(io, 19, (M, K), (N, K), (M, N), (M, K))
    with B.Tokens(M, 64, 64, io=io) as t:
        ref = t.linear(x, W)["y"], t.linear_backward(dy, W, dsum=ds), t.linear_weight_backward(dy, x)["dW"]
        t.set_option(B.PRISM_OPT_WAIT_NS, 1)
        for call in (lambda: t.linear(x, W, residual=dy), lambda: t.linear_backward(dy, W, activation="gelu", pre=x, dsum=ds), lambda: t.linear_weight_backward(dy, x, want=("dW", "dbias"))):
            call()
            torch.cuda.synchronize()
            try:
                t.last_device_status()
            except B.PrismError as e:
                assert e.status == B.PRISM_ERR_TIMEOUT
        t.set_option(B.PRISM_OPT_WAIT_NS, 0)
        again = t.linear(x, W)["y"], t.linear_backward(dy, W, dsum=ds), t.linear_weight_backward(dy, x)["dW"]
        torch.cuda.synchronize()
        t.last_device_status()
    assert all(torch.equal(a, b) for a, b in zip(ref, again))
