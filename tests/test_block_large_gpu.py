"""Tensors of more than 2^31 values: the first and the last rows come out as the same rows of a small call do, bit for bit where the sums are the
same, and the sums over rows as two halves' sums do."""
import pytest
import torch

from ssm_sequence_layer_gb300 import binding as B
from ssm_sequence_layer_gb300 import build

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(scope="module", autouse=True)
def _built():
    build.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    yield
    torch.cuda.empty_cache()


def normal(io, *shape):
    """Normal values, made in pieces of rows."""
    x = torch.empty(*shape, dtype=DT[io], device="cuda")
    for part in x.split(1 << 18):
        part.normal_()
    return x


@pytest.mark.parametrize("io,K", [("bf16", 1040), ("bf16", 1033), ("f32", 1040)])
def test_products_with_far_rows(io, K):
    torch.manual_seed(1)
    M, N = (1 << 21) + 7, 40
    x, W, dy = normal(io, M, K), normal(io, N, K) * 0.03, normal(io, M, N)
    rows = torch.cat([torch.arange(70), torch.arange(M - 70, M)]).cuda()
    with B.Tokens(M, 64, 64, io=io) as t:
        y = t.linear(x, W)["y"]
        dx = t.linear_backward(dy, W, activation="silu", pre=x, dsum=x)
        dW = t.linear_weight_backward(dy, x)["dW"]
        half = M // 2 // 8 * 8
        parts = t.linear_weight_backward(dy[:half], x[:half])["dW"].double() + t.linear_weight_backward(dy[half:], x[half:])["dW"].double()
        few = x[rows].contiguous()
        ref_y, ref_dx = t.linear(few, W)["y"], t.linear_backward(dy[rows].contiguous(), W, activation="silu", pre=few, dsum=few)
        torch.cuda.synchronize()
        t.last_device_status()
    # sums of K or N products in two orders: each within (K + 8) 2^-24 of the sum of magnitudes, and a rounding to the type
    eps = torch.finfo(DT[io]).eps
    for got, ref, size in ((y[rows], ref_y, few.float().abs() @ W.float().abs().t()), (dx[rows], ref_dx, dy[rows].float().abs() @ W.float().abs() * 1.1)):
        assert torch.all((got.float() - ref.float()).abs() <= 2 * (K + 8) * 2.0 ** -24 * size + 2.0 ** -19 * size + eps * ref.float().abs())
    # sums of 2^21 products of normal numbers are about 1400 large, and so is what half of the rows make of them: within a thousandth of that
    assert torch.all((dW.double() - parts).abs() <= 2.0 ** -10 * M ** 0.5)


@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_heads_with_far_rows(io):
    torch.manual_seed(2)
    Bn, T, d, heads = 2, (1 << 20) + 3, 128, (4, 2, 3)
    x = normal(io, Bn * T, 9 * d).view(Bn, T, 9 * d)
    form = dict(heads=heads, d=d, norm="rms", inv_freq=torch.logspace(0, -4, 64, device="cuda"))
    with B.Tokens(Bn * T, 64, 8, io=io) as t:
        out = t.heads(x, **form)
        back = t.heads_backward(x, {"dq": out["q"], "dk": out["k"], "dv": out["v"]}, **form)["dx"]
        for a, b in ((0, 5), (T - 5, T)):
            few = x[:, a:b].contiguous()
            positions = torch.arange(a, b, device="cuda").repeat(Bn, 1)
            ref = t.heads(few, positions=positions, **form)
            for key in out:
                assert torch.equal(out[key][:, :, a:b], ref[key])
            grads = {"d" + key: ref[key] for key in ref}
            assert torch.equal(back[:, a:b], t.heads_backward(few, grads, positions=positions, **form)["dx"])
        torch.cuda.synchronize()
        t.last_device_status()


@pytest.mark.parametrize("io,n,V", [("bf16", 70001, 32003), ("f32", 9000, 250007)])
def test_draws_of_far_rows(io, n, V):
    torch.manual_seed(3)
    x, u = normal(io, n, V), torch.rand(n, device="cuda")
    rows = torch.cat([torch.arange(3), torch.arange(n - 3, n)]).cuda()
    with B.Tokens(n, 64, V, io=io) as t:
        out, ref = t.sample(x, u, 1.5, 50, 0.9), t.sample(x[rows].contiguous(), u[rows].contiguous(), 1.5, 50, 0.9)
        torch.cuda.synchronize()
        t.last_device_status()
    assert all(torch.equal(out[key][rows], ref[key]) for key in out)
