"""The 8-bit product with a scale for each block of 128, and the weights' layout, against the fp64 oracle.

Tolerances, with u = 2^-24 and S = sum_k |a_scale a8 w_scale w8| of an output: products of e4m3 values
are exact in fp32.  A block's sum has at most 128 additions, each within 2 u of the partial sums' magnitude
(tensor cores may truncate where they do not round), the joins of blocks and the scales' product add KB + 4 roundings:
(2 * 128 + KB + 4) u S; plus half a unit in the last place of the output's type.
Weights: w_scale within u of max / 448 relatively (one division); w8 w_scale within half a step of e4m3."""
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


@pytest.fixture(scope="module", autouse=True)
def _built():
    build.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"


def f64(t):
    return t.float().cpu().double().numpy()


def draw(M, N, K, seed):
    g = torch.Generator().manual_seed(seed)
    kb, nb = -(-K // 128), -(-N // 128)
    a8 = (torch.randn(M, K, generator=g) * 60).clamp_(-448, 448).to(torch.float8_e4m3fn)
    w8 = (torch.randn(N, K, generator=g) * 60).clamp_(-448, 448).to(torch.float8_e4m3fn)
    sa = torch.exp(torch.randn(M, kb, generator=g)) / 400
    sw = torch.exp(torch.randn(nb, kb, generator=g)) / 400
    return a8.cuda(), sa.cuda(), w8.cuda(), sw.cuda()


def reference(a8, sa, w8, sw):
    K, N = a8.shape[1], w8.shape[0]
    col, row = np.arange(K) // 128, np.arange(N) // 128
    a, w = f64(a8) * f64(sa)[:, col], f64(w8) * f64(sw)[row][:, col]
    return a @ w.T, np.abs(a) @ np.abs(w).T


SHAPES = [(1, 1, 16), (1, 64, 64), (1, 1000, 768), (4, 777, 272), (8, 5000, 128), (9, 130, 400), (16, 640, 1040), (17, 129, 144),
          (24, 96, 4096), (31, 3000, 256), (33, 500, 768), (64, 2048, 512), (65, 333, 128), (100, 256, 2064), (127, 129, 144), (128, 128, 128),
          (129, 257, 1040), (200, 40, 768), (256, 512, 384), (300, 4626, 256), (1000, 136, 160), (2050, 264, 768), (5000, 16, 64), (1000, 5000, 400),
          (1100, 6000, 272), (200, 20000, 144), (384, 30000, 128), (5000, 1111, 400), (3, 100, 4096), (12, 40, 8192), (2, 20000, 528), (8, 2500, 1024), (16, 33, 2000), (17, 3000, 512),
          (40, 130, 2000), (257, 515, 1600), (1000, 1000, 1536), (20, 7, 16384),
          (9, 3700, 272), (16, 20011, 1040), (13, 5000, 2064), (8, 9001, 4096), (5, 50048, 160), (11, 40001, 128), (7, 8000, 784)]


@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_matmul8(out, M, N, K):
    a8, sa, w8, sw = draw(M, N, K, M + N + K)
    with B.Tokens(M, 64, 64, io="bf16", logits=out) as t:
        got = torch.full((M + 2, N), 9.0, dtype=DT[out], device="cuda")
        t.matmul8(a8, sa, w8, sw, out=got[:M])
        first = got.clone()
        t.matmul8(a8, sa, w8, sw, out=got[:M])
        torch.cuda.synchronize()
        t.last_device_status()
    assert torch.equal(first, got) and torch.all(got[M:] == 9.0)
    ref, S = reference(a8, sa, w8, sw)
    e = (2 * 128 + -(-K // 128) + 4) * u * S
    half = bf16_half_ulp(np.abs(ref) + e) if out == "bf16" else u * np.abs(ref)
    assert np.all(np.abs(f64(got[:M]) - ref) <= e + half)


def test_sums_keep_32_bits():
    """One large product among small ones: 448 * 448 = 200704 < 2^18 and 127 times 2^-6.  Every partial
    sum is a multiple of 2^-6 below 2^18, so it has 24 bits: sums held in fp32 are exact in any order, and
    sums held in fewer bits would drop small products."""
    M, N, K = 130, 256, 128
    a8 = torch.full((M, K), 0.125).to(torch.float8_e4m3fn)
    w8 = torch.full((N, K), 0.125).to(torch.float8_e4m3fn)
    a8[:, 77] = 448.0
    w8[:, 77] = 448.0
    for rows in (1, 8, 16, 40, 130):
        with B.Tokens(M, 64, 64, io="f32") as t:
            got = t.matmul8(a8[:rows].cuda(), torch.ones(rows, 1, device="cuda"), w8.cuda(), torch.ones(2, 1, device="cuda"))
        assert torch.all(got == 448.0 * 448.0 + 127 / 64), rows


@pytest.mark.parametrize("M,N", [(600, 1000), (1100, 8000)])
def test_an_expired_wait_is_reported(M, N):
    """With a bound of 1 ns every wait runs out: the status says so, and the handle works again after it."""
    a8, sa, w8, sw = draw(M, N, 768, 1)
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


def test_special_values():
    """NaN stays in its row or column; an infinite scale gives infinities and NaN as the formula does; zeros give zeros."""
    M, N, K = 140, 300, 256
    a8, sa, w8, sw = draw(M, N, K, 0)
    a8[3, 200] = float("nan")
    w8[7, 10] = float("nan")
    a8[5] = 0.0
    for rows in (8, 140):
        with B.Tokens(M, 64, 64, io="f32") as t:
            got = t.matmul8(a8[:rows].contiguous(), sa[:rows].contiguous(), w8, sw).cpu()
        nan = torch.zeros(rows, N, dtype=torch.bool)
        nan[3] = True
        nan[:, 7] = True
        assert torch.equal(torch.isnan(got), nan)
        assert torch.all(got[5, :7] == 0) and torch.all(got[5, 8:] == 0)


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("N,K", [(1, 16), (128, 128), (300, 272), (1000, 768)])
def test_weights(io, N, K):
    g = torch.Generator().manual_seed(N)
    W = (torch.randn(N, K, generator=g) * torch.exp(torch.randn(N, 1, generator=g))).to(DT[io])
    W[0, :16] = 0.0
    with B.Tokens(1, 64, 64, io=io) as t:
        w8, sw = t.matmul8_weights(W.cuda())
    kb, nb = -(-K // 128), -(-N // 128)
    assert w8.dtype is torch.float8_e4m3fn and w8.shape == (N, K) and sw.shape == (nb, kb)
    W64 = f64(W)
    scale = np.array([[max(np.abs(W64[128 * i:128 * i + 128, 128 * j:128 * j + 128]).max() / 448, 2.0 ** -126) for j in range(kb)] for i in range(nb)])
    got = f64(sw)
    assert np.all(np.abs(got - scale) <= u * scale * 1.0001)
    s = got[np.arange(N) // 128][:, np.arange(K) // 128]
    assert np.all(np.abs(f64(w8) * s - W64) <= (2.0 ** -4 * np.abs(W64) + 2.0 ** -10 * s) * 1.0001)


def test_norm_into_the_product():
    """The 8-bit output of the norm is the product's operand."""
    n, D, V = 40, 272, 500
    g = torch.Generator().manual_seed(0)
    x = torch.randn(n, D, generator=g).bfloat16().cuda()
    W = (torch.randn(V, D, generator=g) / D ** 0.5).bfloat16().cuda()
    with B.Tokens(n, D, V, io="bf16", logits="f32") as t:
        q = t.norm(x, torch.ones(D, dtype=torch.bfloat16, device="cuda"), want=("y8",))
        w8, sw = t.matmul8_weights(W)
        got = f64(t.matmul8(q["y8"], q["y_scale"], w8, sw))
    _, y, _ = O.norm(f64(x), None, np.ones(D), 1e-6)
    ref = y @ f64(W).T
    # both operands within 2^-4 of themselves at worst, independent roundings: the sum's error is about
    # sqrt(D) * 2^-5 * the size of one product, far below this bound of the worst case
    assert np.all(np.abs(got - ref) <= (2 * 2.0 ** -4 + 2.0 ** -8) * (np.abs(y) @ np.abs(f64(W)).T))


def test_matmul8_refusals():
    a8, sa, w8, sw = draw(4, 20, 32, 0)
    with B.Tokens(4, 64, 64, io="bf16") as t:
        for bad in (lambda: t.matmul8(a8.float(), sa, w8, sw), lambda: t.matmul8(a8, sa[:2], w8, sw), lambda: t.matmul8(a8, sa, w8[:, :16].contiguous(), sw),
                    lambda: t.matmul8(a8, sa, w8, sw[:0]), lambda: t.matmul8(a8, sa, w8, sw, out=torch.zeros(4, 20, device="cuda")),
                    lambda: t.matmul8_weights(torch.zeros(4, 32, device="cuda"))):
            with pytest.raises(ValueError):
                bad()
        out = torch.zeros(4, 20, dtype=torch.bfloat16, device="cuda")
        for status, bad in (
                (B.PRISM_ERR_UNSUPPORTED, lambda: t.matmul8(*draw(4, 20, 24, 0))),
                (B.PRISM_ERR_INVALID_ARG, lambda: t.matmul8(*draw(5, 20, 32, 0))),
                (B.PRISM_ERR_INVALID_ARG, lambda: B.prism_matmul8(t.handle, 4, 0, 32, a8, sa, w8, sw, out)),
                (B.PRISM_ERR_INVALID_ARG, lambda: B.prism_matmul8(t.handle, 4, 20, 32, a8, None, w8, sw, out)),
                (B.PRISM_ERR_MISALIGNED, lambda: B.prism_matmul8(t.handle, 3, 20, 32, a8.data_ptr() + 8, sa, w8, sw, out))):
            with pytest.raises(B.PrismError) as ei:
                bad()
            assert ei.value.status == status
        assert t.matmul8(a8[:0], sa[:0], w8, sw).shape == (0, 20)
