"""Token operators on tensors whose offsets pass 32 bits.  Rows are independent, so the last rows of a large call
must have the bits of a small call on copies of them; the product is compared with fp64 (its tolerance:
products are exact and K = 16 additions truncate at most, (2 * 16 + 5) u S, plus half a unit of the output)."""
import pytest
import torch

from ssm_sequence_layer_gb300 import binding as B
from ssm_sequence_layer_gb300 import build
from tests.gpu_util import bf16_half_ulp

pytestmark = pytest.mark.gpu
u = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def _built():
    build.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"


@pytest.fixture(autouse=True)
def _memory():
    yield
    torch.cuda.empty_cache()


def rows_apart(n, V, stride, dtype):
    return torch.empty((n - 1) * stride + V, dtype=dtype, device="cuda").as_strided((n, V), (stride, 1))


@pytest.mark.parametrize("k", [0, 5])
def test_logprobs_with_rows_far_apart(k):
    n, V, stride = 4, 20011, 1_000_000_008
    small = torch.randn(n, V).bfloat16().cuda()
    targets = torch.tensor([5, V - 1, -1, 77], device="cuda")
    x = rows_apart(n, V, stride, torch.bfloat16)
    x.copy_(small)
    aligned = rows_apart(n, V, -(-V // 8) * 8, torch.bfloat16)  # the same alignment of rows
    aligned.copy_(small)
    with B.Tokens(n, 8, V, io="bf16") as t:
        got, ref = t.token_logprobs(x, targets, k=k), t.token_logprobs(aligned, targets, k=k)
        for key in ref:
            assert torch.equal(got[key], ref[key]), key
        dlp = torch.randn(n, device="cuda")
        d = t.token_logprobs_backward(aligned, targets, ref["lse"], None, dlp)
        t.token_logprobs_backward(x, targets, ref["lse"], None, dlp, dlogits=x)  # in place
        assert torch.equal(x, d)


def test_embed_large_tables_and_many_tokens():
    D, V, stride = 64, 5, 1_000_000_000
    table = rows_apart(V, D, stride, torch.bfloat16)
    table.copy_(torch.randn(V, D))
    ids = torch.tensor([4, 0, 3, -1, 4], device="cuda")
    with B.Tokens(5, D, V, io="bf16") as t:
        assert torch.equal(t.embed(ids, table), t.embed(ids, table.contiguous()))
    del table
    torch.cuda.empty_cache()
    n, D, V = 2_200_000, 1024, 2_300_000  # n D and V D above 2^31
    ids = torch.full((n,), -1, dtype=torch.int64, device="cuda")
    ids[-3:] = torch.tensor([V - 1, 7, V - 1], device="cuda")
    dout = torch.zeros(n, D, dtype=torch.bfloat16, device="cuda")
    dout[-3:] = torch.randn(3, D, device="cuda")
    with B.Tokens(n, D, V, io="bf16") as t:
        d = t.embed_backward(ids, dout)
        assert torch.equal(d[V - 1], dout[-3].float() + dout[-1].float()) and torch.equal(d[7], dout[-2].float())
        assert d.count_nonzero().item() == d[V - 1].count_nonzero().item() + d[7].count_nonzero().item()
        t.last_device_status()
        out = t.embed(ids, d.bfloat16())
        assert torch.equal(out[-3], d[V - 1].bfloat16()) and torch.equal(out[-2], d[7].bfloat16()) and not out[-4].any()


@pytest.mark.parametrize("D", [1024, 1026])
def test_norm_of_many_rows(D):
    n, last = 2_200_000, 9
    x = torch.zeros(n, D, dtype=torch.bfloat16, device="cuda")
    x[-last:] = torch.randn(last, D, device="cuda")
    w = torch.randn(D, device="cuda").bfloat16()
    dy = torch.zeros_like(x)
    dy[-last:] = torch.randn(last, D, device="cuda")
    with B.Tokens(n, D, 8, io="bf16") as t:
        got, ref = (t.norm(v, w, residual=v, want=("sum", "y", "y8")) for v in (x, x[-last:].clone()))
        for key in ref:
            assert torch.equal(got[key][-last:].view(torch.uint8), ref[key].view(torch.uint8)), key
        del got
        g, r = (t.norm_backward(x[a:].clone() if a else x, w, dy[a:].clone() if a else dy) for a in (0, n - last))
        assert torch.equal(g["dx"][-last:], r["dx"])
        # zeros add nothing, and the parts are sums of at most 9 terms in another order
        assert torch.allclose(g["dweight"], r["dweight"], rtol=0, atol=9 * 2 * u * 9 * 25)


@pytest.mark.parametrize("N", [70000, 70001])
def test_matmul8_large_outputs(N):
    M, K = 33000, 16
    g = torch.Generator(device="cuda").manual_seed(N)
    a8, w8 = (torch.randn(r, K, device="cuda", generator=g).to(torch.float8_e4m3fn) for r in (M, N))
    sa, sw = torch.rand(M, 1, device="cuda", generator=g), torch.rand(-(-N // 128), 1, device="cuda", generator=g)
    with B.Tokens(M, 8, 8, io="bf16") as t:
        out = t.matmul8(a8, sa, w8, sw)
        t.last_device_status()
    a, w = (a8.double() * sa.double())[-300:], (w8.double() * sw.double().repeat_interleave(128, 0)[:N])[-500:]
    ref, S = a @ w.T, a.abs() @ w.abs().T
    e = (2 * 16 + 5) * u * S
    half = torch.from_numpy(bf16_half_ulp((ref.abs() + e).cpu().numpy())).cuda()
    assert torch.all((out[-300:, -500:].double() - ref).abs() <= e + half)


@pytest.mark.parametrize("M", [8, 40])
def test_matmul8_large_operands(M):
    N, K = 70000, 40960
    w8 = torch.zeros(N, K, device="cuda", dtype=torch.uint8).view(torch.float8_e4m3fn)
    w8[-64:].copy_(torch.randint(-8, 9, (64, K), device="cuda").float().to(torch.float8_e4m3fn))
    a8 = torch.randint(-8, 9, (M, K), device="cuda").float().to(torch.float8_e4m3fn)
    sa, sw = torch.ones(M, K // 128, device="cuda"), torch.ones(-(-N // 128), K // 128, device="cuda")
    with B.Tokens(M, 8, 8, io="f32") as t:
        out = t.matmul8(a8, sa, w8, sw)
        t.last_device_status()
    # integers of at most 8 * 8 * 40960 < 2^24: exact
    assert torch.equal(out[:, -64:].double(), a8.double() @ w8[-64:].double().T) and not out[:, :-64].any()
