"""The token operators' fp64 oracle (oracle/prism_tokens.py) against torch in float64, gradients against its
differentiation, so that what the kernels are compared with is held by something else.  Both sides compute in float64
with sums of at most some hundred terms: 1e-11 relative to the largest value leaves their roundings room."""
import numpy as np
import pytest
import torch

from oracle import prism_tokens as O

F = torch.float64


def near(got, ref):
    ref = ref.detach().numpy() if isinstance(ref, torch.Tensor) else ref
    assert np.array_equal(np.isinf(got), np.isinf(ref)) and np.array_equal(got[np.isinf(got)], ref[np.isinf(ref)])
    ok = np.isfinite(ref)
    assert np.max(np.abs(got - ref)[ok], initial=0) <= 1e-11 * (1 + np.max(np.abs(ref[ok]), initial=0))


def test_e4m3_is_the_nearest_value():
    every = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double()
    every = torch.unique(every[torch.isfinite(every)])
    middle = (every[1:] + every[:-1]) / 2
    g = torch.Generator().manual_seed(0)
    x = torch.cat([every, middle, middle * (1 + 2 ** -20), middle * (1 - 2 ** -20),
                   (torch.randn(20000, generator=g).double() * 60).clamp(-448, 448), torch.randn(20000, generator=g).double() * 0.01])
    x = x.float()  # torch rounds from float32, to which all but the random values are exact
    assert np.array_equal(O.e4m3(x.double().numpy()), x.to(torch.float8_e4m3fn).double().numpy())
    assert np.array_equal(O.e4m3(np.array([449.0, -1e30])), [448.0, -448.0])


def test_embedding_and_its_gradient():
    g = torch.Generator().manual_seed(1)
    table = torch.randn(11, 6, generator=g, dtype=F).requires_grad_()
    ids, dout = torch.randint(-1, 11, (40,), generator=g), torch.randn(40, 6, generator=g, dtype=F)
    out = 1.5 * torch.nn.functional.embedding(ids.clamp_min(0), table) * (ids >= 0)[:, None]
    near(O.embed(ids.numpy(), table.detach().numpy(), 1.5), out)
    out.backward(dout)
    near(O.embed_backward(ids.numpy(), dout.numpy(), 1.5, 11), table.grad)
    onto = torch.randn(11, 6, generator=g, dtype=F)
    near(O.embed_backward(ids.numpy(), dout.numpy(), 1.5, 11, onto.numpy()), table.grad + onto)
    beyond = np.array([12, 11, -7, 3])
    assert np.count_nonzero(O.embed(beyond, table.detach().numpy(), 1.0).any(axis=1)) == 1


@pytest.mark.parametrize("D", [5, 128, 300])
def test_norm_and_its_gradient(D):
    g = torch.Generator().manual_seed(D)
    x, res, dy, ds = (torch.randn(7, D, generator=g, dtype=F) for _ in range(4))
    w = torch.randn(D, generator=g, dtype=F).requires_grad_()
    r = (x + res).requires_grad_()
    y = r * torch.rsqrt(r.square().mean(1, keepdim=True) + 1e-3) * w
    got = O.norm(x.numpy(), res.numpy(), w.detach().numpy(), 1e-3)
    near(got[0], r)
    near(got[1], y)
    blocks = torch.nn.functional.pad(y, (0, -D % 128)).view(7, -1, 128)
    near(got[2], (blocks.abs().amax(2) / 448).clamp_min(2.0 ** -126))
    ((y * dy).sum() + (r * ds).sum()).backward()
    dx, dw = O.norm_backward(r.detach().numpy(), w.detach().numpy(), 1e-3, dy.numpy(), ds.numpy())
    near(dx, r.grad)
    near(dw, w.grad)
    assert np.all(O.norm(np.zeros((1, D)), None, np.ones(D), 1e-3)[2] == 2.0 ** -126)


@pytest.mark.parametrize("c", [1.0, 0.75])
def test_log_probabilities_and_their_gradient(c):
    g = torch.Generator().manual_seed(3)
    n, V, k = 9, 50, 6
    x = torch.randn(n, V, generator=g, dtype=F) * 3
    masked = torch.rand(n, V, generator=g) < 0.3
    targets = torch.randint(0, V, (n,), generator=g)
    targets[4] = -1
    masked[torch.arange(n), targets.clamp_min(0)] = False
    x[masked] = float("-inf")
    x[2, masked[2]] = O.LOWEST  # as a mask's value
    z = x.clone()
    z[masked] = float("-inf")
    z = z.requires_grad_()
    logp = torch.log_softmax(c * z, 1)
    live = (targets >= 0).to(F)
    logprob = logp.gather(1, targets.clamp_min(0)[:, None])[:, 0] * live
    entropy = -(logp.exp() * logp.masked_fill(masked, 0.0)).sum(1)
    out = O.token_logprobs(x.numpy(), targets.numpy(), c, k)
    near(out["lse"], torch.logsumexp(c * z, 1))
    near(out["logprob"], logprob)
    near(out["entropy"], entropy)
    top = torch.topk(logp, k, dim=1)
    near(out["top_logprob"], top.values)
    assert np.array_equal(out["top_ids"], top.indices.numpy())  # no two of the logits are equal
    a, b = torch.randn(n, generator=g, dtype=F), torch.randn(n, generator=g, dtype=F)
    ((logprob * a).sum() + (entropy * b).sum()).backward()
    got = O.token_logprobs_backward(x.numpy(), targets.numpy(), c, out["lse"], out["entropy"], a.numpy(), b.numpy())
    near(got, torch.where(masked, 0.0, z.grad))
    near(O.token_logprobs_backward(x.numpy(), None, c, out["lse"], out["entropy"], None, b.numpy()),
         O.token_logprobs_backward(x.numpy(), np.full(n, -1), c, out["lse"], out["entropy"], a.numpy(), b.numpy()))


def test_ties_masks_and_rows_without_a_value():
    inf, nan = float("inf"), float("nan")
    x = np.array([[1.0, 2.0, 2.0, 1.0], [-inf, -inf, O.LOWEST, -inf], [nan, 3.0, -inf, 9.0], [0.0, inf, 1.0, 2.0]])
    out = O.token_logprobs(x, np.array([0, 1, 3, 2]), 1.0, 4)
    assert out["top_ids"].tolist() == [[1, 2, 0, 3], [-1] * 4, [0, 3, 1, -1], [1, 3, 2, 0]]
    assert out["lse"][1] == -inf and out["entropy"][1] == 0 and out["logprob"][1] == -inf
    assert np.isnan(out["lse"][2:]).all() and np.isnan(out["logprob"][2:]).all() and np.isnan(out["entropy"][2:]).all()
    assert not O.token_logprobs_backward(x[1:2], np.array([1]), 1.0, out["lse"][1:2], out["entropy"][1:2], np.ones(1), np.ones(1)).any()


def test_products_that_overflow_in_float32_are_masked():
    out = O.token_logprobs(np.array([[-2e38, 1.0, -1.7e38]]), np.array([0]), 2.0, 3)
    assert out["logprob"][0] == -np.inf and out["top_ids"].tolist() == [[1, 2, -1]]
    d = O.token_logprobs_backward(np.array([[-2e38, 1.0, 0.0]]), np.array([0]), 2.0, out["lse"], out["entropy"], np.ones(1), None)
    assert d[0, 0] == 0 and d[0, 1] < 0
