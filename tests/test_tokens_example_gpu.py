"""The example runs the token operators together with the layer: training learns, serving follows."""
import importlib.util
import os

import pytest
import torch

from ssm_sequence_layer_gb300 import build

pytestmark = pytest.mark.gpu
PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "next_item.py")


@pytest.fixture(scope="module")
def example():
    build.build()
    spec = importlib.util.spec_from_file_location("next_item", PATH)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def test_next_item_model_learns_and_serves(example):
    model = example.Model().cuda()
    losses, follows = example.train(model, 60)
    # a model that knows nothing loses log V = 6.9 nats an item; one that has the rule loses less than half
    assert losses[0] > 6.0 and losses[-1] < 3.5, losses
    last, items, alternatives, reference = example.serve(model, follows)
    assert items.shape == (example.B, 16) and torch.all((items >= 0) & (items < example.V))
    assert torch.all(alternatives[..., :-1] >= alternatives[..., 1:])
    chain = torch.cat([last[:, None], items], 1)
    assert (follows[chain[:, :-1]] == chain[:, 1:]).float().mean() > 0.5


def test_gradients_agree_with_torch(example):
    """One step's parameter gradients against the same model in fp32 torch, the layer token by token."""
    B, T, H, DK, D, V = example.B, example.T, example.H, example.DK, example.D, example.V
    model = example.Model().cuda()
    g = torch.Generator(device="cuda").manual_seed(5)
    ids = torch.randint(0, V, (B, T + 1), generator=g, device="cuda")
    conv_w = torch.zeros(H, 4, DK, dtype=torch.bfloat16, device="cuda")
    with example.binding.Tokens(B * T, D, V, io="bf16") as tokens, example.binding.Plan(B, H, T, DK, DK, 1, io="bf16") as plan:
        logits = model(tokens, plan, conv_w, ids[:, :-1].contiguous())
        logprob, entropy = example.TokenLogprobs.apply(tokens, logits, ids[:, 1:].reshape(-1).contiguous())
        (-logprob.mean() - 0.01 * entropy.mean()).backward()
        torch.cuda.synchronize()
    got = {k: p.grad.clone() for k, p in model.named_parameters()}
    model.zero_grad()

    def norm(x, w):
        return x * torch.rsqrt((x * x).mean(-1, keepdim=True) + 1e-6) * w

    e = model.table[ids[:, :-1]]
    y = norm(e, model.w_in)
    q, k, v = (y @ model.proj.t()).view(B, T, 3, H, DK).unbind(2)
    q, k = (torch.nn.functional.normalize(x, dim=-1) for x in (q, k))
    b, a = (y @ model.gates.t()).view(B, T, 2, H).unbind(2)
    b, a = torch.sigmoid(b), torch.exp(-torch.nn.functional.softplus(a) / 16)
    S, outs = torch.zeros(B, H, DK, DK, device="cuda"), []
    for t in range(T):
        kt, vt = k[:, t], v[:, t]
        gate, beta = a[:, t, :, None, None], b[:, t, :, None, None]
        Sk = torch.einsum("bhvk,bhk->bhv", S, kt)
        S = gate * (S - beta * Sk[..., None] * kt[..., None, :]) + beta * vt[..., None] * kt[..., None, :]
        outs.append(torch.einsum("bhvk,bhk->bhv", S, q[:, t]))
    o = torch.stack(outs, 1).reshape(B, T, H * DK) @ model.o.t()
    logp = torch.log_softmax(norm(o + e, model.w_out) @ model.table.t(), -1)
    loss = -logp.gather(-1, ids[:, 1:, None]).mean() + 0.01 * (logp.exp() * logp).sum(-1).mean()
    loss.backward()
    for key, p in model.named_parameters():
        # bf16 activations between the operators: a few roundings of 2^-9 relative on each path, which add up
        # without a direction over 2048 tokens
        err = (got[key] - p.grad).norm() / p.grad.norm()
        assert err < 0.05, (key, err.item())
