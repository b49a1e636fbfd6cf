"""The block's operators as a model uses them: a block with its layer and its feed-forward in training, every parameter's gradient against
torch in 64 bits, and in serving, one token at a time and from a graph, against the whole sequence at once.

Tolerance of the gradients: a path from a parameter to the loss passes through at most 16 operators, each within 2^-17 of its
result's size in float32 (sums of at most some hundred terms, exponentials and roots of a few units in the last place), and none of
these, with rows of length one, gates below one and norms, makes an error more than some times larger on its way:
16 2^-17 times 8 is 1e-3."""
import numpy as np
import pytest
import torch

from ssm_sequence_layer_gb300 import binding as Bd
from ssm_sequence_layer_gb300 import build
from ssm_sequence_layer_gb300.rotary import rotary_frequencies

pytestmark = pytest.mark.gpu
B, T, H, DK, D, F, V = 2, 40, 2, 64, 128, 192, 300


@pytest.fixture(scope="module", autouse=True)
def _built():
    build.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"


def parameters(dtype=torch.float32):
    g = torch.Generator().manual_seed(0)
    r = lambda *s, std: (torch.randn(*s, generator=g) * std).to(dtype).cuda()  # noqa: E731
    return {"table": r(V, D, std=0.5), "n1": 1 + r(D, std=0.1), "n2": 1 + r(D, std=0.1), "n3": 1 + r(D, std=0.1), "qkv": r(3 * H * DK, D, std=D ** -0.5), "qkv_b": r(3 * H * DK, std=0.1),
            "q_w": 1 + r(DK, std=0.1), "k_w": (1 + r(DK, std=0.1)) * 0.8, "o": r(D, H * DK, std=(H * DK) ** -0.5), "up": r(F, D, std=D ** -0.5), "up_b": r(F, std=0.1),
            "down": r(D, F, std=F ** -0.5), "down_b": r(D, std=0.1)}


def gates():
    g = torch.Generator().manual_seed(1)
    beta = torch.sigmoid(torch.randn(B, H, T, generator=g)).cuda()
    return beta, (0.9 + 0.1 * torch.rand(B, H, T, generator=g)).cuda()


def form(p, positions=None):
    inv_freq, amplitude = rotary_frequencies(32, scaling="by parts", factor=4, original_length=64, device="cuda")
    # rows of length about one after the norm's weights (the amplitude turns the first half only)
    return dict(heads=(H, H, H), d=DK, norm="unit", q_weight=p["q_w"], k_weight=p["k_w"], inv_freq=inv_freq, amplitude=amplitude, positions=positions)


def run_forward(t, plan, p, ids, beta, alpha, keep):
    e = t.embed(ids, p["table"]).view(-1, D)
    y1 = t.norm(e, p["n1"])["y"]
    rows = t.linear(y1, p["qkv"], bias=p["qkv_b"])["y"].view(B, T, -1)
    h = t.heads(rows, **form(p))
    conv_w = torch.zeros(H, 4, DK, dtype=e.dtype, device="cuda")
    inp = {"q": h["q"], "k": h["k"], "v": h["v"], "beta": beta, "alpha": alpha, "u": None, "gamma": None, "eta": None, "conv_w": conv_w, "L": 1}
    o = plan.forward(inp).transpose(1, 2).reshape(-1, H * DK).contiguous()
    r = t.linear(o, p["o"], residual=e)["y"]
    y2 = t.norm(r, p["n2"])["y"]
    up = t.linear(y2, p["up"], bias=p["up_b"], activation="gelu", want=("y", "pre"))
    s = t.linear(up["y"], p["down"], bias=p["down_b"], residual=r)["y"]
    y3 = t.norm(s, p["n3"])["y"]
    logits = t.linear(y3, p["table"])["y"]
    keep.update(e=e, y1=y1, rows=rows, inp=inp, o=o, r=r, y2=y2, up=up, s=s, y3=y3, logits=logits)
    return logits


def run_backward(t, plan, p, ids, targets, k):
    out = t.token_logprobs(k["logits"], targets)
    n = targets.numel()
    g = {}
    dl = t.token_logprobs_backward(k["logits"], targets, out["lse"], None, torch.full((n,), -1.0 / n, device="cuda"))
    onto = {"dW": torch.zeros(V, D, device="cuda")}
    t.linear_weight_backward(dl, k["y3"], out=onto, accumulate=True)  # the head shares the embedding's table
    d = t.norm_backward(k["s"], p["n3"], t.linear_backward(dl, p["table"]))
    ds, g["n3"] = d["dx"], d["dweight"]
    w = t.linear_weight_backward(ds, k["up"]["y"], want=("dW", "dbias"))
    g["down"], g["down_b"] = w["dW"], w["dbias"]
    dpre = t.linear_backward(ds, p["down"], activation="gelu", pre=k["up"]["pre"])
    w = t.linear_weight_backward(dpre, k["y2"], want=("dW", "dbias"))
    g["up"], g["up_b"] = w["dW"], w["dbias"]
    d = t.norm_backward(k["r"], p["n2"], t.linear_backward(dpre, p["up"]), dsum=ds)
    dr, g["n2"] = d["dx"], d["dweight"]
    g["o"] = t.linear_weight_backward(dr, k["o"])["dW"]
    do = t.linear_backward(dr, p["o"]).float().view(B, T, H, DK).transpose(1, 2).contiguous()
    back = plan.backward(k["inp"], do)
    h = t.heads_backward(k["rows"], back, **form(p))
    g["q_w"], g["k_w"] = h["dq_weight"], h["dk_weight"]
    drows = h["dx"].view(-1, 3 * H * DK)
    w = t.linear_weight_backward(drows, k["y1"], want=("dW", "dbias"))
    g["qkv"], g["qkv_b"] = w["dW"], w["dbias"]
    d = t.norm_backward(k["e"], p["n1"], t.linear_backward(drows, p["qkv"]), dsum=dr)
    g["n1"] = d["dweight"]
    g["table"] = t.embed_backward(ids, d["dx"].view(*ids.shape, D), dtable=onto["dW"], accumulate=True)
    return out["logprob"], g


def reference(p, ids, targets, beta, alpha):
    p = {k: v.double().detach().requires_grad_() for k, v in p.items()}
    norm = lambda x, w: x * torch.rsqrt((x * x).mean(-1, keepdim=True) + 1e-6) * w  # noqa: E731
    e = p["table"][ids]
    rows = norm(e, p["n1"]) @ p["qkv"].t() + p["qkv_b"]
    q, k, v = rows.view(B, T, 3, H, DK).unbind(2)
    f = form(p)
    angle = torch.arange(T, device="cuda").double()[:, None, None] * f["inv_freq"].double()

    def head(x, w):
        x = x * torch.rsqrt((x * x).sum(-1, keepdim=True) + 1e-6) * w
        a, b, rest = x[..., :16], x[..., 16:32], x[..., 32:]
        c, s = torch.cos(angle) * f["amplitude"], torch.sin(angle) * f["amplitude"]
        return torch.cat([a * c - b * s, a * s + b * c, rest], -1)

    q, k = head(q, p["q_w"]), head(k, p["k_w"])
    S, outs = torch.zeros(B, H, DK, DK, device="cuda", dtype=torch.float64), []
    for t in range(T):
        be, al = beta[:, :, t, None, None].double(), alpha[:, :, t, None, None].double()
        Sk = torch.einsum("bhvk,bhk->bhv", S, k[:, t])
        S = al * (S - be * Sk[..., None] * k[:, t][..., None, :]) + be * v[:, t][..., None] * k[:, t][..., None, :]
        outs.append(torch.einsum("bhvk,bhk->bhv", S, q[:, t]))
    r = torch.stack(outs, 1).reshape(B, T, H * DK) @ p["o"].t() + e
    up = norm(r, p["n2"]) @ p["up"].t() + p["up_b"]
    s = torch.nn.functional.gelu(up) @ p["down"].t() + p["down_b"] + r
    logits = norm(s, p["n3"]) @ p["table"].t()
    logprob = torch.log_softmax(logits, -1).gather(-1, targets[..., None])[..., 0]
    (-logprob.mean()).backward()
    return logits.detach(), logprob.detach(), {k: v.grad for k, v in p.items()}


def test_a_block_in_training():
    p, (beta, alpha) = parameters(), gates()
    g = torch.Generator().manual_seed(2)
    ids, targets = torch.randint(0, V, (B, T), generator=g).cuda(), torch.randint(0, V, (B, T), generator=g).cuda()
    with Bd.Tokens(B * T, D, V, io="f32") as t, Bd.Plan(B, H, T, DK, DK, 1, io="f32") as plan:
        keep = {}
        run_forward(t, plan, p, ids, beta, alpha, keep)
        logprob, grads = run_backward(t, plan, p, ids, targets.view(-1), keep)
        torch.cuda.synchronize()
        t.last_device_status()
        plan.last_device_status()
    logits, ref, rgrads = reference(p, ids, targets, beta, alpha)
    assert torch.max(torch.abs(keep["logits"].view(B, T, V) - logits)) <= 1e-3 * logits.square().mean().sqrt()
    assert torch.max(torch.abs(logprob.view(B, T) - ref)) <= 1e-3 * ref.abs().max()
    assert set(grads) == set(rgrads)
    for key, r in rgrads.items():
        err = torch.max(torch.abs(grads[key] - r)) / r.square().mean().sqrt()
        assert err <= 1e-2, (key, err.item())  # the largest of some thousand against the root mean square
        assert (grads[key] - r).norm() <= 1e-3 * r.norm(), key


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_a_block_in_serving(io):
    """Token by token with a carried state, the same step from a graph, against the prompt at once."""
    dtype = torch.float32 if io == "f32" else torch.bfloat16
    p, (beta, alpha) = parameters(dtype), gates()
    g = torch.Generator().manual_seed(3)
    ids, u = torch.randint(0, V, (B, T), generator=g).cuda(), torch.rand(B, generator=g).cuda()
    conv_w = torch.zeros(H, 4, DK, dtype=dtype, device="cuda")
    with Bd.Tokens(B * T, D, V, io=io, logits="f32") as t, Bd.Plan(B, H, T, DK, DK, 1, io=io) as plan:
        keep = {}
        whole = run_forward(t, plan, p, ids, beta, alpha, keep).view(B, T, V).float()
        S, hist = torch.zeros(B, H, DK, DK, device="cuda"), torch.zeros(B, H, 3, DK, dtype=dtype, device="cuda")
        tok, pos = torch.zeros(B, dtype=torch.int64, device="cuda"), torch.zeros(B, 1, dtype=torch.int64, device="cuda")
        gate = {"beta": torch.zeros(B, H, device="cuda"), "alpha": torch.zeros(B, H, device="cuda")}
        w8, w_scale = t.matmul8_weights(p["table"])

        def step():
            e = t.embed(tok, p["table"])
            rows = t.linear(t.norm(e, p["n1"])["y"], p["qkv"], bias=p["qkv_b"])["y"].view(B, 1, -1)
            h = t.heads(rows, **made)
            inp = {"q": h["q"], "k": h["k"], "v": h["v"], "u": None, "gamma": None, "eta": None, "conv_w": conv_w, "L": 1, **gate}
            o = plan.decode_step(inp, hist, S, stream=torch.cuda.current_stream()).reshape(B, H * DK)
            r = t.linear(o, p["o"], residual=e)["y"]
            s = t.linear(t.linear(t.norm(r, p["n2"])["y"], p["up"], bias=p["up_b"], activation="gelu")["y"], p["down"], bias=p["down_b"], residual=r)["y"]
            y = t.norm(s, p["n3"], want=("y", "y8"))
            logits8 = t.matmul8(y["y8"], y["y_scale"], w8, w_scale)
            drawn = t.sample(logits8, u, *rules)
            return h, t.linear(y["y"], p["table"])["y"], drawn["ids"], logits8

        made = form(p, pos)  # the frequencies once: a program keeps them
        rules = torch.full((B,), 0.8, device="cuda"), torch.full((B,), 20, dtype=torch.int32, device="cuda"), torch.full((B,), 0.9, device="cuda")

        def put(i):
            tok.copy_(ids[:, i]), pos.fill_(i), gate["beta"].copy_(beta[:, :, i]), gate["alpha"].copy_(alpha[:, :, i])

        put(0)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):  # the first run outside of the graph, on the stream that is captured
            step()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            held = step()
        S.zero_(), hist.zero_()
        # roundings of the io type on both ways, a path of about ten of them
        tol = 1e-4 if io == "f32" else 10 * 2.0 ** -8
        for i in range(T):
            put(i)
            graph.replay()
            torch.cuda.synchronize()
            h, logits, drawn, logits8 = held
            assert (logits.float() - whole[:, i]).abs().max() <= tol * whole.square().mean().sqrt() * 4, i
            # the same number with the same rules draws the same token from the same logits
            again = t.sample(logits8, u, *rules)
            assert torch.equal(again["ids"], drawn) and torch.all((drawn >= 0) & (drawn < V))
        if io == "f32":  # single rows go through the same sums as the prompt's
            assert torch.allclose(h["q"][:, :, 0], keep["inp"]["q"][:, :, T - 1], atol=1e-6)
        t.last_device_status()
        plan.last_device_status()


@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_two_handles_on_two_streams(io):
    """Calls that run beside each other, each with a handle and a stream of its own, leave the bits that they leave alone."""
    dt = {"bf16": torch.bfloat16, "f32": torch.float32}[io]
    g = torch.Generator().manual_seed(3)

    def side(M, N, K, V):
        new = lambda *s: torch.randn(*s, generator=g).to(dt).cuda()  # noqa: E731
        t = Bd.Tokens(M, 64, V, io=io)
        x, W, dy, logits = new(M, K), new(N, K), new(M, N), new(M, V)
        u, p = torch.rand(M, generator=g).cuda(), torch.full((M,), 0.7, device="cuda")

        def calls(stream=None):
            out = [t.linear(x, W, activation="gelu", want=("y", "pre"), stream=stream)]
            out.append({"dx": t.linear_backward(dy, W, stream=stream)})
            out.append(t.linear_weight_backward(dy, x, stream=stream))
            out.append(t.sample(logits, u, top_p=p, stream=stream))
            return {f"{i} {key}": value for i, d in enumerate(out) for key, value in d.items()}
        return t, calls
    sides = [side(300, 257, 259, 5003), side(40, 768, 768, 2000)]
    alone = [calls() for _, calls in sides]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sides]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    runs = [[calls(stream) for (_, calls), stream in zip(sides, streams)] for _ in range(10)]
    torch.cuda.synchronize()
    for run in runs:
        for got, want in zip(run, alone):
            assert all(torch.equal(got[key], want[key]) for key in want)
    for t, _ in sides:
        t.last_device_status()
        t.close()
