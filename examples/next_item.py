"""A small next-item model around one recurrent layer: training steps, then serving.

Shows the token operators next to the layer they surround:
  training   ids -> embed -> norm -> (q, k, v, gates) -> recurrence -> norm(+ residual) -> head -> token_logprobs,
             and back through token_logprobs_backward, norm_backward, the layer's backward and embed_backward;
  serving    a prompt carried into the state, then one item at a time: embed -> norm -> decode_step ->
             norm into 8 bits -> matmul8 (the head's weights laid out once) -> token_logprobs with alternatives.

    python examples/next_item.py [--steps 60]

The data is synthetic: item i is followed by item f(i) most of the time.  Needs the GPU.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from ssm_sequence_layer_gb300 import binding, build  # noqa: E402

B, T, H, DK, D, V = 4, 512, 4, 64, 256, 1000
BF16 = torch.bfloat16


class Embed(torch.autograd.Function):
    @staticmethod
    def forward(ctx, tokens, ids, table):
        ctx.tokens, ctx.ids = tokens, ids
        return tokens.embed(ids, table.to(BF16))

    @staticmethod
    def backward(ctx, dout):
        return None, None, ctx.tokens.embed_backward(ctx.ids, dout.contiguous())


class Norm(torch.autograd.Function):
    """(sum, y) of x + residual; residual may be None."""

    @staticmethod
    def forward(ctx, tokens, x, residual, weight):
        w = weight.to(BF16)
        out = tokens.norm(x, w, residual=residual, want=("sum", "y"))
        ctx.tokens, ctx.has_residual = tokens, residual is not None
        ctx.save_for_backward(out["sum"], w)
        return out["sum"], out["y"]

    @staticmethod
    def backward(ctx, dsum, dy):
        s, w = ctx.saved_tensors
        g = ctx.tokens.norm_backward(s, w, dy.contiguous(), dsum=dsum.contiguous())
        return None, g["dx"], g["dx"] if ctx.has_residual else None, g["dweight"]


class Recurrence(torch.autograd.Function):
    """The layer with L = 1 (the gated delta rule): q, k, v [B,H,T,64] bf16, beta, alpha [B,H,T] fp32."""

    @staticmethod
    def forward(ctx, plan, conv_w, q, k, v, beta, alpha):
        inp = {"q": q, "k": k, "v": v, "beta": beta, "alpha": alpha, "u": None, "gamma": None, "eta": None, "conv_w": conv_w, "L": 1}
        ctx.plan, ctx.inp = plan, inp
        return plan.forward(inp, stream=torch.cuda.current_stream())

    @staticmethod
    def backward(ctx, dout):
        g = ctx.plan.backward(ctx.inp, dout.float().contiguous(), stream=torch.cuda.current_stream())
        return None, None, g["dq"].to(BF16), g["dk"].to(BF16), g["dv"].to(BF16), g["dbeta"], g["dalpha"]


class TokenLogprobs(torch.autograd.Function):
    @staticmethod
    def forward(ctx, tokens, logits, targets):
        out = tokens.token_logprobs(logits, targets)
        ctx.tokens = tokens
        ctx.save_for_backward(logits, targets, out["lse"], out["entropy"])
        return out["logprob"], out["entropy"]

    @staticmethod
    def backward(ctx, dlogprob, dentropy):
        logits, targets, lse, entropy = ctx.saved_tensors
        return None, ctx.tokens.token_logprobs_backward(logits, targets, lse, entropy, dlogprob.contiguous(), dentropy.contiguous()), None


class Model(torch.nn.Module):
    def __init__(self):
        super().__init__()
        g = torch.Generator().manual_seed(0)
        p = lambda *shape, std: torch.nn.Parameter(torch.randn(*shape, generator=g) * std)  # noqa: E731
        self.table = p(V, D, std=D ** -0.5)  # shared by the embedding and the head
        self.w_in, self.w_out = torch.nn.Parameter(torch.ones(D)), torch.nn.Parameter(torch.ones(D))
        self.proj = p(3 * H * DK, D, std=D ** -0.5)
        self.gates = p(2 * H, D, std=D ** -0.5)
        self.o = p(D, H * DK, std=D ** -0.5)

    def heads(self, y):
        """q, k, v [n, H, 64] and the gates [n, H] of normalised inputs y [n, D]."""
        q, k, v = (y @ self.proj.to(BF16).t()).view(-1, 3, H, DK).unbind(1)
        unit = lambda x: torch.nn.functional.normalize(x.float(), dim=-1).to(BF16)  # noqa: E731
        b, a = (y @ self.gates.to(BF16).t()).float().view(-1, 2, H).unbind(1)
        return unit(q), unit(k), v.contiguous(), torch.sigmoid(b), torch.exp(-torch.nn.functional.softplus(a) / 16)

    def forward(self, tokens, plan, conv_w, ids):
        e = Embed.apply(tokens, ids, self.table).view(-1, D)
        e, y = Norm.apply(tokens, e, None, self.w_in)
        q, k, v, beta, alpha = (x.view(B, T, *x.shape[1:]).transpose(1, 2).contiguous() for x in self.heads(y))
        o = Recurrence.apply(plan, conv_w, q, k, v, beta, alpha)
        o = o.transpose(1, 2).reshape(-1, H * DK) @ self.o.to(BF16).t()
        _, y = Norm.apply(tokens, o, e, self.w_out)
        return y @ self.table.to(BF16).t()


def sequences(follows, g, dev):
    ids = torch.empty(B, T + 1, dtype=torch.int64, device=dev)
    ids[:, 0] = torch.randint(0, V, (B,), generator=g, device=dev)
    stray = torch.rand(B, T, generator=g, device=dev) < 0.1
    other = torch.randint(0, V, (B, T), generator=g, device=dev)
    for t in range(T):
        ids[:, t + 1] = torch.where(stray[:, t], other[:, t], follows[ids[:, t]])
    return ids


def train(model, steps, dev="cuda"):
    g = torch.Generator(device=dev).manual_seed(1)
    follows = torch.randperm(V, generator=g, device=dev)
    conv_w = torch.zeros(H, 4, DK, dtype=BF16, device=dev)
    opt = torch.optim.Adam(model.parameters(), lr=5e-3)
    losses = []
    with binding.Tokens(B * T, D, V, io="bf16") as tokens, binding.Plan(B, H, T, DK, DK, 1, io="bf16") as plan:
        for _ in range(steps):
            ids = sequences(follows, g, dev)
            logits = model(tokens, plan, conv_w, ids[:, :-1].contiguous())
            logprob, _ = TokenLogprobs.apply(tokens, logits, ids[:, 1:].reshape(-1).contiguous())
            loss = -logprob.mean()
            opt.zero_grad()
            loss.backward()
            opt.step()
            losses.append(loss.item())
        tokens.last_device_status()
        plan.last_device_status()
    return losses, follows


@torch.no_grad()
def serve(model, follows, prompt=64, count=16, dev="cuda"):
    """Greedy continuation of B prompts, one item at a time; returns the items and the top alternatives' log
    probabilities of every step beside those of the head in bf16."""
    g = torch.Generator(device=dev).manual_seed(2)
    ids = sequences(follows, g, dev)[:, :prompt].contiguous()
    conv_w = torch.zeros(H, 4, DK, dtype=BF16, device=dev)
    S = torch.zeros(B, H, DK, DK, device=dev)
    hist = torch.zeros(B, H, 3, DK, dtype=BF16, device=dev)
    table, w_in, w_out = model.table.to(BF16), model.w_in.to(BF16), model.w_out.to(BF16)
    stream = torch.cuda.current_stream()
    items, alternatives, reference = [], [], []
    with binding.Tokens(B * prompt, D, V, io="bf16", logits="f32") as tokens, binding.Plan(B, H, prompt, DK, DK, 1, io="bf16") as plan:
        w8, w_scale = tokens.matmul8_weights(table)  # once

        def layer_inputs(tok):
            e = tokens.embed(tok, table).view(-1, D)
            q, k, v, beta, alpha = model.heads(tokens.norm(e, w_in)["y"])
            return e, {"q": q, "k": k, "v": v, "beta": beta, "alpha": alpha, "u": None, "gamma": None, "eta": None, "conv_w": conv_w, "L": 1}

        _, inp = layer_inputs(ids)
        for key in ("q", "k", "v", "beta", "alpha"):
            inp[key] = inp[key].view(B, prompt, *inp[key].shape[1:]).transpose(1, 2).contiguous()
        # the last token of the prompt is the first step below: the prompt's others go into the state
        head = {key: (x[:, :, : prompt - 1].contiguous() if key in ("q", "k", "v", "beta", "alpha") else x) for key, x in inp.items()}
        with binding.Plan(B, H, prompt - 1, DK, DK, 1, io="bf16") as before:
            before.forward_state(head, S_final=S, v_hist_out=hist, stream=stream)
            torch.cuda.synchronize()
        tok = ids[:, -1].contiguous()
        for _ in range(count):
            e, inp = layer_inputs(tok)
            o = plan.decode_step(inp, hist, S, stream=stream).reshape(B, H * DK) @ model.o.to(BF16).t()
            y = tokens.norm(o, w_out, residual=e, want=("y", "y8"))
            logits = tokens.matmul8(y["y8"], y["y_scale"], w8, w_scale)
            top = tokens.token_logprobs(logits, k=5)
            items.append(top["top_ids"][:, 0].clone())
            alternatives.append(top["top_logprob"])
            reference.append(torch.log_softmax(y["y"].float() @ table.float().t(), -1).gather(1, top["top_ids"]))
            tok = top["top_ids"][:, 0].contiguous()
        tokens.last_device_status()
        plan.last_device_status()
    return ids[:, -1], torch.stack(items, 1), torch.stack(alternatives), torch.stack(reference)


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--steps", type=int, default=60)
    a = ap.parse_args()
    build.build()
    model = Model().cuda()
    losses, follows = train(model, a.steps)
    print("loss:", " ".join("%.3f" % x for x in losses[:: max(1, a.steps // 10)] + losses[-1:]))
    last, items, alternatives, reference = serve(model, follows)
    chain = torch.cat([last[:, None], items], 1)
    hit = (follows[chain[:, :-1]] == chain[:, 1:]).float().mean().item()
    print("served %d items; %.0f %% follow the rule; 8-bit head against bf16: largest difference of a log probability %.3f"
          % (items.numel(), 100 * hit, (alternatives - reference).abs().max().item()))


if __name__ == "__main__":
    main()
