"""What the token operators are timed and compared on: the cases, their inputs, one pass, its work.

The operators are what stands between token ids and the recurrent layers and between the layers
and token probabilities: the embedding and its gradient, the root-mean-square norm with the
residual's addition (its 8-bit output and its gradient), the matrix product in 8-bit floating
point with a scale for each block of 128, and the log probabilities of given tokens with entropy
and top alternatives (and their gradient).  ``run`` computes a pass in plain torch operations in 32
bits, or, with ``own`` set, through ``ssm_sequence_layer_gb300.binding.Tokens``.

Sizes: D = 768 and D = 256 are the model widths of the projection workloads, 16384 tokens the
8 x 2048 and the 16K-token shapes, N = 4626 the projections of the language-model layer.
"""
import math

import numpy as np
import torch

own = False

TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
SIZES = {"bf16": 2, "f32": 4}
EPS = 1e-6
BLOCK = 128       # values that share a scale
FP8_MAX = 448.0   # the largest e4m3 value
FP32_TINY = 2.0 ** -126

VOCAB = 50021     # an odd vocabulary ...
VOCAB_PAD = 50048  # ... and the same padded to a multiple of 128, as the head product writes it


def listed():
    return [
        # one new token for each of 16 sequences being served: latency of the lookup
        {"name": "embed_decode", "op": "embed", "dtype": "bf16", "n": 16, "D": 768, "V": VOCAB},
        # the table's gradient of a language-model training step (8 x 2048 tokens)
        {"name": "embed_grad_lm", "op": "embed_grad", "dtype": "bf16", "n": 16384, "D": 768, "V": VOCAB},
        # ... and of a recommendation step: many items, narrow rows, 2 x 16384 tokens, fp32
        {"name": "embed_grad_items", "op": "embed_grad", "dtype": "f32", "n": 32768, "D": 256, "V": 200003},
        # the pre-norm of one served token for each of 16 sequences, into the 8-bit product
        {"name": "norm_decode", "op": "norm", "dtype": "bf16", "n": 16, "D": 768, "residual": True, "y": False, "y8": True},
        # the same for a batch of prompts
        {"name": "norm_prompt", "op": "norm", "dtype": "bf16", "n": 16384, "D": 768, "residual": True, "y": False, "y8": True},
        # the norm's gradient in training, with the residual stream's own cotangent
        {"name": "norm_grad", "op": "norm_grad", "dtype": "bf16", "n": 16384, "D": 768, "dsum": True},
        # the 8-bit head product for 8 served tokens: the weights' bytes bound it
        {"name": "matmul8_decode", "op": "matmul8", "dtype": "bf16", "M": 8, "N": VOCAB_PAD, "K": 768},
        # the head product for scoring 4096 tokens
        {"name": "matmul8_head", "op": "matmul8", "dtype": "bf16", "M": 4096, "N": VOCAB_PAD, "K": 768},
        # a projection with ragged sizes (last tiles and last scale block partly filled), fp32 out
        {"name": "matmul8_ragged", "op": "matmul8", "dtype": "f32", "M": 1003, "N": 4626, "K": 1040},
        # sampling for 4 sequences: a long row each, 20 alternatives, part of the vocabulary masked
        {"name": "logprobs_decode", "op": "logprobs", "dtype": "bf16", "n": 4, "V": VOCAB, "pad": VOCAB_PAD - VOCAB, "k": 20, "masked": True},
        # scoring a batch of prompts with 8 alternatives a token
        {"name": "logprobs_score", "op": "logprobs", "dtype": "bf16", "n": 4096, "V": VOCAB, "pad": VOCAB_PAD - VOCAB, "k": 8, "masked": False},
        # the loss's gradient in training, with an entropy term
        {"name": "logprobs_grad", "op": "logprobs_grad", "dtype": "bf16", "n": 4096, "V": VOCAB, "pad": VOCAB_PAD - VOCAB, "dentropy": True},
    ]


MOST_BYTES = 8e8    # of one pass of a drawn case; the largest listed ones come to this
MOST_FLOPS = 3e11


def _size(rng, low, high, multiple=1):
    """A size spread over the logarithm of [low, high]."""
    s = int(round(math.exp(rng.uniform(math.log(low), math.log(high))) / multiple)) * multiple
    s = min(max(s, low), high)
    return s if s != 3072 else s - multiple


def draw(rng):
    op = rng.choice(["embed", "embed_grad", "norm", "norm_grad", "matmul8", "logprobs", "logprobs_grad"])
    c = {"op": op, "dtype": rng.choice(["bf16", "bf16", "f32"])}
    if op in ("embed", "embed_grad"):
        c |= {"n": _size(rng, 1, 32768), "D": _size(rng, 64, 1024, rng.choice([1, 8, 64])), "V": _size(rng, 1000, 200003)}
    elif op in ("norm", "norm_grad"):
        c |= {"n": _size(rng, 1, 32768), "D": _size(rng, 64, 4096, rng.choice([1, 8, 64]))}
        if op == "norm":
            c |= {"residual": rng.random() < 0.7, "y": rng.random() < 0.5}
            c["y8"] = not c["y"] or rng.random() < 0.3
        else:
            c["dsum"] = rng.random() < 0.5
    elif op == "matmul8":
        c |= {"M": _size(rng, 1, 8192), "N": _size(rng, 64, 65536, rng.choice([1, 8, 128])), "K": _size(rng, 64, 4096, rng.choice([16, 128]))}
    else:
        c |= {"n": _size(rng, 1, 8192), "V": _size(rng, 100, 262144), "pad": rng.choice([0, 0, 3, 64])}
        if op == "logprobs":
            c |= {"k": rng.choice([0, 1, 5, 20, 32]), "masked": rng.random() < 0.5}
        else:
            c["dentropy"] = rng.random() < 0.5
    shrink = "V" if op == "embed_grad" else "M" if op == "matmul8" else "n"
    while c[shrink] > 1 and (work(c)["bytes"] > MOST_BYTES or work(c)["flops"] > MOST_FLOPS):
        c[shrink] = c[shrink] * 3 // 4
    return c


# ------------------------------------------------------------------------------------------- inputs
def _ids(n, V, g, dev, none_share):
    """Token ids whose frequency falls like one over their rank, a few of them -1 (no token)."""
    u = torch.rand(n, generator=g, device=dev, dtype=torch.float64)
    ids = (torch.exp(u * math.log(V + 1)) - 1).to(torch.int64).clamp_(0, V - 1)
    perm = torch.randperm(V, generator=g, device=dev)  # frequent tokens anywhere in the table
    ids = perm[ids]
    return torch.where(torch.rand(n, generator=g, device=dev) < none_share, torch.full_like(ids, -1), ids)


def _distinct(n, V):
    """How many different ids _ids draws, on average."""
    v = np.arange(V, dtype=np.float64)
    p = np.log((v + 2) / (v + 1)) / math.log(V + 1)
    return float(np.sum(-np.expm1(n * np.log1p(-p))))


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(int(seed) * 7919 + 17)
    io = TYPES[case["dtype"]]
    op = case["op"]

    def normal(*shape, std=1.0):
        return torch.randn(*shape, generator=g, device=dev) * std

    s = {"case": dict(case)}
    n = case.get("M", case.get("n"))
    if op == "embed":
        s["ids"] = _ids(n, case["V"], g, dev, 0.02)
        s["table"] = normal(case["V"], case["D"], std=case["D"] ** -0.5).to(io)
        s["scale"] = case["D"] ** 0.5
        s["out"] = torch.empty(n, case["D"], dtype=io, device=dev)
    elif op == "embed_grad":
        s["ids"] = _ids(n, case["V"], g, dev, 0.02)
        s["dout"] = normal(n, case["D"], std=0.05).to(io)
        s["scale"] = case["D"] ** 0.5
        s["dtable"] = torch.empty(case["V"], case["D"], device=dev)
    elif op in ("norm", "norm_grad"):
        D = case["D"]
        # a residual stream: some channels are several times the others
        channel = torch.exp(normal(D, std=0.7))
        s["weight"] = (1.0 + normal(D, std=0.2)).to(io)
        if op == "norm":
            s["x"] = normal(n, D).to(io)
            s["residual"] = (normal(n, D, std=2.0) * channel).to(io) if case["residual"] else None
            s["out"] = {"sum": torch.empty(n, D, dtype=io, device=dev)} if case["residual"] else {}
            if case["y"]:
                s["out"]["y"] = torch.empty(n, D, dtype=io, device=dev)
            if case["y8"]:
                s["out"]["y8"] = torch.empty(n, D, dtype=torch.float8_e4m3fn, device=dev)
                s["out"]["y_scale"] = torch.empty(n, -(-D // BLOCK), device=dev)
        else:
            s["sum"] = (normal(n, D, std=2.0) * channel).to(io)
            s["dy"] = normal(n, D, std=0.1).to(io)
            s["dsum"] = normal(n, D, std=0.1).to(io) if case["dsum"] else None
            s["out"] = {"dx": torch.empty(n, D, dtype=io, device=dev), "dweight": torch.empty(D, device=dev)}
    elif op == "matmul8":
        M, N, K = case["M"], case["N"], case["K"]
        kb, nb = -(-K // BLOCK), -(-N // BLOCK)
        a = torch.nn.functional.pad(normal(M, K) * torch.exp(normal(K, std=0.5)), (0, kb * BLOCK - K))
        sa = (a.view(M, kb, BLOCK).abs().amax(2) / FP8_MAX).clamp_min(FP32_TINY)
        s["a8"] = (a / sa.repeat_interleave(BLOCK, 1)).to(torch.float8_e4m3fn)[:, :K].contiguous()
        s["a_scale"] = sa
        w = torch.nn.functional.pad(normal(N, K, std=K ** -0.5), (0, kb * BLOCK - K, 0, nb * BLOCK - N))
        sw = (w.view(nb, BLOCK, kb, BLOCK).abs().amax((1, 3)) / FP8_MAX).clamp_min(FP32_TINY)
        w = w / sw.repeat_interleave(BLOCK, 0).repeat_interleave(BLOCK, 1)
        s["w8"] = w.to(torch.float8_e4m3fn)[:N, :K].contiguous()
        s["w_scale"] = sw
        s["out"] = torch.empty(M, N, dtype=io, device=dev)
    else:
        V = case["V"]
        full = torch.empty(n, V + case["pad"], dtype=io, device=dev)
        full.copy_(normal(n, V + case["pad"], std=2.5))
        s["logits"] = full[:, :V]
        s["targets"] = _ids(n, V, g, dev, 0.03)
        at = torch.arange(n, device=dev)
        likely = s["targets"].clamp_min(0)
        s["logits"][at, likely] += torch.rand(n, generator=g, device=dev).mul_(12.0).to(io)  # a model that learned something
        if case.get("masked"):
            s["logits"].masked_fill_(torch.rand(n, V, generator=g, device=dev) < 0.1, -math.inf)
        s["inv_temperature"] = 1.25 if op == "logprobs" else 1.0
        if op == "logprobs":
            k = case["k"]
            s["out"] = {x: torch.empty(n, device=dev) for x in ("logprob", "lse", "entropy")}
            if k:
                s["out"]["top_ids"] = torch.empty(n, k, dtype=torch.int64, device=dev)
                s["out"]["top_logprob"] = torch.empty(n, k, device=dev)
        else:
            z = s["logits"].double()
            s["lse"] = torch.logsumexp(z, 1).float()
            s["entropy"] = (s["lse"] - (torch.softmax(z, 1) * z).sum(1)).float()
            del z
            s["dlogprob"] = torch.full((n,), -1.0 / n, device=dev)
            s["dentropy"] = torch.full((n,), -0.01 / n, device=dev) if case["dentropy"] else None
            s["dlogits"] = torch.empty(n, V + case["pad"], dtype=io, device=dev)[:, :V]
    if own:
        from ssm_sequence_layer_gb300 import binding
        s["tokens"] = binding.Tokens(n, D=case.get("D", case.get("K", 64)), V=case.get("V", case.get("N", 64)), io=case["dtype"])
    return s


# ------------------------------------------------------------------------------------------ one pass
def run(s):
    c = s["case"]
    return (_run_own if own else _run_plain)(s, c, c["op"])


def _run_own(s, c, op):
    t = s["tokens"]
    if op == "embed":
        return t.embed(s["ids"], s["table"], scale=s["scale"], out=s["out"])
    if op == "embed_grad":
        return t.embed_backward(s["ids"], s["dout"], scale=s["scale"], dtable=s["dtable"])
    if op == "norm":
        return t.norm(s["x"], s["weight"], residual=s["residual"], eps=EPS, out=s["out"])
    if op == "norm_grad":
        return t.norm_backward(s["sum"], s["weight"], s["dy"], dsum=s["dsum"], eps=EPS, out=s["out"])
    if op == "matmul8":
        return t.matmul8(s["a8"], s["a_scale"], s["w8"], s["w_scale"], out=s["out"])
    if op == "logprobs":
        return t.token_logprobs(s["logits"], s["targets"], inv_temperature=s["inv_temperature"], k=c["k"], out=s["out"])
    return t.token_logprobs_backward(s["logits"], s["targets"], s["lse"], s["entropy"], s["dlogprob"], dentropy=s["dentropy"],
                                     inv_temperature=s["inv_temperature"], dlogits=s["dlogits"])


def _run_plain(s, c, op):
    io = TYPES[c["dtype"]]
    if op == "embed":
        rows = s["table"][s["ids"].clamp_min(0)].float() * s["scale"]
        return (rows * (s["ids"] >= 0).unsqueeze(1)).to(io)
    if op == "embed_grad":
        rows = s["dout"].float() * (s["scale"] * (s["ids"] >= 0)).unsqueeze(1)
        return torch.zeros(c["V"], c["D"], device=rows.device).index_add_(0, s["ids"].clamp_min(0), rows)
    if op == "norm":
        r, out = s["x"].float(), {}
        if c["residual"]:
            r = r + s["residual"].float()
            out["sum"] = r.to(io)
        y = r * torch.rsqrt((r * r).mean(1, keepdim=True) + EPS) * s["weight"].float()
        if c["y"]:
            out["y"] = y.to(io)
        if c["y8"]:
            n, D = y.shape
            kb = -(-D // BLOCK)
            blocks = torch.nn.functional.pad(y, (0, kb * BLOCK - D)).view(n, kb, BLOCK)
            out["y_scale"] = (blocks.abs().amax(2) / FP8_MAX).clamp_min(FP32_TINY)
            out["y8"] = (blocks / out["y_scale"].unsqueeze(2)).to(torch.float8_e4m3fn).view(n, kb * BLOCK)[:, :D].contiguous()
        return out
    if op == "norm_grad":
        r, dy = s["sum"].float(), s["dy"].float()
        rstd = torch.rsqrt((r * r).mean(1, keepdim=True) + EPS)
        hat, wdy = r * rstd, s["weight"].float() * dy
        dx = rstd * (wdy - hat * (wdy * hat).mean(1, keepdim=True))
        if c["dsum"]:
            dx = dx + s["dsum"].float()
        return {"dx": dx.to(io), "dweight": (dy * hat).sum(0)}
    if op == "matmul8":
        a = s["a8"].float() * s["a_scale"].repeat_interleave(BLOCK, 1)[:, :c["K"]]
        w = s["w8"].float() * s["w_scale"].repeat_interleave(BLOCK, 0)[:c["N"]].repeat_interleave(BLOCK, 1)[:, :c["K"]]
        return (a @ w.t()).to(io)
    raw = s["logits"].float()
    z = raw * s["inv_temperature"]
    target = s["targets"].clamp_min(0).unsqueeze(1)
    live = s["targets"] >= 0
    if op == "logprobs":
        m = z.amax(1, keepdim=True)
        e = torch.exp(z - m)
        total = e.sum(1, keepdim=True)
        lse = (m + torch.log(total)).squeeze(1)
        logp = z - lse.unsqueeze(1)
        out = {"lse": lse, "logprob": torch.where(live, logp.gather(1, target).squeeze(1), torch.zeros_like(lse)),
               "entropy": -(e / total * torch.where(e > 0, logp, torch.zeros_like(logp))).sum(1)}
        if c["k"]:
            # one whole number a logit, ordered by value and then by lowest index
            bits = raw.view(torch.int32)
            key = (bits ^ ((bits >> 31) & 0x7FFFFFFF)).to(torch.int64) * (1 << 32) + (c["V"] - 1 - torch.arange(c["V"], device=raw.device))
            ids = c["V"] - 1 - (torch.topk(key, c["k"], dim=1).values & 0xFFFFFFFF)
            top = raw.gather(1, ids)
            out["top_ids"] = torch.where(top == -math.inf, torch.full_like(ids, -1), ids)
            out["top_logprob"] = top * s["inv_temperature"] - lse.unsqueeze(1)
        return out
    logp = z - s["lse"].unsqueeze(1)
    p = torch.exp(logp)
    dlp = (s["dlogprob"] * live).unsqueeze(1)
    d = -p * dlp
    d.scatter_add_(1, target, dlp)
    if c["dentropy"]:
        d = d - s["dentropy"].unsqueeze(1) * p * (torch.where(p > 0, logp, torch.zeros_like(logp)) + s["entropy"].unsqueeze(1))
    return (d * s["inv_temperature"]).to(io)


# ---------------------------------------------------------------------------------------------- work
def work(case):
    """Bytes that one pass has to read and write, and its operations."""
    op, e = case["op"], SIZES[case["dtype"]]
    if op == "embed":
        n, D = case["n"], case["D"]
        return {"bytes": 8 * n + e * D * (n + _distinct(n, case["V"])), "flops": n * D}
    if op == "embed_grad":
        n, D = case["n"], case["D"]
        return {"bytes": 8 * n + e * n * D + 4 * case["V"] * D, "flops": 2 * n * D}
    if op == "norm":
        n, D = case["n"], case["D"]
        tensors = 1 + 2 * case["residual"] + case["y"]
        quant = n * D + 4 * n * -(-D // BLOCK) if case["y8"] else 0
        return {"bytes": e * n * D * tensors + e * D + quant, "flops": 6 * n * D}
    if op == "norm_grad":
        n, D = case["n"], case["D"]
        return {"bytes": e * n * D * (3 + case["dsum"]) + e * D + 4 * D, "flops": 12 * n * D}
    if op == "matmul8":
        M, N, K = case["M"], case["N"], case["K"]
        kb, nb = -(-K // BLOCK), -(-N // BLOCK)
        return {"bytes": M * K + N * K + 4 * kb * (M + nb) + e * M * N, "flops": 2 * M * N * K}
    n, V = case["n"], case["V"]
    if op == "logprobs":
        return {"bytes": e * n * V + 8 * n + 12 * n + 8 * n * case["k"], "flops": 6 * n * V}
    return {"bytes": 2 * e * n * V + 8 * n + 4 * n * (3 + case["dentropy"]), "flops": 8 * n * V}


# --------------------------------------------------------------------------------------------- exact
def exact(case, seed):
    """run()'s outputs from the definitions, in 64 bits."""
    s, op = prepare(case, seed), case["op"]
    f = torch.float64
    if op == "embed":
        onto = torch.cat([s["table"].to(f) * s["scale"], torch.zeros(1, case["D"], dtype=f, device=s["table"].device)])
        return onto[torch.where(s["ids"] < 0, torch.full_like(s["ids"], case["V"]), s["ids"])]
    if op == "embed_grad":
        keep = torch.nonzero(s["ids"] >= 0).flatten()
        full = torch.zeros(case["V"], case["D"], dtype=f, device=keep.device)
        full.index_put_((s["ids"][keep],), s["dout"][keep].to(f) * s["scale"], accumulate=True)
        return full
    if op == "norm":
        r = s["x"].to(f)
        if case["residual"]:
            r = r + s["residual"].to(f)
        D = case["D"]
        length = torch.linalg.vector_norm(r, dim=1, keepdim=True)
        y = r / torch.sqrt(length ** 2 / D + EPS) * s["weight"].to(f)
        out = {"sum": r} if case["residual"] else {}
        if case["y"]:
            out["y"] = y
        if case["y8"]:
            group = torch.arange(D, device=y.device) // BLOCK
            peak = torch.zeros(y.shape[0], -(-D // BLOCK), dtype=f, device=y.device)
            peak.scatter_reduce_(1, group.expand(y.shape[0], D), y.abs(), "amax")
            out["y_scale"] = torch.clamp(peak / FP8_MAX, min=FP32_TINY)
            out["y8"] = (y / out["y_scale"][:, group]).float().to(torch.float8_e4m3fn).to(f)
        return out
    if op == "norm_grad":
        r, dy, w = s["sum"].to(f), s["dy"].to(f), s["weight"].to(f)
        q = (r ** 2).sum(1, keepdim=True) / case["D"] + EPS
        along = (w * dy * r).sum(1, keepdim=True) / (case["D"] * q)
        dx = (w * dy - r * along) / q.sqrt()
        return {"dx": dx + s["dsum"].to(f) if case["dsum"] else dx, "dweight": torch.einsum("nd,nd->d", dy, r / q.sqrt())}
    if op == "matmul8":
        dev = s["a8"].device
        col = torch.arange(case["K"], device=dev) // BLOCK
        row = torch.arange(case["N"], device=dev) // BLOCK
        a = s["a8"].float().to(f) * s["a_scale"].to(f)[:, col]
        w = s["w8"].float().to(f) * s["w_scale"].to(f)[row][:, col]
        return torch.einsum("mk,nk->mn", a, w)
    z = s["logits"].to(f) * s["inv_temperature"]
    live = s["targets"] >= 0
    if op == "logprobs":
        lse = torch.logsumexp(z, 1)
        p = torch.softmax(z, 1)
        out = {"lse": lse, "entropy": lse - torch.nansum(p * z, 1)}
        mine = z[torch.arange(z.shape[0], device=z.device), s["targets"].clamp_min(0)]
        out["logprob"] = torch.where(live, mine - lse, torch.zeros_like(lse))
        if case["k"]:
            out["top_logprob"] = torch.sort(z, dim=1, descending=True).values[:, :case["k"]] - lse.unsqueeze(1)
            out["top_ids"] = None
        return out
    logp = z - s["lse"].to(f).unsqueeze(1)
    p = logp.exp()
    hit = torch.zeros_like(p)
    hit[live, s["targets"][live]] = 1.0
    d = torch.where(live, s["dlogprob"], torch.zeros_like(s["dlogprob"])).to(f).unsqueeze(1) * (hit - p)
    if case["dentropy"]:
        d -= s["dentropy"].to(f).unsqueeze(1) * p * (logp + s["entropy"].to(f).unsqueeze(1))
    return d * s["inv_temperature"]
