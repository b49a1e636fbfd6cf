"""What the operators of a model's block and of serving are timed and compared on: the cases, their inputs, one pass, its work.

The operators are the matrix product with bias, activation and residual (and both of its gradients), the queries', keys' and
values' way from a projection's rows into the layer's layout with the norm of each head and the position rotation (and its
gradient), and the drawing of a token from logits under temperature, top-k, top-p and min-p.  ``run`` computes a pass in plain
torch operations in 32 bits (angles and sampling masses in 64), or, with ``own`` set, through
``ssm_sequence_layer_gb300.binding.Tokens``.

Sizes: D = 768 with 6 heads of 128 and D = 256 with 4 heads of 64 are the widths of the projection workloads, 8 x 2048 and
2 x 16384 tokens their lengths, 2048 a feed-forward width for D = 768, 50021 an odd vocabulary.
"""
import math

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
SIZES = {"bf16": 2, "f32": 4}
EPS = 1e-6
VOCAB = 50021


def listed():
    return [
        # the q, k, v projection of one new token for each of 16 served sequences: the weights' bytes and latency
        {"name": "linear_decode", "op": "linear", "dtype": "bf16", "M": 16, "N": 2304, "K": 768, "bias": False, "act": "none", "residual": False, "pre": False},
        # the first product of a feed-forward in training (8 x 2048 tokens), the pre-activation kept for the gradient
        {"name": "linear_mlp", "op": "linear", "dtype": "bf16", "M": 16384, "N": 2048, "K": 768, "bias": True, "act": "gelu", "residual": False, "pre": True},
        # its second product's gradient, through the activation to the pre-activation
        {"name": "linear_dx_mlp", "op": "linear_dx", "dtype": "bf16", "M": 16384, "N": 768, "K": 2048, "act": "gelu", "dsum": False},
        # a small model in fp32 with ragged sizes, the residual stream's cotangent added
        {"name": "linear_dx_ragged", "op": "linear_dx", "dtype": "f32", "M": 1003, "N": 770, "K": 1041, "act": "none", "dsum": True},
        # the first product's weight and bias gradient: sums over all tokens
        {"name": "linear_dw_mlp", "op": "linear_dw", "dtype": "bf16", "M": 16384, "N": 2048, "K": 768, "dbias": True},
        # ... and of the small fp32 model
        {"name": "linear_dw_ragged", "op": "linear_dw", "dtype": "f32", "M": 2979, "N": 515, "K": 770, "dbias": True},
        # one new token for each of 16 served sequences at positions of their own, unit rows as the layer takes them
        {"name": "heads_decode", "op": "heads", "dtype": "bf16", "B": 16, "T": 1, "heads": 6, "d": 128, "norm": "unit", "weight": False, "rot": 128, "interleaved": False},
        # the same for a batch of prompts, root-mean-square norm with weights
        {"name": "heads_prompt", "op": "heads", "dtype": "bf16", "B": 8, "T": 2048, "heads": 6, "d": 128, "norm": "rms", "weight": True, "rot": 128, "interleaved": False},
        # training: the layer's fp32 cotangents back to the projection's rows
        {"name": "heads_grad_lm", "op": "heads_grad", "dtype": "bf16", "B": 8, "T": 2048, "heads": 6, "d": 128, "norm": "rms", "weight": True, "rot": 128, "interleaved": False},
        # long sequences of narrow heads in fp32, a part of each head rotated, pairs interleaved
        {"name": "heads_grad_items", "op": "heads_grad", "dtype": "f32", "B": 2, "T": 16384, "heads": 4, "d": 64, "norm": "unit", "weight": False, "rot": 32, "interleaved": True},
        # drawing the next token of 4 sequences: few long rows
        {"name": "sample_decode", "op": "sample", "dtype": "bf16", "n": 4, "V": VOCAB, "pad": 27, "rules": "both", "masked": True},
        # ... of 512 sequences, each with rules of its own
        {"name": "sample_batch", "op": "sample", "dtype": "f32", "n": 512, "V": VOCAB, "pad": 27, "rules": "mixed", "masked": False},
    ]


MOST_BYTES = 2.7e8    # of one pass of a drawn case ...
MOST_FLOPS = 5.2e10   # ... and its operations; the largest listed ones come to this
MOST_SAMPLED = 2.6e7  # logits of a drawn sampling case


def _size(rng, low, high, multiple=1):
    """A size spread over the logarithm of [low, high]."""
    s = int(round(math.exp(rng.uniform(math.log(low), math.log(high))) / multiple)) * multiple
    return min(max(s, low), high)


def draw(rng):
    op = rng.choice(["linear", "linear_dx", "linear_dw", "heads", "heads_grad", "sample", "sample"])
    c = {"op": op, "dtype": rng.choice(["bf16", "bf16", "f32"])}
    if op.startswith("linear"):
        c |= {"M": _size(rng, 1, 16384), "N": _size(rng, 64, 4096, rng.choice([1, 8, 64])), "K": _size(rng, 64, 4096, rng.choice([1, 8, 64]))}
        if op == "linear":
            c |= {"bias": rng.random() < 0.6, "act": rng.choice(["none", "gelu", "silu"]), "residual": rng.random() < 0.5, "pre": rng.random() < 0.3}
        elif op == "linear_dx":
            c |= {"act": rng.choice(["none", "gelu", "silu"]), "dsum": rng.random() < 0.5}
        else:
            c["dbias"] = rng.random() < 0.7
        shrink = "M"
    elif op in ("heads", "heads_grad"):
        d = rng.choice([16, 64, 64, 80, 128, 128])
        c |= {"B": _size(rng, 1, 32), "T": _size(rng, 1, 16384), "heads": rng.choice([1, 3, 4, 6, 8]), "d": d, "norm": rng.choice(["none", "unit", "rms"]),
              "weight": rng.random() < 0.5, "rot": rng.choice([0, d // 2, d, d]), "interleaved": rng.random() < 0.4}
        c["weight"] = c["weight"] and c["norm"] == "rms"
        shrink = "T"
    else:
        c |= {"n": _size(rng, 1, 2048), "V": _size(rng, 100, 262144), "pad": rng.choice([0, 0, 3, 64]),
              "rules": rng.choice(["none", "top_k", "top_p", "min_p", "both", "mixed", "mixed"]), "masked": rng.random() < 0.5}
        while c["n"] * c["V"] > MOST_SAMPLED:
            c["n"] = c["n"] * 3 // 4
        return c
    while c[shrink] > 1 and (work(c)["bytes"] > MOST_BYTES or work(c)["flops"] > MOST_FLOPS):
        c[shrink] = c[shrink] * 3 // 4
    return c


# ------------------------------------------------------------------------------------------- inputs
def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(int(seed) * 7927 + 23)
    io, op = TYPES[case["dtype"]], case["op"]

    def normal(*shape, std=1.0):
        return torch.randn(*shape, generator=g, device=dev) * std

    def uniform(*shape):
        return torch.rand(*shape, generator=g, device=dev)

    s = {"case": dict(case)}
    if op.startswith("linear"):
        M, N, K = case["M"], case["N"], case["K"]
        rows = M
        if op != "linear_dx":  # a layer's input: some channels are larger than the others
            s["x"] = (normal(M, K) * torch.exp(normal(K, std=0.5))).to(io)
        if op != "linear_dw":
            s["W"] = normal(N, K, std=K ** -0.5).to(io)
        if op == "linear":
            s["bias"] = normal(N, std=0.3).to(io) if case["bias"] else None
            s["residual"] = normal(M, N).to(io) if case["residual"] else None
            s["out"] = {key: torch.empty(M, N, dtype=io, device=dev) for key in (("y", "pre") if case["pre"] else ("y",))}
        else:
            s["dy"] = normal(M, N, std=0.1).to(io)
        if op == "linear_dx":
            s["pre"] = normal(M, K, std=1.5).to(io) if case["act"] != "none" else None
            s["dsum"] = normal(M, K, std=0.1).to(io) if case["dsum"] else None
            s["dx"] = torch.empty(M, K, dtype=io, device=dev)
        if op == "linear_dw":
            s["out"] = {"dW": torch.empty(N, K, device=dev)}
            if case["dbias"]:
                s["out"]["dbias"] = torch.empty(N, device=dev)
    elif op in ("heads", "heads_grad"):
        B, T, H, d, rot = (case[key] for key in ("B", "T", "heads", "d", "rot"))
        rows = B * T
        s["x"] = (normal(B, T, 3 * H * d) * torch.exp(normal(3 * H * d, std=0.5))).to(io)
        # sequences that go on: consecutive positions from a start of each sequence's own
        s["positions"] = (torch.randint(0, 100000, (B, 1), generator=g, device=dev) + torch.arange(T, device=dev)).contiguous()
        s["inv_freq"] = (10000.0 ** (-torch.arange(rot // 2, device=dev, dtype=torch.float64) * 2 / max(rot, 1))).float()
        s["q_weight"], s["k_weight"] = ((1.0 + normal(d, std=0.2)).to(io) if case["weight"] else None for _ in "qk")
        if op == "heads":
            s["out"] = {key: torch.empty(B, H, T, d, dtype=io, device=dev) for key in "qkv"}
        else:
            s["grads"] = {key: normal(B, H, T, d, std=0.1) for key in ("dq", "dk", "dv")}  # fp32, as the layer's backward leaves them
            s["out"] = {"dx": torch.empty(B, T, 3 * H * d, dtype=io, device=dev)}
            if case["weight"]:
                s["out"] |= {key: torch.empty(d, device=dev) for key in ("dq_weight", "dk_weight")}
    else:
        n, V = case["n"], case["V"]
        rows = n
        full = torch.empty(n, V + case["pad"], dtype=io, device=dev)
        full.copy_(normal(n, V + case["pad"], std=2.5))
        s["logits"] = full[:, :V]
        # a model that has learned something: a few likely tokens in each row
        likely = torch.randint(0, V, (n, 8), generator=g, device=dev)
        s["logits"].scatter_add_(1, likely, (uniform(n, 8) * 10.0).to(io))
        if case["masked"]:
            s["logits"].masked_fill_(uniform(n, V) < 0.1, -math.inf)
        s["u"] = uniform(n)
        rules, pick = case["rules"], lambda *of: torch.tensor(of, device=dev)[torch.randint(0, len(of), (n,), generator=g, device=dev)]  # noqa: E731
        mixed = rules == "mixed"
        s["inv_temperature"] = 0.7 + 0.8 * uniform(n)
        s["top_k"] = pick(0, 1, 20, 50, 1000).int() if mixed else pick(20, 50, 200).int() if rules in ("top_k", "both") else None
        s["top_p"] = pick(1.0, 0.5, 0.9, 0.95) if mixed else pick(0.8, 0.9, 0.95) if rules in ("top_p", "both") else None
        s["min_p"] = pick(0.0, 0.0, 0.02, 0.1) if mixed else pick(0.02, 0.05, 0.1) if rules == "min_p" else None
        s["out"] = {"ids": torch.empty(n, dtype=torch.int64, device=dev), "logprob": torch.empty(n, device=dev),
                    "kept": torch.empty(n, dtype=torch.int32, device=dev)}
    if own:
        from ssm_sequence_layer_gb300 import binding
        s["tokens"] = binding.Tokens(rows, D=case.get("K", case.get("d", 64)), V=case.get("V", 64), io=case["dtype"])
    return s


# ------------------------------------------------------------------------------------------ one pass
def run(s):
    c = s["case"]
    return (_run_own if own else _run_plain)(s, c, c["op"])


def _run_own(s, c, op):
    t = s["tokens"]
    if op == "linear":
        return t.linear(s["x"], s["W"], bias=s["bias"], activation=c["act"], residual=s["residual"], out=s["out"])
    if op == "linear_dx":
        return t.linear_backward(s["dy"], s["W"], activation=c["act"], pre=s["pre"], dsum=s["dsum"], dx=s["dx"])
    if op == "linear_dw":
        return t.linear_weight_backward(s["dy"], s["x"], out=s["out"])
    if op in ("heads", "heads_grad"):
        form = {"heads": (c["heads"],) * 3, "d": c["d"], "norm": c["norm"], "eps": EPS, "q_weight": s["q_weight"], "k_weight": s["k_weight"],
                "inv_freq": s["inv_freq"] if c["rot"] else None, "interleaved": c["interleaved"], "positions": s["positions"]}
        if op == "heads":
            return t.heads(s["x"], out=s["out"], **form)
        return t.heads_backward(s["x"], s["grads"], out=s["out"], **form)
    return t.sample(s["logits"], s["u"], inv_temperature=s["inv_temperature"], top_k=s["top_k"], top_p=s["top_p"], min_p=s["min_p"], out=s["out"])


def _act(z, act):
    if act == "gelu":
        return 0.5 * z * torch.special.erfc(z * -math.sqrt(0.5))
    return z / (1 + torch.exp(-z)) if act == "silu" else z


def _act_slope(z, act):
    if act == "gelu":
        return 0.5 * torch.special.erfc(z * -math.sqrt(0.5)) + z * torch.exp(-0.5 * z * z) * (2 * math.pi) ** -0.5
    p = 1 / (1 + torch.exp(-z))
    return p * (1 + z * (1 - p))


def _rotate(x, cos, sin, rot, interleaved):
    """The pairs of the first rot values of the last axis, turned by the angles whose cos and sin [B, 1, T, rot / 2] are."""
    if rot == 0:
        return x
    a, b = (x[..., 0:rot:2], x[..., 1:rot:2]) if interleaved else (x[..., :rot // 2], x[..., rot // 2:rot])
    a, b = a * cos - b * sin, a * sin + b * cos
    turned = torch.stack([a, b], -1).flatten(-2) if interleaved else torch.cat([a, b], -1)
    return torch.cat([turned, x[..., rot:]], -1)


def _run_plain(s, c, op):
    io = TYPES[c["dtype"]]
    if op == "linear":
        z = s["x"].float() @ s["W"].float().t()
        if c["bias"]:
            z = z + s["bias"].float()
        y = _act(z, c["act"])
        if c["residual"]:
            y = y + s["residual"].float()
        return {"y": y.to(io), "pre": z.to(io)} if c["pre"] else {"y": y.to(io)}
    if op == "linear_dx":
        dx = s["dy"].float() @ s["W"].float()
        if c["act"] != "none":
            dx = dx * _act_slope(s["pre"].float(), c["act"])
        return (dx + s["dsum"].float() if c["dsum"] else dx).to(io)
    if op == "linear_dw":
        dy = s["dy"].float()
        out = {"dW": dy.t() @ s["x"].float()}
        return out | {"dbias": dy.sum(0)} if c["dbias"] else out
    if op in ("heads", "heads_grad"):
        B, T, H, d, rot = (c[key] for key in ("B", "T", "heads", "d", "rot"))
        rows = s["x"].view(B, T, 3, H, d).permute(2, 0, 3, 1, 4).float()
        angle = s["positions"].double()[:, None, :, None] * s["inv_freq"].double()
        cos, sin = torch.cos(angle).float(), torch.sin(angle).float()
        out, back, dw = {}, [], {}
        for i, key in enumerate("qk"):
            x = rows[i]
            square = x * x
            scale = 1.0 if c["norm"] == "none" else torch.rsqrt((square.mean(-1, keepdim=True) if c["norm"] == "rms" else square.sum(-1, keepdim=True)) + EPS)
            w = s[key + "_weight"].float() if c["weight"] else 1.0
            if op == "heads":
                out[key] = _rotate(x * scale * w, cos, sin, rot, c["interleaved"]).to(io)
                continue
            g = _rotate(s["grads"]["d" + key], cos, -sin, rot, c["interleaved"])
            hat, wg = x * scale, w * g
            along = (wg * hat).sum(-1, keepdim=True) * {"none": 0.0, "unit": 1.0, "rms": 1.0 / d}[c["norm"]]
            back.append(scale * (wg - hat * along))
            if c["weight"]:
                dw["d%s_weight" % key] = (g * hat).sum((0, 1, 2))
        if op == "heads":
            return out | {"v": rows[2].to(io).contiguous()}
        back.append(s["grads"]["dv"])
        return {"dx": torch.stack(back).permute(1, 3, 0, 2, 4).reshape(B, T, 3 * H * d).to(io)} | dw
    # the draw, in 64 bits: whole numbers come out of sums that have to be on the right side of a border
    raw, V = s["logits"].float(), c["V"]
    bits = raw.view(torch.int32)
    key = (bits ^ ((bits >> 31) & 0x7FFFFFFF)).to(torch.int64) * (1 << 32) + (V - 1 - torch.arange(V, device=raw.device))
    ids = V - 1 - (torch.sort(key, dim=1, descending=True).values & 0xFFFFFFFF)  # by falling logit, then by rising id
    del key, bits
    z = raw.double() * s["inv_temperature"].double().unsqueeze(1)
    e = torch.exp(z - z.amax(1, keepdim=True))
    ordered = e.gather(1, ids)
    place = torch.arange(V, device=raw.device)
    keep = ordered > 0
    if s["top_k"] is not None:
        k = s["top_k"].long().unsqueeze(1)
        keep &= (place < k) | (k <= 0)
    ordered = ordered * keep
    if s["top_p"] is not None:
        before = torch.cumsum(ordered, 1) - ordered
        p = s["top_p"].double().unsqueeze(1)
        keep &= (before < p * ordered.sum(1, keepdim=True)) | (p >= 1)
    if s["min_p"] is not None:
        keep &= ordered >= s["min_p"].double().unsqueeze(1)
    kept = keep.sum(1)
    e = e * torch.zeros_like(e).scatter_(1, ids, keep.double())  # the kept ones, in the order of ids
    running = torch.cumsum(e, 1)
    chosen = (running <= s["u"].double().unsqueeze(1) * running[:, -1:]).sum(1, keepdim=True)
    logprob = torch.log(e.gather(1, chosen) / running[:, -1:])
    return {"ids": chosen.squeeze(1), "logprob": logprob.squeeze(1).float(), "kept": kept.int()}


# ---------------------------------------------------------------------------------------------- work
def work(case):
    """Bytes that one pass has to read and write, and its operations."""
    op, e = case["op"], SIZES[case["dtype"]]
    if op.startswith("linear"):
        M, N, K = case["M"], case["N"], case["K"]
        if op == "linear":
            data = e * (M * K + N * K + M * N * (1 + case["residual"] + case["pre"]) + N * case["bias"])
        elif op == "linear_dx":
            data = e * (M * N + N * K + M * K * (1 + (case["act"] != "none") + case["dsum"]))
        else:
            data = e * (M * N + M * K) + 4 * (N * K + N * case["dbias"])
        return {"bytes": data, "flops": 2 * M * N * K}
    if op in ("heads", "heads_grad"):
        n, width = case["B"] * case["T"], 3 * case["heads"] * case["d"]
        if op == "heads":
            return {"bytes": 2 * e * n * width + 8 * n, "flops": 8 * n * width}
        # the values' rows need no input beside their cotangent
        return {"bytes": e * n * width * 5 // 3 + 4 * n * width + 8 * n, "flops": 14 * n * width}
    return {"bytes": e * case["n"] * case["V"] + 36 * case["n"], "flops": 4 * case["n"] * case["V"]}


# --------------------------------------------------------------------------------------------- exact
def exact(case, seed):
    """run()'s outputs from the definitions, in 64 bits."""
    s, op, f = prepare(case, seed), case["op"], torch.float64
    if op == "linear":
        z = torch.einsum("mk,nk->mn", s["x"].to(f), s["W"].to(f))
        if case["bias"]:
            z += s["bias"].to(f)
        y = {"none": lambda v: v.clone(), "gelu": lambda v: v * torch.special.ndtr(v), "silu": lambda v: v * torch.sigmoid(v)}[case["act"]](z)
        if case["residual"]:
            y += s["residual"].to(f)
        return {"y": y, "pre": z} if case["pre"] else {"y": y}
    if op == "linear_dx":
        dx = torch.einsum("mn,nk->mk", s["dy"].to(f), s["W"].to(f))
        if case["act"] != "none":
            z = s["pre"].to(f)
            if case["act"] == "gelu":
                dx *= torch.special.ndtr(z) + z * torch.exp(-z ** 2 / 2) / math.sqrt(2 * math.pi)
            else:
                p = torch.sigmoid(z)
                dx *= p + z * p * torch.sigmoid(-z)
        if case["dsum"]:
            dx += s["dsum"].to(f)
        return dx
    if op == "linear_dw":
        out = {"dW": torch.einsum("mn,mk->nk", s["dy"].to(f), s["x"].to(f))}
        if case["dbias"]:
            out["dbias"] = torch.einsum("mn->n", s["dy"].to(f))
        return out
    if op in ("heads", "heads_grad"):
        B, T, H, d, rot = (case[key] for key in ("B", "T", "heads", "d", "rot"))
        half = rot // 2
        angle = torch.einsum("bt,i->bti", s["positions"].to(f), s["inv_freq"].to(f))
        turn = torch.polar(torch.ones_like(angle), angle)[:, :, None]  # a pair as one complex number
        first = torch.arange(half, device=angle.device) * (2 if case["interleaved"] else 1)
        second = first + (1 if case["interleaved"] else half)

        def turned(x, by):
            x = x.clone()
            pair = torch.complex(x[..., first], x[..., second]) * by
            x[..., first], x[..., second] = pair.real, pair.imag
            return x

        rows = s["x"].to(f).view(B, T, 3, H, d)
        out, back, dw = {}, [], {}
        for i, key in enumerate("qk"):
            x = rows[:, :, i]
            w = s[key + "_weight"].to(f) if case["weight"] else torch.ones(d, dtype=f, device=x.device)
            length = torch.linalg.vector_norm(x, dim=-1, keepdim=True)
            size = {"none": torch.ones_like(length), "unit": torch.sqrt(length ** 2 + EPS), "rms": torch.sqrt(length ** 2 / d + EPS)}[case["norm"]]
            if op == "heads":
                out[key] = turned(x / size * w, turn).transpose(1, 2)
                continue
            g = turned(s["grads"]["d" + key].to(f).transpose(1, 2), turn.conj())
            dx = w * g / size
            if case["norm"] != "none":
                dx -= x * (w * g * x).sum(-1, keepdim=True) / (size ** 3 * (d if case["norm"] == "rms" else 1))
            back.append(dx)
            if case["weight"]:
                dw["d%s_weight" % key] = torch.einsum("bthd,bthd->d", g, x / size)
        if op == "heads":
            return out | {"v": rows[:, :, 2].transpose(1, 2)}
        back.append(s["grads"]["dv"].to(f).transpose(1, 2))
        return {"dx": torch.stack(back, 2).reshape(B, T, 3 * H * d)} | dw
    # one row after the other
    out = {"ids": [], "logprob": [], "kept": []}
    for i in range(case["n"]):
        z = s["logits"][i].to(f) * s["inv_temperature"][i].to(f)
        z, ids = torch.sort(z, descending=True, stable=True)
        p = torch.exp(z - z[0])
        k = int(s["top_k"][i]) if s["top_k"] is not None else 0
        m = torch.count_nonzero(p)
        if k > 0:
            m = torch.clamp(m, max=k)
            p[k:] = 0
        if s["top_p"] is not None:
            part = s["top_p"][i].to(f)
            reach = torch.searchsorted(torch.cumsum(p, 0), part * p.sum())
            m = torch.where(part < 1, torch.minimum(m, reach + 1), m)
        if s["min_p"] is not None:
            m = torch.minimum(m, torch.count_nonzero(p >= s["min_p"][i].to(f)))
        p[torch.arange(p.numel(), device=p.device) >= m] = 0
        mass = torch.zeros_like(p)
        mass[ids] = p
        up = torch.cumsum(mass, 0)
        chosen = torch.searchsorted(up, s["u"][i].to(f) * up[-1], right=True)
        out["ids"].append(chosen)
        out["logprob"].append(torch.log(mass[chosen]) - torch.log(up[-1]))
        out["kept"].append(m)
    return {"ids": torch.stack(out["ids"]), "logprob": torch.stack(out["logprob"]), "kept": torch.stack(out["kept"]).int()}
