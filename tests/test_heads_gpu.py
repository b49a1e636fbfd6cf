"""The heads' norm, rotation and layout, and their gradient, against the fp64 oracle.

Tolerances, with u = 2^-24 and h = half a unit in the last place of the io type.  A head's row is x, its normalised row y0 = r x w.
  y        r: the sum of squares within (d + 4) u of itself (d additions in any order), halved by the root, and four roundings of
    the mean, eps, the root (2 units) and its use; the weight one.  The angle is exact to 2^-38 turns at these positions; its rest of an
    eighth of a turn at most is rounded to fp32 (2^-27 turns 2 pi < 2^-24), cos and sin are within 2 u of themselves, the amplitude one
    more.  A pair's magnitude is m = hypot(a, b) amplitude:  ((d / 2 + 8) u + 8 u) m and h.
  dx       g as y above: 8 u hypot(g) amplitude.  Each of the two terms of dx within (d + 24) u of its magnitude; the sum over the row
    may cancel, so its magnitude is r |y1| sum |w g y1| with y1 = r x (times 1/d for rms); plus u |dx| and h.
  dw       a sum over tokens and heads: n terms, each within (d / 2 + 16) u of |g| |y1|: (n + d / 2 + 16) u sum |g y1|."""
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


def frequencies(rot, base=10000.0):
    return (base ** (-torch.arange(rot // 2, dtype=torch.float64) * 2 / max(rot, 1))).float()


# B, T, heads, d, dv, rot, norm, weights, interleaved, amplitude, positions, padding of the rows
FORMS = [
    (1, 1, (1, 1, 1), 64, 64, 64, "unit", False, False, 1.0, True, 0),
    (3, 5, (6, 6, 6), 128, 128, 128, "rms", True, False, 1.0, True, 0),
    (2, 70, (4, 2, 2), 64, 64, 32, "unit", False, True, 1.0, True, 0),
    (2, 33, (4, 4, 4), 128, 64, 64, "rms", True, True, 0.75, True, 8),
    (2, 9, (3, 1, 0), 80, 1, 40, "rms", True, False, 1.0, False, 0),
    (1, 7, (2, 2, 2), 64, 128, 0, "unit", False, False, 1.0, True, 16),
    (2, 6, (1, 0, 3), 17, 5, 6, "rms", True, False, 1.25, True, 0),
    (2, 6, (1, 2, 1), 30, 30, 30, "unit", True, True, 1.0, True, 3),
    (1, 4, (0, 0, 5), 64, 24, 0, "none", False, False, 1.0, False, 0),
    (2, 4, (2, 2, 1), 512, 512, 512, "rms", True, False, 1.0, True, 0),
    (2, 4, (2, 2, 1), 511, 509, 254, "unit", True, False, 1.0, True, 0),
    (1, 4, (2, 1, 1), 512, 16, 256, "rms", True, True, 1.0, True, 0),
    (1, 3, (1, 1, 1), 1, 1, 0, "rms", True, False, 1.0, False, 0),
    (1, 3, (1, 1, 1), 2, 3, 2, "none", False, True, 1.0, True, 0),
    (2, 300, (2, 2, 2), 16, 16, 16, "none", True, False, 1.0, True, 0),
    (40, 1, (6, 6, 6), 128, 128, 128, "unit", False, False, 1.0, True, 0),
    (1, 1000, (3, 3, 3), 72, 72, 24, "rms", True, False, 1.0, True, 0),
]
FORM = "Bn,T,heads,d,dv,rot,norm,weights,interleaved,amplitude,positions,pad"


def setup(io, Bn, T, heads, d, dv, rot, norm, weights, interleaved, amplitude, positions, pad, seed=0):
    g = torch.Generator().manual_seed(seed + d * T)
    width = (heads[0] + heads[1]) * d + heads[2] * dv
    x = (torch.randn(Bn, T, width + pad, generator=g) * torch.exp(torch.randn(width + pad, generator=g) * 0.5)).to(DT[io]).cuda()
    qw, kw = ((1 + 0.2 * torch.randn(d, generator=g)).to(DT[io]).cuda() if weights else None for _ in "qk")
    freq = frequencies(rot)
    pos = (torch.randint(-1000, 100000, (Bn, 1), generator=g) + torch.arange(T)).contiguous() if positions else torch.arange(T).repeat(Bn, 1)
    form = dict(heads=heads, d=d, dv=dv, norm=norm, q_weight=qw, k_weight=kw, eps=1e-6, inv_freq=freq.cuda() if rot else None,
                interleaved=interleaved, amplitude=amplitude, positions=pos.cuda() if positions else None)
    eps = float(np.float32(1e-6))
    args = (heads, d, dv, norm, eps, None if qw is None else f64(qw), None if kw is None else f64(kw), f64(freq), interleaved, amplitude, pos.numpy())
    return x, width, form, args


def pair_size(y, rot, interleaved, amplitude):
    """The magnitude of each value's pair before it is turned (its own where it is not turned); y [..., d]."""
    first, second = O._pairs(rot, interleaved)
    m = np.abs(y).copy()
    both = np.hypot(y[..., first], y[..., second]) * (abs(amplitude) if rot else 1.0)
    m[..., first] = m[..., second] = both
    return m


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize(FORM, FORMS)
def test_heads(io, Bn, T, heads, d, dv, rot, norm, weights, interleaved, amplitude, positions, pad):
    x, width, form, args = setup(io, Bn, T, heads, d, dv, rot, norm, weights, interleaved, amplitude, positions, pad)
    with B.Tokens(Bn * T, 64, 8, io=io) as t:
        out = t.heads(x, **form)
        cut = t.heads(x[:, :, :width], **form)
        torch.cuda.synchronize()
        t.last_device_status()
    q, k, v = O.heads(f64(x)[:, :, :width], *args)
    for key, ref in (("q", q), ("k", k)):
        if ref.shape[1] == 0:
            assert key not in out
            continue
        # turning keeps a pair's size: taken from the result
        e = ((d / 2 + 16) * u) * pair_size(ref / (amplitude if rot else 1.0), rot, interleaved, amplitude)
        got = f64(out[key])
        assert got.shape == ref.shape and np.all(np.abs(got - ref) <= e + half_ulp(io, np.abs(ref) + e) * 1.0001), key
        assert torch.equal(cut[key], out[key])
    if heads[2]:
        assert torch.equal(out["v"], x[:, :, width - heads[2] * dv:width].view(Bn, T, heads[2], dv).transpose(1, 2))


@pytest.mark.parametrize("io,grads_io", [("bf16", "f32"), ("bf16", "bf16"), ("f32", "f32")])
@pytest.mark.parametrize(FORM, FORMS)
def test_heads_backward(io, grads_io, Bn, T, heads, d, dv, rot, norm, weights, interleaved, amplitude, positions, pad):
    x, width, form, args = setup(io, Bn, T, heads, d, dv, rot, norm, weights, interleaved, amplitude, positions, pad, seed=1)
    g = torch.Generator().manual_seed(7)
    grads = {key: torch.randn(Bn, H, T, size, generator=g).to(DT[grads_io]).cuda() for key, H, size in
             (("dq", heads[0], d), ("dk", heads[1], d), ("dv", heads[2], dv))}
    with B.Tokens(Bn * T, 64, 8, io=io) as t:
        out = t.heads_backward(x, grads, **form)
        into = torch.full((Bn, T, width + 24), 42.0, dtype=DT[io], device="cuda")
        t.heads_backward(x, grads, out={"dx": into}, **form)
        again = t.heads_backward(x, grads, **form)
        torch.cuda.synchronize()
        t.last_device_status()
    assert all(torch.equal(out[key], again[key]) for key in out)
    if heads[0] + heads[1] == 0 or True:
        assert torch.all(into[:, :, width:] == 42)
    X, G = f64(x)[:, :, :width], [f64(grads[key]) for key in ("dq", "dk", "dv")]
    dx, dqw, dkw = O.heads_backward(X, G, *args)
    tol, dws, at = np.zeros_like(dx), [], 0
    for i, (H, key) in enumerate(((heads[0], "q"), (heads[1], "k"))):
        y = X[:, :, at:at + H * d].reshape(Bn, T, H, d)
        size = O._size(y, norm, args[4])
        y1 = y / size
        gs = pair_size(G[i].transpose(0, 2, 1, 3), rot, interleaved, amplitude)
        w = np.abs(args[5 + i]) if weights else 1.0
        share = {"none": 0.0, "unit": 1.0, "rms": 1.0 / d}[norm]
        along = np.abs(y1) * share * (w * gs * np.abs(y1)).sum(-1, keepdims=True)
        tol[:, :, at:at + H * d] = ((d + 24) * u * (w * gs + along) / size).reshape(Bn, T, H * d)
        dws.append((H * Bn * T + d / 2 + 16) * u * (gs * np.abs(y1)).sum((0, 1, 2)))
        at += H * d
    got = f64(out["dx"])
    tol += u * np.abs(dx)
    assert np.all(np.abs(got - dx) <= tol + half_ulp(io, np.abs(dx) + tol) * 1.0001)
    assert torch.equal(into[:, :, :width], out["dx"])
    if weights:
        for key, ref, e, H in (("dq_weight", dqw, dws[0], heads[0]), ("dk_weight", dkw, dws[1], heads[1])):
            if H:
                assert np.all(np.abs(f64(out[key]) - ref) <= e + u * np.abs(ref)), key


def test_far_positions_in_both_signs():
    """Positions up to 2^40: the angle is reduced without loss, so a rotation is as exact as near zero."""
    pos = torch.tensor([[0, 1, -1, 2 ** 20 + 1, -(2 ** 31) - 7, 2 ** 40 - 3, 10 ** 12, -(2 ** 40)]])
    d, freq = 8, torch.tensor([1.0, 0.7310585, 1e-3, 3.3e-7])
    x = torch.tensor([1.0, 1, 1, 1, 0, 0, 0, 0]).repeat(1, pos.numel(), 1)
    with B.Tokens(pos.numel(), 64, 8, io="f32") as t:
        q = f64(t.heads(x.cuda(), (1, 0, 0), d, norm="none", inv_freq=freq.cuda(), positions=pos.cuda())["q"])[0, 0]
    ref = np.array([[O.angle(p, f) for f in f64(freq)] for p in pos[0].tolist()])
    # 2^-62 of a turn a position, times 2^40 of them, 2^-19 radians at most; the rest as above
    slack = 8 * u + 2 * np.pi * 2.0 ** -62 * np.abs(pos[0].numpy())[:, None]
    assert np.all(np.abs(q[:, :4] - np.cos(ref)) <= slack) and np.all(np.abs(q[:, 4:] - np.sin(ref)) <= slack)


@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_empty_and_zero_rows(io):
    x = torch.zeros(2, 3, 192, dtype=DT[io], device="cuda")
    grads = {key: torch.ones(2, 1, 3, 64, device="cuda") for key in ("dq", "dk", "dv")}
    w = torch.ones(64, dtype=DT[io], device="cuda")
    with B.Tokens(6, 64, 8, io=io) as t:
        for norm in ("unit", "rms"):
            out = t.heads(x, (1, 1, 1), 64, norm=norm, q_weight=w, k_weight=w)
            assert not any(o.any() for o in out.values())
            back = t.heads_backward(x, grads, (1, 1, 1), 64, norm=norm, q_weight=w, k_weight=w)
            # r = 1 / sqrt(eps): the cotangent scaled, nothing along x
            assert np.allclose(f64(back["dx"])[:, :, :128], 1e3, rtol=2.0 ** -8) and not back["dq_weight"].any()
        none = torch.empty(2, 0, 192, dtype=DT[io], device="cuda")
        assert t.heads(none, (1, 1, 1), 64)["q"].shape == (2, 1, 0, 64)
        empty = {key: torch.empty(2, 1, 0, 64, device="cuda") for key in grads}
        out = {"dx": none.clone(), "dq_weight": torch.ones(64, device="cuda"), "dk_weight": torch.ones(64, device="cuda")}
        t.heads_backward(none, empty, (1, 1, 1), 64, out=out, q_weight=w, k_weight=w)
        assert not out["dq_weight"].any() and not out["dk_weight"].any()
        t.last_device_status()


def test_refusals():
    x = torch.zeros(2, 3, 192, dtype=torch.bfloat16, device="cuda")
    o = torch.zeros(2, 1, 3, 64, dtype=torch.bfloat16, device="cuda")
    f = torch.ones(32, device="cuda")

    def form(**kw):
        v = dict(B=2, T=3, Hq=1, Hk=1, Hv=1, d=64, dv=64, norm=1, eps=1e-6, q_weight=None, k_weight=None, rot=64, interleaved=0,
                 inv_freq=f.data_ptr(), amplitude=1.0, positions=None)
        v.update(kw)
        return B.prism_heads_form(*v.values())

    bad, unsupported, misaligned = B.PRISM_ERR_INVALID_ARG, B.PRISM_ERR_UNSUPPORTED, B.PRISM_ERR_MISALIGNED
    with B.Tokens(6, 64, 8) as t:
        B.prism_heads(t.handle, form(), x, 192, o, o.clone(), o.clone())
        for kw, status in [(dict(B=3), bad), (dict(T=-1), bad), (dict(B=1 << 20, T=1 << 20), bad), (dict(Hq=-1), bad), (dict(Hq=0, Hk=0, Hv=0), bad),
                           (dict(Hq=65536), unsupported), (dict(d=0), bad), (dict(dv=0), bad), (dict(d=513), unsupported), (dict(dv=600), unsupported),
                           (dict(norm=3), bad), (dict(eps=-1.0), bad), (dict(eps=float("nan")), bad), (dict(rot=63), bad), (dict(rot=66), bad),
                           (dict(rot=-2), bad), (dict(inv_freq=None), bad), (dict(inv_freq=f.data_ptr() + 2), misaligned),
                           (dict(amplitude=float("inf")), bad), (dict(d=65, rot=0), bad), (dict(q_weight=x.data_ptr() + 2), misaligned),
                           (dict(positions=x.data_ptr() + 4), misaligned)]:
            with pytest.raises(B.PrismError) as e:
                B.prism_heads(t.handle, form(**kw), x, 192, o, o, o)
            assert e.value.status == status, kw
        for call, status in [(lambda: B.prism_heads(t.handle, form(), x, 191, o, o, o), bad), (lambda: B.prism_heads(t.handle, form(), x, 192, None, o, o), bad),
                             (lambda: B.prism_heads(t.handle, form(), x, 192, o, o, o.data_ptr() + 2), misaligned),
                             (lambda: B.prism_heads_backward(t.handle, form(), x, 192, 7, o, o, o, x, 192, None, None), bad),
                             (lambda: B.prism_heads_backward(t.handle, form(), x, 192, 1, o, o, o, x, 100, None, None), bad),
                             (lambda: B.prism_heads_backward(t.handle, form(), x, 192, 1, None, o, o, x, 192, None, None), bad),
                             (lambda: B.prism_heads_backward(t.handle, form(Hk=0), x, 192, 1, o, None, o, x, 192, None, f), bad)]:
            with pytest.raises(B.PrismError) as e:
                call()
            assert e.value.status == status
        torch.cuda.synchronize()


@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_streams_graphs_and_equal_bits(io):
    x, width, form, _ = setup(io, 3, 50, (4, 4, 4), 64, 64, 64, "rms", True, False, 1.0, True, 0)
    grads = {key: torch.randn(3, 4, 50, 64, device="cuda") for key in ("dq", "dk", "dv")}
    with B.Tokens(150, 64, 8, io=io) as t:
        def call():
            return [*t.heads(x, **form).values(), *t.heads_backward(x, grads, **form).values()]
        first = call()
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        own = t.heads(x, stream=side, **form)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(own.values(), first))
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            held = call()
        x.neg_()
        graph.replay()
        torch.cuda.synchronize()
        changed = [h.clone() for h in held]
        assert all(torch.equal(a, b) for a, b in zip(call(), changed)) and not torch.equal(changed[0], first[0])
        x.neg_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(first, held))
