"""What the block's operators refuse without a GPU: null handles in the library, and in the Python layer tensors of another device,
type, shape or layout."""
import ctypes
import inspect

import pytest
import torch

from ssm_sequence_layer_gb300 import binding as B
from ssm_sequence_layer_gb300 import build
from tests.test_tokens_binding_host import OnDevice, tokens  # noqa: F401  (a fixture without a handle)


@pytest.fixture(scope="module")
def lib():
    build.build()
    return B.lib()


def test_null_handle(lib):
    form = B.prism_heads_form(1, 1, 1, 1, 1, 64, 64, 1, 1e-6, None, None, 0, 0, None, 1.0, None)
    bad = B.PRISM_ERR_INVALID_ARG
    assert lib.prism_linear(None, 1, 16, 16, 16, 16, None, 0, None, 16, None, None) == bad
    assert lib.prism_linear_backward(None, 1, 16, 16, 16, 16, 0, None, None, 16, None) == bad
    assert lib.prism_linear_weight_backward(None, 1, 16, 16, 16, 16, 0, 16, None, None) == bad
    assert lib.prism_heads(None, ctypes.byref(form), 16, 192, 16, 16, 16, None) == bad
    assert lib.prism_heads_backward(None, ctypes.byref(form), 16, 192, 0, 16, 16, 16, 16, 192, None, None, None) == bad
    assert lib.prism_sample(None, 1, 16, 10, 16, None, None, None, None, 16, None, None, None) == bad
    assert B.prism_last_error_message()


def test_the_forms_layout_is_the_headers():
    """Field by field: the sizes and offsets that a C compiler gives the struct (pointers of 8 bytes)."""
    offsets = {name: getattr(B.prism_heads_form, name).offset for name, _ in B.prism_heads_form._fields_}
    assert offsets == {"B": 0, "T": 4, "Hq": 8, "Hk": 12, "Hv": 16, "d": 20, "dv": 24, "norm": 28, "eps": 32, "q_weight": 40, "k_weight": 48,
                       "rot": 56, "interleaved": 60, "inv_freq": 64, "amplitude": 72, "positions": 80}
    assert ctypes.sizeof(B.prism_heads_form) == 88


def arguments():
    x, W, b, r, f = (torch.zeros(*s) for s in ((4, 16), (8, 16), (8,), (4, 8), (2,)))
    rows, q = torch.zeros(2, 2, 16), torch.zeros(2, 1, 2, 4)
    ints, pos = torch.zeros(4, dtype=torch.int32), torch.zeros(2, 2, dtype=torch.int64)
    w4, one = torch.zeros(4), torch.zeros(4)
    heads = dict(heads=(2, 1, 1), d=4, q_weight=w4, k_weight=w4, inv_freq=f, positions=pos)
    q2 = torch.zeros(2, 2, 2, 4)
    return {
        "linear": dict(x=x, W=W, bias=b, residual=r, out={"y": r, "pre": r}),
        "linear_backward": dict(dy=r, W=W, activation="silu", pre=x, dsum=x, dx=x),
        "linear_weight_backward": dict(dy=r, x=x, out={"dW": W, "dbias": b}),
        "heads": dict(x=rows, out={"q": q2, "k": q, "v": q}, **heads),
        "heads_backward": dict(x=rows, grads={"dq": q2, "dk": q, "dv": q}, out={"dx": rows, "dq_weight": w4, "dk_weight": w4}, **heads),
        "sample": dict(logits=torch.zeros(4, 9), u=one, inv_temperature=one, top_k=ints, top_p=one, min_p=one,
                       out={"ids": torch.zeros(4, dtype=torch.int64), "logprob": one, "kept": ints}),
    }


def _walk(args):
    for key, a in args.items():
        if isinstance(a, torch.Tensor):
            yield (key,)
        elif isinstance(a, dict):
            for sub in a:
                yield key, sub


def _with(args, path, change):
    out = {k: dict(v) if isinstance(v, dict) else v for k, v in args.items()}
    if len(path) == 1:
        out[path[0]] = change(out[path[0]])
    else:
        out[path[0]][path[1]] = change(out[path[0]][path[1]])
    return out


def _on(device, a):
    if isinstance(a, torch.Tensor):
        return OnDevice(a, device)
    return {k: _on(device, v) for k, v in a.items()} if isinstance(a, dict) else a


@pytest.mark.parametrize("method", list(arguments()))
def test_tensors_that_do_not_fit_are_refused(tokens, monkeypatch, method):  # noqa: F811
    calls = []
    monkeypatch.setattr(B, "prism_" + method, lambda *a, **k: calls.append(method))
    args = {k: _on(0, a) for k, a in arguments()[method].items()}
    getattr(tokens, method)(**args)
    assert calls == [method]
    calls.clear()
    plain = arguments()[method]

    def broken(t):
        yield "device", OnDevice(t, 1)
        yield "type", OnDevice(t.to(torch.float64), 0)
        yield "size", OnDevice(torch.zeros(*t.shape[:-1], t.shape[-1] + 1, dtype=t.dtype), 0)
        turned = t.transpose(0, 1).contiguous().transpose(0, 1) if t.dim() > 1 else t
        if not turned.is_contiguous():
            yield "layout", OnDevice(turned, 0)

    for path in _walk(plain):
        leaf = plain[path[0]] if len(path) == 1 else plain[path[0]][path[1]]
        for what, bad in broken(leaf):
            if what == "size" and path[-1] in ("x", "dx") and method.startswith("heads"):
                continue  # rows may hold more columns than the heads'
            if what == "size" and path == ("inv_freq",):
                continue  # its length is the rotation's choice; beyond the head the library refuses it
            if what == "layout" and path[-1] == "logits":
                continue  # covered below: padded rows are allowed, other strides are not
            with pytest.raises(ValueError):
                getattr(tokens, method)(**_with(args, path, lambda _, bad=bad: bad))
            assert not calls, (path, what)


def test_names_and_missing_tensors_are_refused(tokens, monkeypatch):  # noqa: F811
    for name in ("prism_linear", "prism_linear_backward", "prism_linear_weight_backward", "prism_heads", "prism_heads_backward", "prism_sample"):
        monkeypatch.setattr(B, name, lambda *a, **k: pytest.fail("the library was called"))
    plain = {m: {k: _on(0, a) for k, a in kw.items()} for m, kw in arguments().items()}
    bad = [("linear", dict(activation="relu")), ("linear", dict(out={"z": plain["linear"]["residual"]})), ("linear", dict(out=None, want=("pre",))),
           ("linear_backward", dict(pre=None)), ("linear_backward", dict(activation="tanh")),
           ("linear_weight_backward", dict(out=None, accumulate=True)), ("linear_weight_backward", dict(out=None, want=("dbias",))),
           ("heads", dict(norm="layer")), ("heads", dict(out={"q": plain["heads"]["out"]["q"]})), ("heads_backward", dict(out={"dx": plain["heads"]["x"], "dz": 0})),
           ("sample", dict(out={"id": 0})), ("sample", dict(out={})), ("linear", dict(out={})), ("linear_weight_backward", dict(out={})), ("heads_backward", dict(out={}))]
    for method, change in bad:
        with pytest.raises(ValueError):
            getattr(tokens, method)(**{**plain[method], **change})
    with pytest.raises(ValueError):  # logits of another stride than padded rows
        tokens.sample(OnDevice(torch.zeros(9, 4).t(), 0), plain["sample"]["u"])


def test_every_method_takes_a_stream():
    for name in arguments():
        assert list(inspect.signature(getattr(B.Tokens, name)).parameters)[-1] == "stream"
