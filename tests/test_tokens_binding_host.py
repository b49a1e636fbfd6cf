"""What the Python side of the token operators refuses before the library is called; needs no GPU."""
import pytest
import torch

from ssm_sequence_layer_gb300 import binding as B


class OnDevice:
    """A tensor's face: a contiguous CUDA tensor of one device."""
    is_cuda = True

    def __init__(self, like, device):
        self.like, self.index = like, device
        self.dtype, self.shape = like.dtype, like.shape
        self.device = torch.device("cuda", device)

    def get_device(self):
        return self.index

    def __getattr__(self, name):
        return getattr(self.like, name)


@pytest.fixture
def tokens():
    t = B.Tokens.__new__(B.Tokens)  # no handle: the refusals come first
    t.handle, t.device = None, 0
    t.max_rows, t.D, t.V, t.io, t.logits = 4, 16, 9, "f32", "f32"
    t._io = t._logits = torch.float32
    t._current_stream = lambda device: 0
    return t


def test_tensors_of_another_device_are_refused(tokens, monkeypatch):
    ids, x, w = torch.zeros(4, dtype=torch.int64), torch.zeros(4, 16), torch.zeros(16)
    table, logits, rows = torch.zeros(9, 16), torch.zeros(4, 9), torch.zeros(4)
    calls = []
    for name in ("prism_embed", "prism_embed_backward", "prism_norm", "prism_norm_backward", "prism_token_logprobs",
                 "prism_token_logprobs_backward", "prism_matmul8", "prism_matmul8_weights"):
        monkeypatch.setattr(B, name, lambda *a, name=name, **k: calls.append(name))
    a8, w8 = torch.zeros(4, 16).to(torch.float8_e4m3fn), torch.zeros(9, 16).to(torch.float8_e4m3fn)
    s, out8 = torch.zeros(4, 1), torch.zeros(4, 9)
    arguments = {
        "embed": (ids, table, 1.0, x), "embed_backward": (ids, x, 1.0, table), "norm": (x, w, x, 1e-6, (), {"y": x}),
        "norm_backward": (x, w, x, x, 1e-6, {"dx": x, "dweight": w}), "matmul8": (a8, s, w8, torch.zeros(1, 1), out8),
        "token_logprobs": (logits, ids, 1.0, 0, {"lse": rows}),
        "token_logprobs_backward": (logits, ids, rows, rows, rows, rows, 1.0, logits)}

    def on(device, a):
        if isinstance(a, torch.Tensor):
            return OnDevice(a, device)
        return {k: on(device, v) for k, v in a.items()} if isinstance(a, dict) else a

    for method, args in arguments.items():
        getattr(tokens, method)(*(on(0, a) for a in args))  # all on the handle's device: the call is made
        assert calls.pop() == "prism_" + method
        for i, a in enumerate(args):
            if isinstance(a, (torch.Tensor, dict)):
                with pytest.raises(ValueError):
                    getattr(tokens, method)(*(on(1 if j == i else 0, b) for j, b in enumerate(args)))
                assert not calls, (method, i)
    with pytest.raises(ValueError):
        tokens.matmul8_weights(OnDevice(torch.zeros(9, 16), 1))
