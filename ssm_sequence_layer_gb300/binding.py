"""Thin ctypes binding of the C ABI in ``include/prism.h``.

Argument marshalling only: every step of the forward runs in the CUDA library
``libprism_gb300.so``.  The functions keep the C names.  Tensors are passed as
``torch.Tensor`` (device memory for ``prism_forward``, ``prism_forward_state`` and
``prism_decode_step``, host memory for ``prism_forward_host``) or as raw integer addresses.  There is no fallback: if
the library is missing, the first call raises.
"""
from __future__ import annotations

import ctypes
import os
import threading

from . import build as _build

PRISM_OK = 0
PRISM_ERR_INVALID_ARG = 1
PRISM_ERR_UNSUPPORTED = 2
PRISM_ERR_MISALIGNED = 3
PRISM_ERR_ARCH = 4
PRISM_ERR_CUDA = 5
PRISM_ERR_TIMEOUT = 6
PRISM_ERR_DEVICE = 7

PRISM_F32 = 0
PRISM_BF16 = 1

PRISM_OPT_SEGMENTS = 0
PRISM_OPT_PATH = 1
PRISM_OPT_WAIT_NS = 2
PRISM_OPT_TIMING = 3
PRISM_OPT_OUT_DTYPE = 4

EXPORTED = ("prism_plan", "prism_plan_set_option", "prism_forward", "prism_forward_host",
            "prism_plan_destroy", "prism_workspace_bytes", "prism_plan_last_device_status",
            "prism_status_string", "prism_last_error_message", "prism_version", "prism_plan_kernel_times",
            "prism_forward_noalloc", "prism_forward_state", "prism_decode_step", "prism_forward_nonlinear",
            "prism_project", "prism_backward", "prism_backward_nonlinear",
            "prism_tokens_plan", "prism_tokens_set_option", "prism_tokens_destroy", "prism_tokens_workspace_bytes",
            "prism_tokens_last_device_status", "prism_tokens_kernel_times", "prism_embed", "prism_embed_backward",
            "prism_norm", "prism_norm_backward", "prism_token_logprobs", "prism_token_logprobs_backward",
            "prism_matmul8", "prism_matmul8_weights")


class prism_kernel_time(ctypes.Structure):
    _fields_ = [("name", ctypes.c_char_p), ("ms", ctypes.c_float)]

_lock = threading.Lock()
_LIB = None


class PrismError(RuntimeError):
    def __init__(self, status, message):
        super().__init__(f"{prism_status_string(status)} -- {message}")
        self.status = status


def library_path() -> str:
    return _build.LIB_PATH


def lib():
    """Load the CUDA library (raises if it has not been built)."""
    global _LIB
    if _LIB is not None:
        return _LIB
    with _lock:
        if _LIB is None:
            path = library_path()
            if not os.path.exists(path):
                raise RuntimeError(f"{os.path.basename(path)} is not built; run "
                                   "`python -m ssm_sequence_layer_gb300.build` (needs nvcc)")
            L = ctypes.CDLL(path)
            vp, i, f = ctypes.c_void_p, ctypes.c_int, ctypes.c_void_p
            L.prism_plan.argtypes = [i, i, i, i, i, i, i, ctypes.POINTER(vp)]
            L.prism_plan_set_option.argtypes = [vp, i, ctypes.c_longlong]
            fwd = [vp, vp, vp, vp, f, f, vp, f, f, vp, i, vp, vp]
            L.prism_forward.argtypes = fwd
            L.prism_forward_host.argtypes = fwd
            L.prism_plan_destroy.argtypes = [vp]
            L.prism_workspace_bytes.argtypes = [vp]
            L.prism_workspace_bytes.restype = ctypes.c_size_t
            L.prism_plan_last_device_status.argtypes = [vp]
            L.prism_status_string.argtypes = [i]
            L.prism_status_string.restype = ctypes.c_char_p
            L.prism_last_error_message.restype = ctypes.c_char_p
            L.prism_version.restype = ctypes.c_char_p
            L.prism_plan_kernel_times.argtypes = [vp, ctypes.POINTER(prism_kernel_time), i]
            L.prism_forward_noalloc.argtypes = [i] * 6 + [vp, vp, vp, f, f, vp, f, f, vp, vp, vp,
                                                          ctypes.POINTER(ctypes.c_int)]
            L.prism_forward_noalloc.restype = ctypes.c_int
            L.prism_forward_state.argtypes = fwd[:11] + [vp, f, vp, f, vp, vp]
            L.prism_decode_step.argtypes = fwd[:11] + [vp, f, vp, vp]
            L.prism_forward_nonlinear.argtypes = fwd[:11] + [vp, f, vp, f, vp, vp]
            L.prism_project.argtypes = [vp, i, vp, vp, vp, vp, vp, f, vp]
            L.prism_backward.argtypes = fwd[:11] + [vp, f, f, f] + [f] * 11 + [vp]
            L.prism_backward_nonlinear.argtypes = L.prism_backward.argtypes
            L.prism_plan_kernel_times.restype = ctypes.c_int
            c_f, ll = ctypes.c_float, ctypes.c_longlong
            L.prism_tokens_plan.argtypes = [i, i, i, i, ctypes.POINTER(vp)]
            L.prism_tokens_set_option.argtypes = [vp, i, ll]
            L.prism_tokens_destroy.argtypes = [vp]
            L.prism_tokens_workspace_bytes.argtypes = [vp]
            L.prism_tokens_workspace_bytes.restype = ctypes.c_size_t
            L.prism_tokens_last_device_status.argtypes = [vp]
            L.prism_tokens_kernel_times.argtypes = [vp, ctypes.POINTER(prism_kernel_time), i]
            L.prism_tokens_kernel_times.restype = ctypes.c_int
            L.prism_embed.argtypes = [vp, i, vp, vp, ll, c_f, vp, vp]
            L.prism_embed_backward.argtypes = [vp, i, vp, vp, c_f, i, vp, vp]
            L.prism_norm.argtypes = [vp, i, vp, vp, vp, c_f, vp, vp, vp, vp, vp]
            L.prism_norm_backward.argtypes = [vp, i, vp, vp, c_f, vp, vp, vp, vp, vp]
            L.prism_token_logprobs.argtypes = [vp, i, vp, ll, vp, c_f, i, vp, vp, vp, vp, vp, vp]
            L.prism_token_logprobs_backward.argtypes = [vp, i, vp, ll, vp, c_f, vp, vp, vp, vp, vp, ll, vp]
            L.prism_matmul8.argtypes = [vp, i, i, i, vp, vp, vp, vp, vp, vp]
            L.prism_matmul8_weights.argtypes = [vp, i, i, vp, vp, vp, vp]
            for name in ("prism_tokens_plan", "prism_tokens_set_option", "prism_tokens_destroy",
                         "prism_tokens_last_device_status", "prism_embed", "prism_embed_backward", "prism_norm",
                         "prism_norm_backward", "prism_token_logprobs", "prism_token_logprobs_backward",
                         "prism_matmul8", "prism_matmul8_weights"):
                getattr(L, name).restype = ctypes.c_int
            for name in ("prism_plan", "prism_plan_set_option", "prism_forward", "prism_forward_host",
                         "prism_plan_destroy", "prism_plan_last_device_status", "prism_forward_state",
                         "prism_decode_step", "prism_forward_nonlinear", "prism_project", "prism_backward",
                         "prism_backward_nonlinear"):
                getattr(L, name).restype = ctypes.c_int
            _LIB = L
    return _LIB


def _check(status):
    if status != PRISM_OK:
        raise PrismError(status, prism_last_error_message())
    return status


def _addr(x):
    if x is None:
        return None
    if isinstance(x, int):
        return x
    return x.data_ptr()


def _stream(stream):
    if stream is None:
        return None
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream  # torch.cuda.Stream


def prism_status_string(status: int) -> str:
    return lib().prism_status_string(int(status)).decode()


def prism_last_error_message() -> str:
    return lib().prism_last_error_message().decode()


def prism_version() -> str:
    return lib().prism_version().decode()


def prism_plan(B, H, T, dk, dv, L, io=PRISM_BF16) -> int:
    h = ctypes.c_void_p()
    _check(lib().prism_plan(B, H, T, dk, dv, L, int(io), ctypes.byref(h)))
    return h.value


def prism_plan_set_option(plan, opt, value):
    return _check(lib().prism_plan_set_option(plan, int(opt), int(value)))


def prism_plan_destroy(plan):
    return _check(lib().prism_plan_destroy(plan))


def prism_workspace_bytes(plan) -> int:
    return int(lib().prism_workspace_bytes(plan))


def prism_plan_last_device_status(plan):
    return _check(lib().prism_plan_last_device_status(plan))


def prism_plan_kernel_times(plan, max_kernels=16):
    """[(name, ms), ...] of the last forward (ms = -1 when timing was off)."""
    buf = (prism_kernel_time * max_kernels)()
    n = lib().prism_plan_kernel_times(plan, buf, max_kernels)
    if n < 0:
        raise PrismError(PRISM_ERR_INVALID_ARG, prism_last_error_message())
    return [(buf[i].name.decode(), float(buf[i].ms)) for i in range(min(n, max_kernels))]


def prism_forward(plan, q, k, v, beta, alpha, u, gamma, eta, conv_w, L, out, stream=None):
    return _check(lib().prism_forward(plan, _addr(q), _addr(k), _addr(v), _addr(beta), _addr(alpha), _addr(u),
                                      _addr(gamma), _addr(eta), _addr(conv_w), int(L), _addr(out),
                                      _stream(stream)))


def prism_forward_host(plan, q, k, v, beta, alpha, u, gamma, eta, conv_w, L, out, stream=None):
    return _check(lib().prism_forward_host(plan, _addr(q), _addr(k), _addr(v), _addr(beta), _addr(alpha),
                                           _addr(u), _addr(gamma), _addr(eta), _addr(conv_w), int(L), _addr(out),
                                           _stream(stream)))


def prism_forward_state(plan, q, k, v, beta, alpha, u, gamma, eta, conv_w, L, v_hist, S_init, out, S_final,
                        v_hist_out, stream=None):
    return _check(lib().prism_forward_state(plan, _addr(q), _addr(k), _addr(v), _addr(beta), _addr(alpha),
                                            _addr(u), _addr(gamma), _addr(eta), _addr(conv_w), int(L),
                                            _addr(v_hist), _addr(S_init), _addr(out), _addr(S_final),
                                            _addr(v_hist_out), _stream(stream)))


def prism_forward_nonlinear(plan, q, k, v, beta, alpha, u, gamma, p_gain, conv_w, L, v_hist, S_init, out, S_final,
                            v_hist_out, stream=None):
    return _check(lib().prism_forward_nonlinear(plan, _addr(q), _addr(k), _addr(v), _addr(beta), _addr(alpha),
                                                _addr(u), _addr(gamma), _addr(p_gain), _addr(conv_w), int(L),
                                                _addr(v_hist), _addr(S_init), _addr(out), _addr(S_final),
                                                _addr(v_hist_out), _stream(stream)))


def prism_project(plan, D, X, conv_x, W, u, p, gamma, stream=None):
    return _check(lib().prism_project(plan, int(D), _addr(X), _addr(conv_x), _addr(W), _addr(u), _addr(p),
                                      _addr(gamma), _stream(stream)))


def prism_decode_step(plan, q, k, v, beta, alpha, u, gamma, eta, conv_w, L, v_hist, S, out, stream=None):
    return _check(lib().prism_decode_step(plan, _addr(q), _addr(k), _addr(v), _addr(beta), _addr(alpha),
                                          _addr(u), _addr(gamma), _addr(eta), _addr(conv_w), int(L),
                                          _addr(v_hist), _addr(S), _addr(out), _stream(stream)))


def prism_backward(plan, q, k, v, beta, alpha, u, gamma, eta, conv_w, L, v_hist, S_init, dout, dS_final, dq, dk, dv,
                   dbeta, dalpha, du, dgamma, deta, dconv_w, dv_hist, dS_init, stream=None):
    return _check(lib().prism_backward(plan, _addr(q), _addr(k), _addr(v), _addr(beta), _addr(alpha), _addr(u),
                                       _addr(gamma), _addr(eta), _addr(conv_w), int(L), _addr(v_hist),
                                       _addr(S_init), _addr(dout), _addr(dS_final), _addr(dq), _addr(dk), _addr(dv),
                                       _addr(dbeta), _addr(dalpha), _addr(du), _addr(dgamma), _addr(deta),
                                       _addr(dconv_w), _addr(dv_hist), _addr(dS_init), _stream(stream)))


def prism_backward_nonlinear(plan, q, k, v, beta, alpha, u, gamma, p_gain, conv_w, L, v_hist, S_init, dout, dS_final,
                             dq, dk, dv, dbeta, dalpha, du, dgamma, dp_gain, dconv_w, dv_hist, dS_init, stream=None):
    return _check(lib().prism_backward_nonlinear(plan, _addr(q), _addr(k), _addr(v), _addr(beta), _addr(alpha),
                                                 _addr(u), _addr(gamma), _addr(p_gain), _addr(conv_w), int(L),
                                                 _addr(v_hist), _addr(S_init), _addr(dout), _addr(dS_final),
                                                 _addr(dq), _addr(dk), _addr(dv), _addr(dbeta), _addr(dalpha),
                                                 _addr(du), _addr(dgamma), _addr(dp_gain), _addr(dconv_w),
                                                 _addr(dv_hist), _addr(dS_init), _stream(stream)))


def prism_forward_noalloc(B, H, T, dk, dv, L, q, k, v, beta, alpha, u, gamma, eta, conv_w, out, stream=None,
                          wait=True):
    """The allocation-free forward (see include/prism.h).  With wait=True the call waits for
    the stream and returns the device status word (0 = no condition recorded)."""
    status = ctypes.c_int(0)
    _check(lib().prism_forward_noalloc(B, H, T, dk, dv, L, _addr(q), _addr(k), _addr(v), _addr(beta),
                                       _addr(alpha), _addr(u), _addr(gamma), _addr(eta), _addr(conv_w), _addr(out),
                                       _stream(stream), ctypes.byref(status) if wait else None))
    return status.value


def prism_tokens_plan(max_rows, D, V, io=PRISM_BF16) -> int:
    h = ctypes.c_void_p()
    _check(lib().prism_tokens_plan(max_rows, D, V, int(io), ctypes.byref(h)))
    return h.value


def prism_tokens_set_option(tokens, opt, value):
    return _check(lib().prism_tokens_set_option(tokens, int(opt), int(value)))


def prism_tokens_destroy(tokens):
    return _check(lib().prism_tokens_destroy(tokens))


def prism_tokens_workspace_bytes(tokens) -> int:
    return int(lib().prism_tokens_workspace_bytes(tokens))


def prism_tokens_last_device_status(tokens):
    return _check(lib().prism_tokens_last_device_status(tokens))


def prism_tokens_kernel_times(tokens, max_kernels=16):
    """[(name, ms), ...] of the handle's last call (ms = -1 when timing was off)."""
    buf = (prism_kernel_time * max_kernels)()
    n = lib().prism_tokens_kernel_times(tokens, buf, max_kernels)
    if n < 0:
        raise PrismError(PRISM_ERR_INVALID_ARG, prism_last_error_message())
    return [(buf[i].name.decode(), float(buf[i].ms)) for i in range(min(n, max_kernels))]


def prism_embed(tokens, n, ids, table, ld_table, scale, out, stream=None):
    return _check(lib().prism_embed(tokens, n, _addr(ids), _addr(table), ld_table, scale, _addr(out), _stream(stream)))


def prism_embed_backward(tokens, n, ids, dout, scale, accumulate, dtable, stream=None):
    return _check(lib().prism_embed_backward(tokens, n, _addr(ids), _addr(dout), scale, int(accumulate), _addr(dtable),
                                             _stream(stream)))


def prism_norm(tokens, n, x, residual, weight, eps, sum, y, y8, y_scale, stream=None):
    return _check(lib().prism_norm(tokens, n, _addr(x), _addr(residual), _addr(weight), eps, _addr(sum), _addr(y), _addr(y8),
                                   _addr(y_scale), _stream(stream)))


def prism_norm_backward(tokens, n, sum, weight, eps, dy, dsum, dx, dweight, stream=None):
    return _check(lib().prism_norm_backward(tokens, n, _addr(sum), _addr(weight), eps, _addr(dy), _addr(dsum), _addr(dx),
                                            _addr(dweight), _stream(stream)))


def prism_matmul8(tokens, M, N, K, a8, a_scale, w8, w_scale, out, stream=None):
    return _check(lib().prism_matmul8(tokens, M, N, K, _addr(a8), _addr(a_scale), _addr(w8), _addr(w_scale), _addr(out),
                                      _stream(stream)))


def prism_matmul8_weights(tokens, N, K, W, w8, w_scale, stream=None):
    return _check(lib().prism_matmul8_weights(tokens, N, K, _addr(W), _addr(w8), _addr(w_scale), _stream(stream)))


def prism_token_logprobs(tokens, n, logits, ld, targets, inv_temperature, k, lse, logprob, entropy, top_ids, top_logprob,
                         stream=None):
    return _check(lib().prism_token_logprobs(tokens, n, _addr(logits), ld, _addr(targets), inv_temperature, k, _addr(lse),
                                             _addr(logprob), _addr(entropy), _addr(top_ids), _addr(top_logprob),
                                             _stream(stream)))


def prism_token_logprobs_backward(tokens, n, logits, ld, targets, inv_temperature, lse, entropy, dlogprob, dentropy, dlogits,
                                  ld_d, stream=None):
    return _check(lib().prism_token_logprobs_backward(tokens, n, _addr(logits), ld, _addr(targets), inv_temperature, _addr(lse),
                                                      _addr(entropy), _addr(dlogprob), _addr(dentropy), _addr(dlogits), ld_d,
                                                      _stream(stream)))


# ------------------------------------------------------------------------------------------------
class Plan:
    """Owns a ``prism_plan_t``; ``forward`` marshals a dict of tensors into ``prism_forward``."""

    def __init__(self, B, H, T, dk, dv, L, io="bf16", segments=None, path=None, out=None):
        self.shape = (B, H, T, dk, dv, L)
        self.io = io
        self.out = out or io
        self.handle = prism_plan(B, H, T, dk, dv, L, PRISM_BF16 if io == "bf16" else PRISM_F32)
        if self.out != io:
            prism_plan_set_option(self.handle, PRISM_OPT_OUT_DTYPE, PRISM_BF16 if self.out == "bf16" else PRISM_F32)
        if segments is not None:
            prism_plan_set_option(self.handle, PRISM_OPT_SEGMENTS, segments)
        if path is not None:
            prism_plan_set_option(self.handle, PRISM_OPT_PATH, path)

    @classmethod
    def for_inputs(cls, inp, **kw):
        B, H, T, dk = inp["q"].shape
        dv = inp["v"].shape[-1]
        io = "bf16" if str(inp["q"].dtype).endswith("bfloat16") else "f32"
        return cls(B, H, T, dk, dv, inp["L"], io=io, **kw)

    def set_option(self, opt, value):
        prism_plan_set_option(self.handle, opt, value)

    def workspace_bytes(self):
        return prism_workspace_bytes(self.handle)

    def _tensors(self, inp):
        L = inp["L"]
        lv = L > 1
        return (inp["q"], inp["k"], inp["v"], inp["beta"], inp["alpha"], inp["u"] if lv else None,
                inp["gamma"] if lv else None, inp["eta"] if lv else None, inp["conv_w"], L)

    def forward(self, inp, out=None, stream=None):
        """Device tensors in, device tensor out (allocated if not given)."""
        import torch
        ts = self._tensors(inp)
        for t in ts[:-1]:
            if t is not None and (not t.is_cuda or not t.is_contiguous()):
                raise ValueError("prism_forward takes contiguous CUDA tensors")
        if out is None:
            out = torch.empty(inp["v"].shape, dtype=self._out_torch_dtype(), device=inp["v"].device)
        prism_forward(self.handle, *ts, out, stream)
        return out

    @staticmethod
    def _check_device(ts, what):
        for t in ts:
            if t is not None and (not t.is_cuda or not t.is_contiguous()):
                raise ValueError(f"{what} takes contiguous CUDA tensors")

    def forward_state(self, inp, v_hist=None, S_init=None, S_final=None, v_hist_out=None, out=None, stream=None):
        """One part of a sequence evaluated over consecutive calls (see prism_forward_state):
        v_hist [B,H,3,dv] and S_init [B,H,dv,dk] (fp32) carry the sequence in, S_final and
        v_hist_out carry it out (each may be None; S_final may be S_init, v_hist_out v_hist)."""
        import torch
        ts = self._tensors(inp)
        self._check_device(ts[:-1] + (v_hist, S_init, S_final, v_hist_out), "prism_forward_state")
        if out is None:
            out = torch.empty(inp["v"].shape, dtype=self._out_torch_dtype(), device=inp["v"].device)
        prism_forward_state(self.handle, *ts, v_hist, S_init, out, S_final, v_hist_out, stream)
        return out

    def forward_nonlinear(self, inp, p_gain, v_hist=None, S_init=None, S_final=None, v_hist_out=None, out=None,
                          stream=None):
        """The non-linear residual variant (see prism_forward_nonlinear): p_gain [B,H,T,R,dv] in
        the io dtype takes the place of eta; the state arguments are those of forward_state."""
        import torch
        q, k, v, beta, alpha, u, gamma, _eta, conv_w, L = self._tensors(inp)
        lv = L > 1
        self._check_device((q, k, v, beta, alpha, u, gamma, conv_w, p_gain if lv else None, v_hist, S_init,
                            S_final, v_hist_out), "prism_forward_nonlinear")
        if out is None:
            out = torch.empty(inp["v"].shape, dtype=self._out_torch_dtype(), device=inp["v"].device)
        prism_forward_nonlinear(self.handle, q, k, v, beta, alpha, u, gamma, p_gain if lv else None, conv_w, L,
                                v_hist, S_init, out, S_final, v_hist_out, stream)
        return out

    def project(self, X, conv_x, W, out=None, stream=None):
        """The block's input projections (see prism_project): X [B,T,D], conv_x [4,D], W [N,D],
        bf16 CUDA tensors; returns (u, p, gamma), allocated unless `out` gives them."""
        import torch
        self._check_device((X, conv_x, W), "prism_project")
        B, H, T, dk, dv, L = self.shape
        R = L - 1
        if out is None:
            dev = X.device
            out = (torch.empty(B, H, T, R, dk, dtype=torch.bfloat16, device=dev),
                   torch.empty(B, H, T, R, dv, dtype=torch.bfloat16, device=dev),
                   torch.empty(B, H, T, R, dtype=torch.float32, device=dev))
        u, p, gamma = out
        prism_project(self.handle, X.shape[-1], X, conv_x, W, u, p, gamma, stream)
        return u, p, gamma

    def decode_step(self, inp, v_hist, S, out=None, stream=None):
        """One token per sequence (see prism_decode_step): q, k [B,H,dk], v [B,H,dv], u [B,H,R,dk],
        beta, alpha [B,H], gamma, eta [B,H,R] (a T axis of length 1 is accepted too); v_hist and
        S are updated in place."""
        import torch
        ts = self._tensors(inp)
        self._check_device(ts[:-1] + (v_hist, S), "prism_decode_step")
        if out is None:
            B, H = self.shape[:2]
            out = torch.empty((B, H, self.shape[4]), dtype=self._out_torch_dtype(), device=inp["v"].device)
        prism_decode_step(self.handle, *ts, v_hist, S, out, stream)
        return out

    def backward(self, inp, dout, dS_final=None, v_hist=None, S_init=None, want_dv_hist=False,
                 want_dS_init=False, grads=None, stream=None, p_gain=None):
        """Cotangents of the inputs (see prism_backward): dout [B,H,T,dv] and dS_final
        [B,H,dv,dk] are float32 CUDA tensors (dS_final may be None).  Returns a dict of float32
        tensors dq, dk, dv, dbeta, dalpha, du, dgamma, deta, dconv_w (plus dv_hist and dS_init on
        request), allocated unless `grads` holds them.  With p_gain [B,H,T,R,dv] (io dtype) the
        forward is the non-linear residual variant (see prism_backward_nonlinear): eta is not read
        and dp_gain [B,H,T,R,dv] takes the place of deta."""
        import torch
        ts = self._tensors(inp)
        B, H, T, dk, dv, L = self.shape
        R = L - 1
        nl = p_gain is not None
        if nl:
            ts = ts[:7] + (None,) + ts[8:]
        self._check_device(ts[:-1] + (dout, dS_final, v_hist, S_init, p_gain if R > 0 else None), "prism_backward")
        if grads is None:
            dev = inp["v"].device
            e = lambda *shape: torch.empty(*shape, dtype=torch.float32, device=dev)  # noqa: E731
            grads = {"dq": e(B, H, T, dk), "dk": e(B, H, T, dk), "dv": e(B, H, T, dv), "dbeta": e(B, H, T),
                     "dalpha": e(B, H, T), "du": e(B, H, T, R, dk), "dgamma": e(B, H, T, R),
                     ("dp_gain" if nl else "deta"): e(B, H, T, R, dv) if nl else e(B, H, T, R),
                     "dconv_w": e(H, 4, dv)}
            if want_dv_hist:
                grads["dv_hist"] = e(B, H, 3, dv)
            if want_dS_init:
                grads["dS_init"] = e(B, H, dv, dk)
        g = grads
        lv = R > 0
        self._check_device(tuple(g.values()), "prism_backward")
        if nl:
            q, k, v, beta, alpha, u, gamma, _eta, conv_w, L = ts
            prism_backward_nonlinear(self.handle, q, k, v, beta, alpha, u, gamma, p_gain if lv else None, conv_w, L,
                                     v_hist, S_init, dout, dS_final, g["dq"], g["dk"], g["dv"], g["dbeta"],
                                     g["dalpha"], g["du"] if lv else None, g["dgamma"] if lv else None,
                                     g["dp_gain"] if lv else None, g["dconv_w"], g.get("dv_hist"), g.get("dS_init"),
                                     stream)
            return g
        prism_backward(self.handle, *ts, v_hist, S_init, dout, dS_final, g["dq"], g["dk"], g["dv"], g["dbeta"],
                       g["dalpha"], g["du"] if lv else None, g["dgamma"] if lv else None, g["deta"] if lv else None,
                       g["dconv_w"], g.get("dv_hist"), g.get("dS_init"), stream)
        return g

    def _out_torch_dtype(self):
        import torch
        return torch.bfloat16 if self.out == "bf16" else torch.float32

    def forward_host(self, inp, out=None, stream=None):
        """Host tensors in (pinned for speed), host tensor out; synchronous."""
        import torch
        ts = self._tensors(inp)
        for t in ts[:-1]:
            if t is not None and (t.is_cuda or not t.is_contiguous()):
                raise ValueError("prism_forward_host takes contiguous host tensors")
        if out is None:
            out = torch.empty(inp["v"].shape, dtype=self._out_torch_dtype())
        prism_forward_host(self.handle, *ts, out, stream)
        return out

    def kernel_times(self):
        return prism_plan_kernel_times(self.handle)

    def last_device_status(self):
        return prism_plan_last_device_status(self.handle)

    def close(self):
        if self.handle:
            prism_plan_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def __enter__(self):
        return self

    def __exit__(self, *a):
        self.close()


# ------------------------------------------------------------------------------------------------
class Tokens:
    """Owns a ``prism_tokens_t``: the operators between token ids and the layer, and between the layer
    and token probabilities (see the token operators of include/prism.h).

    ``max_rows`` is the largest number of rows of a call, ``D`` the model width, ``V`` the vocabulary,
    ``io`` the dtype of activations and tables ("bf16" or "f32"), ``logits`` that of logits (``io``
    unless given).  Rows are tokens; leading axes of the arguments are flattened.  Outputs are
    allocated unless given.  ``stream`` (a torch stream or a raw one) is torch's current stream unless
    given; one that is given is the current stream of the call, for the outputs' memory too.
    """

    def __init__(self, max_rows, D, V, io="bf16", logits=None):
        import torch
        self.max_rows, self.D, self.V, self.io = max_rows, D, V, io
        self.logits = logits or io
        dtypes = {"bf16": torch.bfloat16, "f32": torch.float32}
        self._io, self._logits = dtypes[self.io], dtypes[self.logits]
        self._current_stream = torch._C._cuda_getCurrentRawStream
        self.handle = prism_tokens_plan(max_rows, D, V, PRISM_BF16 if io == "bf16" else PRISM_F32)
        self.device = torch.cuda.current_device()
        if self.logits != io:
            self.set_option(PRISM_OPT_OUT_DTYPE, PRISM_BF16 if self.logits == "bf16" else PRISM_F32)

    def set_option(self, opt, value):
        prism_tokens_set_option(self.handle, opt, value)

    def workspace_bytes(self):
        return prism_tokens_workspace_bytes(self.handle)

    def kernel_times(self):
        return prism_tokens_kernel_times(self.handle)

    def last_device_status(self):
        return prism_tokens_last_device_status(self.handle)

    @staticmethod
    def _on(stream, method, *args):
        """The call with ``stream`` as the current one, whose memory the outputs then come from."""
        import torch
        if isinstance(stream, int):
            stream = torch.cuda.ExternalStream(stream) if stream else torch.cuda.default_stream()
        with torch.cuda.stream(stream):
            return method(*args)

    def _need(self, name, t, dtype, numel=None, width=None):
        """Refuses a tensor that the library would misread: its device, type, layout and size."""
        if t.dtype is not dtype or t.get_device() != self.device or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous tensor of {dtype} on the handle's device")
        if (numel is not None and t.numel() != numel) or (width is not None and t.shape[-1] != width):
            raise ValueError(f"{name} has shape {tuple(t.shape)}, which does not fit the other arguments")

    def embed(self, ids, table, scale=1.0, out=None, stream=None):
        """scale * table[ids] (see prism_embed): ids [...] int64, table [V, D] whose rows may be
        padded (a stride); returns [..., D].  Negative ids give rows of zeros."""
        import torch
        if stream is not None:
            return self._on(stream, self.embed, ids, table, scale, out)
        n = ids.numel()
        self._need("ids", ids, torch.int64)
        dense = table.is_contiguous()  # an axis of one element may have any stride
        if table.dtype is not self._io or table.get_device() != self.device or table.shape != (self.V, self.D) or not (dense or table.stride(1) == 1):
            raise ValueError(f"table must be [{self.V}, {self.D}] of {self._io} with contiguous rows on the handle's device")
        if out is None:
            out = torch.empty(*ids.shape, self.D, dtype=self._io, device=ids.device)
        else:
            self._need("out", out, self._io, n * self.D)
        prism_embed(self.handle, n, ids, table, self.D if dense else table.stride(0), scale, out, self._current_stream(self.device))
        return out

    def embed_backward(self, ids, dout, scale=1.0, dtable=None, accumulate=False, stream=None):
        """The table's gradient [V, D] float32 (see prism_embed_backward); with ``accumulate`` it is
        added to ``dtable``."""
        import torch
        if stream is not None:
            return self._on(stream, self.embed_backward, ids, dout, scale, dtable, accumulate)
        n = ids.numel()
        self._need("ids", ids, torch.int64)
        self._need("dout", dout, self._io, n * self.D, self.D)
        if dtable is None:
            if accumulate:
                raise ValueError("accumulate needs a dtable to add to")
            dtable = torch.empty(self.V, self.D, dtype=torch.float32, device=ids.device)
        else:
            self._need("dtable", dtable, torch.float32, self.V * self.D)
        prism_embed_backward(self.handle, n, ids, dout, scale, accumulate, dtable, self._current_stream(self.device))
        return dtable

    def norm(self, x, weight, residual=None, eps=1e-6, want=("y",), out=None, stream=None):
        """The norm of x + residual (see prism_norm): x, residual [..., D], weight [D].  Returns a dict
        of the outputs that ``want`` names -- "sum" and "y" [..., D], "y8" (float8_e4m3fn) with its
        "y_scale" [..., ceil(D/128)] -- or fills and returns ``out``, a dict of them."""
        import torch
        if stream is not None:
            return self._on(stream, self.norm, x, weight, residual, eps, want, out)
        D = self.D
        n = x.numel() // D
        need = self._need
        need("x", x, self._io, n * D, D)
        need("weight", weight, self._io, D)
        if residual is not None:
            need("residual", residual, self._io, n * D)
        if out is None:
            out, lead = {}, x.shape[:-1]
            for key in want:
                if key in ("sum", "y"):
                    out[key] = torch.empty_like(x)
                elif key == "y8":
                    out["y8"] = torch.empty(x.shape, dtype=torch.float8_e4m3fn, device=x.device)
                    out["y_scale"] = torch.empty(*lead, -(-D // 128), dtype=torch.float32, device=x.device)
                else:
                    raise ValueError(f"prism_norm has no output {key!r}")
        else:
            for key, t in out.items():
                if key in ("sum", "y"):
                    need(key, t, self._io, n * D)
                elif key == "y8":
                    need(key, t, torch.float8_e4m3fn, n * D)
                elif key == "y_scale":
                    need(key, t, torch.float32, n * -(-D // 128))
                else:
                    raise ValueError(f"prism_norm has no output {key!r}")
        get = out.get
        prism_norm(self.handle, n, x, residual, weight, eps, get("sum"), get("y"), get("y8"), get("y_scale"), self._current_stream(self.device))
        return out

    def norm_backward(self, sum, weight, dy, dsum=None, eps=1e-6, out=None, stream=None):
        """The norm's gradient (see prism_norm_backward): ``sum`` is the forward's "sum" (x itself
        where there was no residual), dsum the cotangent that reaches it besides the norm's.
        Returns {"dx" [..., D], "dweight" [D] float32}."""
        import torch
        if stream is not None:
            return self._on(stream, self.norm_backward, sum, weight, dy, dsum, eps, out)
        D = self.D
        n = sum.numel() // D
        need = self._need
        need("sum", sum, self._io, n * D, D)
        need("weight", weight, self._io, D)
        need("dy", dy, self._io, n * D)
        if dsum is not None:
            need("dsum", dsum, self._io, n * D)
        if out is None:
            out = {"dx": torch.empty_like(sum), "dweight": torch.empty(D, dtype=torch.float32, device=sum.device)}
        else:
            need("dx", out["dx"], self._io, n * D)
            need("dweight", out["dweight"], torch.float32, D)
        prism_norm_backward(self.handle, n, sum, weight, eps, dy, dsum, out["dx"], out["dweight"], self._current_stream(self.device))
        return out

    def matmul8(self, a8, a_scale, w8, w_scale, out=None, stream=None):
        """The 8-bit product (see prism_matmul8): a8 [..., K] float8_e4m3fn with a_scale
        [..., ceil(K/128)] (norm's "y8" and "y_scale"), w8 [N, K] with w_scale
        [ceil(N/128), ceil(K/128)] (matmul8_weights); returns [..., N] in the logits' dtype."""
        import torch
        if stream is not None:
            return self._on(stream, self.matmul8, a8, a_scale, w8, w_scale, out)
        need, f8, f32 = self._need, torch.float8_e4m3fn, torch.float32
        N, K = w8.shape
        M, kb = a8.numel() // K, -(-K // 128)
        need("a8", a8, f8, M * K, K)
        need("a_scale", a_scale, f32, M * kb, kb)
        need("w8", w8, f8)
        need("w_scale", w_scale, f32, -(-N // 128) * kb, kb)
        if out is None:
            out = torch.empty(*a8.shape[:-1], N, dtype=self._logits, device=a8.device)
        else:
            need("out", out, self._logits, M * N)
        prism_matmul8(self.handle, M, N, K, a8, a_scale, w8, w_scale, out, self._current_stream(self.device))
        return out

    def matmul8_weights(self, W, stream=None):
        """Weights W [N, K] (io dtype) laid out once for matmul8: (w8, w_scale)."""
        import torch
        if stream is not None:
            return self._on(stream, self.matmul8_weights, W)
        N, K = W.shape
        self._need("W", W, self._io)
        w8 = torch.empty(N, K, dtype=torch.float8_e4m3fn, device=W.device)
        w_scale = torch.empty(-(-N // 128), -(-K // 128), dtype=torch.float32, device=W.device)
        prism_matmul8_weights(self.handle, N, K, W, w8, w_scale, self._current_stream(self.device))
        return w8, w_scale

    def _logit_rows(self, name, t):
        """(rows, row stride) of logits [..., V], or [n, V] with padded rows."""
        V = self.V
        if t.dtype is not self._logits or t.get_device() != self.device or t.shape[-1] != V:
            raise ValueError(f"{name} must be [..., {V}] of {self._logits} on the handle's device")
        if t.is_contiguous():
            return t.numel() // V, V
        if t.dim() != 2 or t.stride(1) != 1 or t.stride(0) < V:
            raise ValueError(f"{name} must be contiguous, or [n, {V}] with contiguous rows")
        return t.shape[0], t.stride(0)

    def token_logprobs(self, logits, targets=None, inv_temperature=1.0, k=0, out=None, stream=None):
        """Log probabilities of ``targets`` [...] int64 under softmax(inv_temperature * logits) with
        entropy and the k most likely tokens (see prism_token_logprobs).  Returns a dict of "lse",
        "entropy" [...], with targets "logprob" [...], with k > 0 "top_ids" [..., k] int64 and
        "top_logprob" [..., k]; or fills and returns ``out``, a dict of those that are wanted."""
        import torch
        if stream is not None:
            return self._on(stream, self.token_logprobs, logits, targets, inv_temperature, k, out)
        n, ld = self._logit_rows("logits", logits)
        need, f32, i64 = self._need, torch.float32, torch.int64
        if targets is not None:
            need("targets", targets, i64, n)
        if out is None:
            lead, dev = logits.shape[:-1], logits.device
            out = {key: torch.empty(lead, dtype=f32, device=dev) for key in ("lse", "entropy")}
            if targets is not None:
                out["logprob"] = torch.empty(lead, dtype=f32, device=dev)
            if k > 0:
                out["top_ids"] = torch.empty(*lead, k, dtype=i64, device=dev)
                out["top_logprob"] = torch.empty(*lead, k, dtype=f32, device=dev)
        else:
            for key, t in out.items():
                if key in ("lse", "entropy", "logprob"):
                    need(key, t, f32, n)
                elif key in ("top_ids", "top_logprob"):
                    need(key, t, i64 if key == "top_ids" else f32, n * k)
                else:
                    raise ValueError(f"prism_token_logprobs has no output {key!r}")
        get = out.get
        prism_token_logprobs(self.handle, n, logits, ld, targets, inv_temperature, k, get("lse"), get("logprob"), get("entropy"),
                             get("top_ids"), get("top_logprob"), self._current_stream(self.device))
        return out

    def token_logprobs_backward(self, logits, targets, lse, entropy, dlogprob, dentropy=None, inv_temperature=1.0, dlogits=None,
                                stream=None):
        """The logits' cotangent (see prism_token_logprobs_backward), given the forward's lse and
        entropy (may be None without dentropy); dlogits may be the logits themselves.  Unless given it
        is contiguous where the logits are, and has rows padded by less than 16 bytes where theirs are."""
        import torch
        if stream is not None:
            return self._on(stream, self.token_logprobs_backward, logits, targets, lse, entropy, dlogprob, dentropy, inv_temperature, dlogits)
        n, ld = self._logit_rows("logits", logits)
        need, f32 = self._need, torch.float32
        for name, t in (("lse", lse), ("entropy", entropy), ("dlogprob", dlogprob), ("dentropy", dentropy)):
            if t is not None:
                need(name, t, f32, n)
        if targets is not None:
            need("targets", targets, torch.int64, n)
        if dlogits is None:
            # rows as far from a 16-byte boundary as the logits' are, so that both go in 16-byte units
            ld_d = self.V + (ld - self.V) % (16 // logits.element_size())
            dlogits = torch.empty(*logits.shape[:-1], ld_d, dtype=self._logits, device=logits.device)[..., :self.V]
        else:
            rows, ld_d = self._logit_rows("dlogits", dlogits)
            if rows != n:
                raise ValueError("dlogits must have the logits' rows")
        prism_token_logprobs_backward(self.handle, n, logits, ld, targets, inv_temperature, lse, entropy, dlogprob, dentropy,
                                      dlogits, ld_d, self._current_stream(self.device))
        return dlogits

    def close(self):
        if self.handle:
            prism_tokens_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def __enter__(self):
        return self

    def __exit__(self, *a):
        self.close()
