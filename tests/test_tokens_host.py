"""Checks of the token operators' entry points that need no GPU: sizes and null handles are refused
before a device is touched."""
import ctypes

import pytest

from ssm_sequence_layer_gb300 import binding as B
from ssm_sequence_layer_gb300 import build


@pytest.fixture(scope="module")
def lib():
    build.build()
    return B.lib()


@pytest.mark.parametrize("args,status", [
    ((0, 64, 10, 1), B.PRISM_ERR_INVALID_ARG),
    ((8, 0, 10, 1), B.PRISM_ERR_INVALID_ARG),
    ((8, 64, 0, 1), B.PRISM_ERR_INVALID_ARG),
    ((8, 64, 10, 5), B.PRISM_ERR_INVALID_ARG),
    ((1 << 25, 64, 10, 1), B.PRISM_ERR_UNSUPPORTED),
    ((8, 65537, 10, 1), B.PRISM_ERR_UNSUPPORTED),
    ((8, 64, (1 << 30) + 1, 1), B.PRISM_ERR_UNSUPPORTED),
])
def test_plan_refuses_bad_sizes(lib, args, status):
    h = ctypes.c_void_p(1234)
    assert lib.prism_tokens_plan(*args, ctypes.byref(h)) == status
    assert h.value is None
    assert B.prism_last_error_message()
    assert lib.prism_tokens_plan(8, 64, 10, 1, None) == B.PRISM_ERR_INVALID_ARG


def test_null_handle(lib):
    assert lib.prism_tokens_destroy(None) == B.PRISM_OK
    assert lib.prism_tokens_workspace_bytes(None) == 0
    assert lib.prism_tokens_last_device_status(None) == B.PRISM_ERR_INVALID_ARG
    assert lib.prism_tokens_set_option(None, 3, 1) == B.PRISM_ERR_INVALID_ARG
    assert lib.prism_tokens_kernel_times(None, None, 0) == -1
    assert lib.prism_embed(None, 1, 16, 16, 64, 1.0, 16, None) == B.PRISM_ERR_INVALID_ARG
    assert lib.prism_embed_backward(None, 1, 16, 16, 1.0, 0, 16, None) == B.PRISM_ERR_INVALID_ARG
    assert lib.prism_norm(None, 1, 16, None, 16, 1e-6, None, 16, None, None, None) == B.PRISM_ERR_INVALID_ARG
    assert lib.prism_norm_backward(None, 1, 16, 16, 1e-6, 16, None, 16, 16, None) == B.PRISM_ERR_INVALID_ARG
    assert lib.prism_token_logprobs(None, 1, 16, 10, 16, 1.0, 0, 16, 16, 16, None, None, None) == B.PRISM_ERR_INVALID_ARG
    assert lib.prism_token_logprobs_backward(None, 1, 16, 10, 16, 1.0, 16, 16, 16, None, 16, 10, None) == B.PRISM_ERR_INVALID_ARG
    assert lib.prism_matmul8(None, 1, 16, 16, 16, 16, 16, 16, 16, None) == B.PRISM_ERR_INVALID_ARG
    assert lib.prism_matmul8_weights(None, 16, 16, 16, 16, 16, None) == B.PRISM_ERR_INVALID_ARG
