"""Expired waits of the product's tile kernels: they are reported, what was on its way lands before a block leaves, and the handle goes on.

A bound of one nanosecond lets a wait run out that the hardware's own suspension of the waiting thread (some microseconds) does not cover: the sums
here are so long that the warps that finish a tile wait for tens of microseconds."""
import pytest
import torch

from ssm_sequence_layer_gb300 import binding as B
from ssm_sequence_layer_gb300 import build

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
ATTEMPTS = 8


@pytest.fixture(scope="module", autouse=True)
def _built():
    build.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"


def expire(t, calls):
    """Each call reports an expired wait in at least one of its attempts; every other outcome is none."""
    t.set_option(B.PRISM_OPT_WAIT_NS, 1)
    for call in calls:
        n = 0
        for _ in range(ATTEMPTS):
            call()
            torch.cuda.synchronize()
            try:
                t.last_device_status()
            except B.PrismError as e:
                assert e.status == B.PRISM_ERR_TIMEOUT
                n += 1
        assert n > 0
    t.set_option(B.PRISM_OPT_WAIT_NS, 0)


def holds(io, rows, calls):
    """calls(t): before and after the expired waits they give the same bits."""
    with B.Tokens(rows, 64, 64, io=io) as t:
        calls = calls(t)
        before = [call() for call in calls]
        expire(t, calls)
        after = [call() for call in calls]
        torch.cuda.synchronize()
        t.last_device_status()
    assert all(torch.equal(a, b) for a, b in zip(before, after))


def normal(io, *shapes):
    g = torch.Generator().manual_seed(sum(map(sum, shapes)))
    return [torch.randn(*s, generator=g).to(DT[io]).cuda() for s in shapes]


# rows and columns of the result and the length of its sums: tiles of one SM, a block each; single tiles whose sum is split; rows that are no
# whole units, split and not
SINGLE = [(2048, 768, 4096), (1024, 512, 16384), (300, 257, 4097), (2050, 770, 2049)]


def both_ways(t, io, I, J, S):
    x, W, V, add, pre = normal(io, (I, S), (J, S), (S, J), (I, J), (I, J))
    return [lambda: t.linear(x, W, residual=add)["y"], lambda: t.linear(x, W, activation="silu", want=("y", "pre"))["pre"],
            lambda: t.linear_backward(x, V, dsum=add), lambda: t.linear_backward(x, V, activation="gelu", pre=pre, dsum=add)]


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("I,J,S", SINGLE)
def test_expired_waits_are_reported(io, I, J, S):
    holds(io, I, lambda t: both_ways(t, io, I, J, S))
