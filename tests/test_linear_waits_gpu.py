"""Expired waits of the product's tile kernels: they are reported, what was on its way lands before a block leaves, and the handle goes on.

A bound of one nanosecond lets a wait run out that the hardware's own suspension of the waiting thread (some microseconds) does not cover: the sums
here are so long that the warps that finish a tile wait for tens of microseconds.  Only the weights' gradient with operands by TMA has no such wait:
its accumulators hold 512 terms, eight blocks of at most 0.4 microseconds; there every outcome is good that leaves the handle usable."""
import pytest
import torch

from ssm_sequence_layer_gb300 import binding as B
from ssm_sequence_layer_gb300 import build

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
BOUNDS = (1, 1, 1, 2000, 6000, 12000, 25000, 50000)  # nanoseconds: the later ones run out somewhere on the way


@pytest.fixture(scope="module", autouse=True)
def _built():
    build.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"


def expire(t, calls, must):
    """Each call reports an expired wait under at least one of the bounds where it must; every other outcome is none."""
    for call in calls:
        n = 0
        for bound in BOUNDS:
            t.set_option(B.PRISM_OPT_WAIT_NS, bound)
            call()
            torch.cuda.synchronize()
            try:
                t.last_device_status()
            except B.PrismError as e:
                assert e.status == B.PRISM_ERR_TIMEOUT
                n += 1
        assert n > 0 or not must
    t.set_option(B.PRISM_OPT_WAIT_NS, 0)


def holds(io, rows, calls, must=True):
    """calls(t): before and after the expired waits they give the same bits."""
    with B.Tokens(rows, 64, 64, io=io) as t:
        calls = calls(t)
        before = [call() for call in calls]
        expire(t, calls, must)
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


# tiles that two SMs share, in whole turns and with a last one in part
@pytest.mark.parametrize("I,J,S", [(2560, 2304, 4096), (4900, 2000, 8200)])
def test_expired_waits_of_pairs(I, J, S):
    """Either SM of a pair may be ahead with its loads when the waits run out: they land before both leave, time after time."""
    holds("bf16", I, lambda t: both_ways(t, "bf16", I, J, S))


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("rows,I,J", [(16384, 2048, 768), (40000, 300, 520), (20000, 515, 770)])
def test_expired_waits_of_the_weights_gradient(io, rows, I, J):
    """Sums over many rows, split over a cluster of blocks or of pairs of them."""
    dy, x = normal(io, (rows, I), (rows, J))
    holds(io, rows, lambda t: [lambda: t.linear_weight_backward(dy, x)["dW"], lambda: t.linear_weight_backward(dy, x, want=("dW", "dbias"))["dbias"]],
          must=io == "f32" or I % 8 != 0 or J % 8 != 0)
