"""Bounded waits of the output layer's products, without a GPU fault.

The self-test runs the product of one pair of CTAs with the copies of either CTA, the word that an
accumulator is complete, or the word that it is free again withheld, so that waits run out after a
short limit. Every launch reports TB_ERR_TIMEOUT and returns with nothing in flight; the calls behind
it are right.
"""
import ctypes
import time

import pytest
import torch

OK, INVALID, TIMEOUT = 0, 1, 9


@pytest.fixture(scope="module")
def tb():
    import __graft_entry__
    __graft_entry__.build()
    import ln_backward_gb300
    return ln_backward_gb300


def test_refusals(tb):
    f, n = tb._binding.lib.tb_linear_xent_selftest_timeout, ctypes.c_int(5)
    for bad in (-1, 0, 999, 1_000_000_001):
        assert f(bad, ctypes.byref(n), None) == INVALID
    assert f(2_000_000, None, None) == INVALID
    with pytest.raises(tb.TbError):
        tb.tb_linear_xent_selftest_timeout(999, stream=0)


# a limit that copies and products keep, and the shortest: waits that nothing withholds give up too, and
# the two CTAs' producers at different stages
@pytest.mark.gpu
@pytest.mark.parametrize("limit_ns", [2_000_000, 1_000])
@pytest.mark.parametrize("times", [1, 4])
def test_waits_run_out_and_the_next_calls_are_right(tb, limit_ns, times):
    import test_linear_xent_gpu as cases
    H, W, t, dloss = cases.problem(300, 200, 2049, torch.bfloat16, 31)
    want = cases.forward(tb, H, W, t)
    want += cases.backward(tb, dloss, H, W, t, want[1])
    assert tb.tb_device_error(reset=True) in (OK, TIMEOUT)
    for _ in range(times):
        began = time.perf_counter()
        assert tb.tb_linear_xent_selftest_timeout(limit_ns) == tb._binding.TB_LINEAR_XENT_SELFTEST_LAUNCHES
        # the way out ends with the last copy, not by its own limit of four seconds
        assert time.perf_counter() - began < 0.9
        assert tb.tb_device_error(reset=True) == TIMEOUT
        assert tb.tb_device_error(reset=True) == OK
        got = cases.forward(tb, H, W, t)
        got += cases.backward(tb, dloss, H, W, t, got[1])
        assert tb.tb_device_error() == OK
        for x, y in zip(got, want):
            assert torch.equal(x, y)
    cases.check_forward(*want[:2], H, W, t)
    cases.check_backward(*want[2:], dloss, H, W, t, want[1])
