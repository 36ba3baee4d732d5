"""Bounded waits of attention and of the gated projections, without a GPU fault.

The self-tests run the kernels on small problems with the loads of either CTA of a pair, or a word that
hands over what lies in tensor memory, withheld, so that waits run out after a short limit. Every launch
reports TB_ERR_TIMEOUT and returns with nothing in flight; the calls behind it are right.
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


@pytest.mark.parametrize("name", ["tb_attention_selftest_timeout", "tb_gated_linear_selftest_timeout"])
def test_refusals(tb, name):
    f, n = getattr(tb._binding.lib, name), ctypes.c_int(5)
    for bad in (-1, 0, 999, 1_000_000_001):
        assert f(bad, ctypes.byref(n), None) == INVALID
    assert f(2_000_000, None, None) == INVALID


# a limit that loads and products keep, and the shortest: waits that nothing withholds give up too
@pytest.mark.gpu
@pytest.mark.parametrize("limit_ns", [2_000_000, 1_000])
@pytest.mark.parametrize("name, launches", [("tb_gated_linear_selftest_timeout", 8), ("tb_attention_selftest_timeout", 30)])
def test_waits_run_out_and_the_next_calls_are_right(tb, name, launches, limit_ns):
    from test_attention_and_gated_use_gpu import Attention, Gated, outcome
    calls = [Attention(tb), Gated(tb)]
    want = [outcome(c) for c in calls]
    assert tb.tb_device_error(reset=True) in (OK, TIMEOUT)
    for _ in range(2):
        began = time.perf_counter()
        assert getattr(tb, name)(limit_ns) == launches
        # the way out ends with the last load, not by its own limit of four seconds
        assert time.perf_counter() - began < 3
        assert tb.tb_device_error(reset=True) == TIMEOUT
        assert tb.tb_device_error(reset=True) == OK
        for c, w in zip(calls, want):
            assert all(torch.equal(x, y) for x, y in zip(outcome(c), w))
        assert tb.tb_device_error() == OK
