"""Bounded waits of attention where a sequence ends inside a tile: the self-test's sequence has such an end, whose
loads are counted, mended and handed over by other warps than a whole tile's.  Limits from one that no load keeps to one
that all of them do: whichever warp gives up first, the launches report it, end with their last load (the way out's own
limit is four seconds, of every wait that somebody's missing word would make run out), and the calls behind are right."""
import time

import pytest
import torch

pytestmark = pytest.mark.gpu
OK, TIMEOUT = 0, 9


@pytest.fixture(scope="module")
def tb():
    import ln_backward_gb300
    return ln_backward_gb300


@pytest.mark.parametrize("limit_ns", [1_000, 1_500, 2_000, 2_500, 3_000, 4_000, 5_000, 7_000, 10_000, 20_000, 100_000, 1_000_000])
def test_whichever_wait_runs_out_first(tb, limit_ns):
    from test_attention_and_gated_use_gpu import Attention, outcome
    call = Attention(tb)
    want = outcome(call)
    assert tb.tb_device_error(reset=True) == OK
    for _ in range(4):
        began = time.perf_counter()
        assert tb.tb_attention_selftest_timeout(limit_ns) == tb._binding.TB_ATTENTION_SELFTEST_LAUNCHES
        assert time.perf_counter() - began < 3
        assert tb.tb_device_error(reset=True) == TIMEOUT
        assert all(torch.equal(x, y) for x, y in zip(outcome(call), want))
        assert tb.tb_device_error() == OK
