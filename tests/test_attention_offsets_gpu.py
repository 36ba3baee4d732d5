"""Offsets that do not count up within the row: reported by the forward and by the gradient, one list at a time, and
nothing is written but results."""
import pytest
import torch

from test_attention_bwd_gpu import problem
from test_attention_gpu import inputs

pytestmark = pytest.mark.gpu
BF, HALF = torch.bfloat16, torch.float16
S, ROOM = 300, 4096
BAD = {"down": [0, 200, 100, 300], "before": [-5, 100], "behind": [0, S + 100], "far behind": [2 ** 40, 2 ** 41], "far before": [-2 ** 62, -2 ** 61],
       "again": [0, S, 0, S, 0, S], "last": [0, 100, 200, 199], "first": [1, 0, 300], "last end": [0, 100, S + 1],
       "many down": list(range(0, 280)) + [10], "many": [5] * 200 + [4] + [5] * 200, "many behind": [300] * 400 + [301],
       "wide": [0, 2 ** 63 - 1], "none in reach": [-9, -8, -7]}


@pytest.fixture(scope="module")
def tb():
    import ln_backward_gb300
    return ln_backward_gb300


def guarded(like):
    n = like.numel() * like.element_size()
    mem = torch.full((n + 2 * ROOM,), 0xA5, dtype=torch.uint8, device="cuda")
    return mem, mem[ROOM:ROOM + n].view(like.dtype).view(like.shape)


def untouched(held):
    return all((mem[:ROOM] == 0xA5).all() and (mem[-ROOM:] == 0xA5).all() for mem, _ in held)


@pytest.mark.parametrize("name", BAD)
def test_forward(tb, name):
    q, k, v = inputs(1, S, 2, 1, 64, BF, "bshd")
    held = [guarded(q), guarded(torch.empty(1, 2, S, device="cuda"))]
    tb.tb_attention(q, k, v, held[0][1], held[1][1], offsets=torch.tensor(BAD[name], device="cuda"))
    assert tb.tb_device_error() == 1 and tb.tb_device_error() == 0
    assert untouched(held)


# 16 query heads over one: several pieces of them, whose sums are joined
@pytest.mark.parametrize("hq, hk, dtype", [(2, 1, BF), (2, 2, HALF), (16, 1, BF)])
@pytest.mark.parametrize("name", BAD)
def test_gradient(tb, name, hq, hk, dtype):
    dout, q, k, v, out, lse = problem(tb, 1, S, hq, hk, 64, dtype, "bshd")
    size = tb.tb_attention_bwd_workspace_size(1, S, hq, hk, 64, dtype)
    held = [guarded(x) for x in (q, k, v, torch.empty(size, dtype=torch.uint8, device="cuda"))]
    assert tb.tb_device_error() == 0
    tb.tb_attention_bwd(dout, q, k, v, out, lse, *(x for _, x in held), offsets=torch.tensor(BAD[name], device="cuda"))
    assert tb.tb_device_error() == 1 and tb.tb_device_error() == 0
    assert untouched(held)


def test_good_ones_are_not(tb):
    q, k, v = inputs(1, S, 2, 1, 64, BF)
    for good in ([0, S], [0, 0], [S, S], [7], [0] * 300 + [S], [3, 3, 200, 200, 299]):
        tb.tb_attention(q, k, v, torch.empty_like(q), offsets=torch.tensor(good, device="cuda"))
        assert tb.tb_device_error() == 0
