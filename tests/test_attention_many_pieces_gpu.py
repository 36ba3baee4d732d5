"""Attention and its gradient where a pair of CTAs works on piece after piece: rings, barriers and the boxes that
results leave through are taken over from the piece before, whatever its size was.  A pair takes up to 512
queries (forward) or 256 tokens (gradients) of one head at a time, and a GB300 has 76 of them."""
import pytest
import torch

import test_attention_bwd_gpu as bwd
import test_attention_gpu as fwd

pytestmark = pytest.mark.gpu
BF, HALF = torch.bfloat16, torch.float16


@pytest.fixture(scope="module")
def tb():
    import ln_backward_gb300
    return ln_backward_gb300


def lengths(kind, n):
    """Lengths of n sequences: all of 32 rows and more, all of fewer, or in turn, with whole blocks among them."""
    few, more = [1, 31, 7, 17], [32, 64, 96, 128]
    mixed = [64, 20, 33, 128, 32, 1, 40, 257, 31, 300, 129]
    of = {"few": few, "more": more, "mixed": mixed}[kind]
    return [0] + torch.tensor([of[i % len(of)] for i in range(n)]).cumsum(0).tolist()


def check(tb, b, s, hq, hk, d, dtype, layout="joint", offsets=None):
    q, k, v = fwd.inputs(b, s, hq, hk, d, dtype, layout, seed=d + s)
    out, lse = fwd.check(tb, q, k, v, offsets)
    given = bwd.problem(tb, b, s, hq, hk, d, dtype, layout, seed=d + s, offsets=offsets)
    grads = bwd.check(tb, given, offsets, layout=layout)
    for _ in range(5):
        again, sums = fwd.run(tb, q, k, v, offsets)
        assert torch.equal(again, out) and torch.equal(sums, lse)
        assert all(torch.equal(x, y) for x, y in zip(bwd.run(tb, *given, offsets, layout=layout), grads))


# one box of 32 columns a warp, two in turn, or three of which the first follows the last
@pytest.mark.parametrize("d", [8, 32, 64, 72, 96, 128])
@pytest.mark.parametrize("kind", ["few", "more", "mixed"])
def test_short_sequences_of_many_heads(tb, kind, d):
    offsets = lengths(kind, 33)
    check(tb, 1, offsets[-1], 24, 8, d, [BF, HALF][d // 8 % 2], offsets=offsets)


@pytest.mark.parametrize("b, s, hq, hk, d, dtype", [(2, 1300, 32, 8, 128, BF), (3, 1290, 30, 30, 128, HALF), (1, 2600, 40, 5, 96, BF),
                                                    (4, 1100, 32, 32, 64, HALF)])
def test_pieces_of_several_blocks(tb, b, s, hq, hk, d, dtype):
    check(tb, b, s, hq, hk, d, dtype, "bhsd")


@pytest.mark.parametrize("d", [64, 128])
def test_sequences_of_any_length(tb, d):
    offsets = [0, 700, 701, 1214, 1214, 2504, 2568, 2697, 4430]
    check(tb, 1, 4500, 16, 4, d, BF, offsets=offsets)
