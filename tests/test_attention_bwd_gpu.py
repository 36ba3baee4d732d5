"""The gradient of causal attention on the GPU, against its formula in 64 bits (attention_reference.py)."""
import math

import pytest
import torch

import attention_reference as ref
from test_attention_gpu import PACKED, views

pytestmark = pytest.mark.gpu
BF, HALF = torch.bfloat16, torch.float16


@pytest.fixture(scope="module")
def tb():
    import ln_backward_gb300
    return ln_backward_gb300


def problem(tb, b, s, hq, hk, d, dtype, layout="joint", seed=0, std=1.0, grad=None, offsets=None, scale=None):
    """dout, q, k, v, out, lse: the forward's results by the framework's own forward."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    make = lambda shape: (torch.randn(shape, generator=g, device="cuda") * std).to(dtype)
    q, k, v = views(layout, b, s, (hq, hk, hk), d, make)
    dout, = views("bhsd" if layout == "bhsd" else "bshd", b, s, (hq,), d, make)
    dout.mul_((1e-3 if dtype == BF else 0.1) if grad is None else grad / std)
    out, lse = torch.zeros_like(dout), torch.zeros(b, hq, s, device="cuda")
    tb.tb_attention(q, k, v, out, lse, offsets=None if offsets is None else torch.tensor(offsets, device="cuda"), scale=scale)
    return dout, q, k, v, out, lse


def run(tb, dout, q, k, v, out, lse, offsets=None, scale=None, layout="joint"):
    b, s, hq, d = q.shape
    hk = k.shape[2]
    grads = views(layout, b, s, (hq, hk, hk), d, lambda shape: torch.full(shape, -7.0, dtype=q.dtype, device="cuda"))
    ws = torch.full((tb.tb_attention_bwd_workspace_size(b, s, hq, hk, d, q.dtype),), 0xFF, dtype=torch.uint8, device="cuda")
    tb.tb_attention_bwd(dout, q, k, v, out, lse, *grads, ws,
                        offsets=None if offsets is None else torch.tensor(offsets, device="cuda"), scale=scale)
    assert tb.tb_device_error() == 0
    return grads


def check(tb, given, offsets=None, scale=None, layout="joint"):
    grads = run(tb, *given, offsets, scale, layout)
    q = given[1]
    want, off = ref.backward(*given, q.shape[3] ** -0.5 if scale is None else scale, offsets)
    for got, w, o, name in zip(grads, want, off, ("dq", "dk", "dv")):
        ref.near(got, w, o, name)
        assert (got[w.isnan()] == -7.0).all()     # tokens of no sequence are left as they were
    return grads


@pytest.mark.parametrize("dtype", [BF, HALF])
@pytest.mark.parametrize("s", [1, 2, 7, 8, 64, 127, 128, 129, 255, 256, 257, 300, 384, 511, 513, 1000])
def test_lengths(tb, s, dtype):
    check(tb, problem(tb, 2, s, 4, 2, 128, dtype, seed=s))


@pytest.mark.parametrize("layout", ["joint", "bhsd", "bshd"])
@pytest.mark.parametrize("d", [8, 16, 24, 40, 64, 72, 80, 96, 104, 128])
def test_head_sizes(tb, d, layout):
    check(tb, problem(tb, 2, 333, 3, 1, d, [BF, HALF][d // 8 % 2], layout, seed=d), layout=layout)


@pytest.mark.parametrize("hq, hk", [(1, 1), (8, 1), (6, 3), (5, 5), (16, 2)])
def test_groups(tb, hq, hk):
    check(tb, problem(tb, 1, 400, hq, hk, 64, BF, seed=hq))


@pytest.mark.parametrize("layout", ["joint", "bhsd"])
@pytest.mark.parametrize("b, s, hq, hk, d, dtype", [(1, 600, 8, 1, 128, BF), (2, 300, 12, 1, 64, HALF), (1, 2100, 8, 2, 72, BF),
                                                    (1, 1030, 30, 3, 64, HALF), (3, 257, 16, 2, 128, HALF), (1, 129, 64, 1, 24, BF)])
def test_query_heads_in_several_pieces(tb, b, s, hq, hk, d, dtype, layout):
    """Few tiles of keys, many query heads: several pairs of CTAs share a key head, and their sums are joined."""
    check(tb, problem(tb, b, s, hq, hk, d, dtype, layout, seed=s), layout=layout)


@pytest.mark.parametrize("offsets", [[0, 130, 300], [7, 8, 8, 640], [0, 1000]])
def test_packed_in_several_pieces(tb, offsets):
    check(tb, problem(tb, 1, 1000, 8, 1, 64, BF, seed=5, offsets=offsets), offsets)


@pytest.mark.parametrize("dtype", [BF, HALF])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("name", PACKED)
def test_packed(tb, name, d, dtype):
    check(tb, problem(tb, 1, 1000, 4, 2, d, dtype, seed=d, offsets=PACKED[name]), PACKED[name])


def test_many_short_sequences(tb):
    g = torch.Generator().manual_seed(3)
    o = [0] + torch.randint(0, 12, (1500,), generator=g).cumsum(0).tolist()
    check(tb, problem(tb, 1, o[-1] + 3, 2, 1, 64, BF, seed=1, offsets=o), o)


@pytest.mark.parametrize("dtype", [BF, HALF])
@pytest.mark.parametrize("d", [64, 128])
def test_what_lies_outside_a_sequence_reaches_nothing(tb, d, dtype):
    offsets = [10, 200, 201, 465]
    given = problem(tb, 1, 700, 4, 2, d, dtype, "bshd", seed=2, offsets=offsets)
    want = check(tb, given, offsets)
    for t in given[:5]:
        t[:, :10] = math.nan
        t[:, 465:] = math.inf
    given[0][:, 600:] = 3e4                       # a large gradient of a token that takes no part
    given[5][..., :10] = math.nan
    given[5][..., 465:] = -math.inf
    for a, b in zip(run(tb, *given, offsets), want):
        assert torch.equal(a, b)
    if dtype == BF:                               # (fp16's powers of two go by all sequences)
        for t in given[:5]:
            t[:, 10:200] = math.nan
            t[:, 201:465] = math.nan
        for a, b in zip(run(tb, *given, offsets), want):
            assert torch.equal(a[:, 200], b[:, 200])


@pytest.mark.parametrize("dtype", [BF, HALF])
@pytest.mark.parametrize("std", [0.01, 4.0])
def test_flat_and_peaked_rows(tb, std, dtype):
    check(tb, problem(tb, 1, 700, 2, 2, 128, dtype, seed=5, std=std, grad=1e-3 if dtype == BF else 0.1))


@pytest.mark.parametrize("grad", [2.0 ** -13, 1.0, 60.0])
def test_fp16_gradients_of_any_size(tb, grad):
    check(tb, problem(tb, 1, 900, 2, 1, 64, HALF, seed=6, grad=grad))


def test_against_differences(tb):
    """The loss sum(dout * out) of the forward in 64 bits, a step along the gradient's direction to either side."""
    given = problem(tb, 1, 140, 2, 1, 64, BF, seed=8, grad=1.0)
    dout, q, k, v = given[:4]
    grads = run(tb, *given)
    gen = torch.Generator(device="cuda").manual_seed(9)
    for i, (x, g) in enumerate(zip((q, k, v), grads)):
        way = torch.randn(x.shape, generator=gen, device="cuda", dtype=torch.float64)
        h, side = 1e-4, []
        for sign in (1, -1):
            args = [t.double() for t in (q, k, v)]
            args[i] = args[i] + sign * h * way
            side.append((ref.forward(*args, 64 ** -0.5)[0] * dout.double()).sum().item())
        slope = (side[0] - side[1]) / (2 * h)
        # dq, dk, dv have a half step of rounding on the way and at the end, out and lse one each
        assert abs(slope - (g.double() * way).sum().item()) <= 4 * 2.0 ** -8 * (g.double() * way).norm().item() * 3


def test_twice_the_same(tb):
    given = problem(tb, 2, 700, 8, 2, 128, BF, seed=11)
    for a, b in zip(run(tb, *given), run(tb, *given)):
        assert torch.equal(a, b)
