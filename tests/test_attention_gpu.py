"""Causal attention over whole prompts on the GPU, against its formula in 64 bits (attention_reference.py)."""
import math

import pytest
import torch

import attention_reference as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def tb():
    import ln_backward_gb300
    return ln_backward_gb300


def views(layout, b, s, heads, d, make):
    """Tensors of heads, [b, s, h, d], as they lie in a joint projection's output ("joint"), with heads before
    tokens ("bhsd"), or one behind another ("bshd")."""
    if layout == "joint":
        buf = make((b, s, sum(heads), d))
        return [x for x in buf.split(heads, 2)]
    if layout == "bhsd":
        return [make((b, h, s, d)).transpose(1, 2) for h in heads]
    return [make((b, s, h, d)) for h in heads]


def inputs(b, s, hq, hk, d, dtype, layout="joint", seed=0, std=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return views(layout, b, s, (hq, hk, hk), d, lambda shape: (torch.randn(shape, generator=g, device="cuda") * std).to(dtype))


def run(tb, q, k, v, offsets=None, scale=None, lse=True):
    b, s, hq, d = q.shape
    out = torch.full((b, s, hq, d), -7.0, dtype=q.dtype, device="cuda")
    sums = torch.full((b, hq, s), -7.0, device="cuda")
    o = None if offsets is None else torch.tensor(offsets, device="cuda")
    tb.tb_attention(q, k, v, out, sums if lse else None, offsets=o, scale=scale)
    assert tb.tb_device_error() == 0
    return out, sums


def check(tb, q, k, v, offsets=None, scale=None):
    out, lse = run(tb, q, k, v, offsets, scale)
    want, want_lse, off, lse_off = ref.forward(q, k, v, q.shape[3] ** -0.5 if scale is None else scale, offsets)
    ref.near(out, want, off, "out")
    ref.near(lse, want_lse, lse_off, "lse")
    # tokens of no sequence are left as they were
    assert (out[want.isnan()] == -7.0).all() and (lse[want_lse.isnan()] == -7.0).all()
    return out, lse


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("s", [1, 2, 7, 8, 64, 127, 128, 129, 255, 256, 257, 300, 384, 511, 513, 1000])
def test_lengths(tb, s, dtype):
    check(tb, *inputs(2, s, 4, 2, 128, dtype, seed=s))


@pytest.mark.parametrize("layout", ["joint", "bhsd", "bshd"])
@pytest.mark.parametrize("d", [8, 16, 24, 40, 64, 72, 80, 96, 104, 128])
def test_head_sizes(tb, d, layout):
    check(tb, *inputs(2, 333, 3, 1, d, [torch.bfloat16, torch.float16][d // 8 % 2], layout, seed=d))


@pytest.mark.parametrize("hq, hk", [(1, 1), (8, 1), (6, 3), (5, 5), (16, 2)])
def test_groups(tb, hq, hk):
    check(tb, *inputs(1, 400, hq, hk, 64, torch.bfloat16, seed=hq))


PACKED = {"ragged": [0, 97, 98, 98, 226, 482, 483, 900, 1000], "tail": [0, 130, 300], "head": [5, 133, 260],
          "one": [0, 1], "empty": [0, 0, 0, 0], "aligned": [0, 128, 256, 512], "end": [990, 1000, 1000]}


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("name", PACKED)
def test_packed(tb, name, d, dtype):
    q, k, v = inputs(1, 1000, 4, 2, d, dtype, seed=d)
    check(tb, q, k, v, PACKED[name])


def test_many_short_sequences(tb):
    g = torch.Generator().manual_seed(3)
    lens = torch.randint(0, 12, (1500,), generator=g)
    o = [0] + lens.cumsum(0).tolist()
    check(tb, *inputs(1, o[-1] + 3, 2, 1, 64, torch.bfloat16, seed=1), o)


@pytest.mark.parametrize("d", [64, 128])
def test_what_lies_outside_a_sequence_reaches_nothing(tb, d):
    q, k, v = inputs(1, 700, 4, 2, d, torch.bfloat16, "bshd", seed=2)
    offsets = [10, 200, 201, 465]
    want, lse = check(tb, q, k, v, offsets)
    for t in (q, k, v):
        t[:, :10] = math.nan
        t[:, 465:] = math.inf
    out, sums = run(tb, q, k, v, offsets)
    assert torch.equal(out, want) and torch.equal(sums, lse)
    # nor does one sequence's token reach another's
    q, k, v = inputs(1, 700, 4, 2, d, torch.bfloat16, "bshd", seed=2)
    for t in (q, k, v):
        t[:, 10:200] = math.nan
        t[:, 201:465] = math.nan
    out, sums = run(tb, q, k, v, offsets)
    assert torch.equal(out[:, 200], want[:, 200]) and torch.equal(sums[..., 200], lse[..., 200])


@pytest.mark.parametrize("std", [0.01, 4.0, 30.0])
def test_flat_and_peaked_rows(tb, std):
    check(tb, *inputs(1, 700, 2, 2, 128, torch.bfloat16, seed=5, std=std))


def test_growing_scores(tb):
    """Keys whose scores grow from the last to the first: the maximum moves in every block."""
    q, k, v = inputs(1, 1200, 2, 1, 64, torch.bfloat16, "bshd", seed=6)
    q[..., 0] = 8.0
    k[..., 0] = torch.linspace(60, 0, 1200, device="cuda").to(torch.bfloat16)[None, :, None]
    check(tb, q, k, v)


def test_no_sums_wanted(tb):
    q, k, v = inputs(2, 200, 4, 4, 64, torch.bfloat16)
    out, lse = run(tb, q, k, v)
    again, sums = run(tb, q, k, v, lse=False)
    assert torch.equal(out, again) and (sums == -7.0).all() and not (lse == -7.0).any()


def test_bad_offsets_are_reported(tb):
    q, k, v = inputs(1, 300, 2, 1, 64, torch.bfloat16)
    for bad in ([0, 200, 100, 300], [-5, 100], [0, 400], [2 ** 40, 2 ** 41]):
        out = torch.zeros_like(q)
        tb.tb_attention(q, k, v, out, offsets=torch.tensor(bad, device="cuda"))
        torch.cuda.synchronize()
    assert tb.tb_device_error() == 1 and tb.tb_device_error() == 0
