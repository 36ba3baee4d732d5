"""Attention whose scores lie far from zero: keys masked by low values, rows of large scores only, and scores beyond
fp32's range, against the formula in 64 bits.

Every score here is a sum of products that fp32 holds exactly, whatever their order: multiples of the last place of
the largest.  So P differs from the formula's by what is done behind the scores: a row's maximum is taken off (exact
between neighbours), the difference times scale * log2(e) has three roundings of itself, the power 2 ulp.  A log
sum is a score, rounded to fp32, and the logarithm of a sum, added with one rounding.
"""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu
F32 = 2.0 ** -23
BF, HALF = torch.bfloat16, torch.float16


@pytest.fixture(scope="module")
def tb():
    import ln_backward_gb300
    return ln_backward_gb300


def zeros(n, h, d, dtype):
    return torch.zeros(1, n, h, d, dtype=dtype, device="cuda")


def values(n, h, d, dtype, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(1, n, h, d, generator=g, device="cuda").to(dtype)


def small(n, h, d, seed, dims=8):
    """Quarters up to 2 in a few elements: products of two are multiples of 2^-4, their sums exact."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.zeros(1, n, h, d, device="cuda")
    x[..., 1:1 + dims] = torch.randint(-8, 9, (1, n, h, dims), generator=g, device="cuda") / 4
    return x


def scores(q, k, scale):
    """[heads, n, n] in 64 bits, keys behind the query at -inf."""
    n, group = q.shape[1], q.shape[2] // k.shape[2]
    s = torch.einsum("ihd,jhd->hij", q[0].double(), k[0].double().repeat_interleave(group, 1)) * scale
    return s.masked_fill_(torch.ones(n, n, dtype=torch.bool, device="cuda").triu(1), -math.inf)


def forward(tb, q, k, v, scale):
    out, lse = torch.full_like(q, -7.0), torch.full((1, q.shape[2], q.shape[1]), -7.0, device="cuda")
    tb.tb_attention(q, k, v, out, lse, scale=scale)
    assert tb.tb_device_error() == 0
    return out, lse


def check_forward(tb, q, k, v, scale):
    scale = torch.tensor(scale, dtype=torch.float32).item()
    out, lse = forward(tb, q, k, v, scale)
    half, group = torch.finfo(q.dtype).eps / 2, q.shape[2] // k.shape[2]
    n = q.shape[1]
    s = scores(q, k, scale)
    vv = v[0].double().repeat_interleave(group, 1)
    p = torch.softmax(s, -1)
    near = (s - s.amax(-1, keepdim=True)).clamp(min=-200).abs()
    e = 8 * F32 * (1 + near)
    want = torch.einsum("hij,jhd->ihd", p, vv)
    # the sums are off by what their P are; one rounding of P, sums that truncate, and powers below the type's numbers
    slack = torch.einsum("hij,jhd->ihd", p * (e + half + (n / 16 + 32) * F32), vv.abs()) \
        + want.abs() * ((p * e).sum(-1).T[..., None] + 4 * F32) \
        + torch.finfo(q.dtype).smallest_normal * half * vv.abs().sum(0)
    off = (out[0].double() - want).abs()
    assert (off <= half * (want.abs() + slack) + slack).all(), off.max().item()
    sums = torch.logsumexp(s, -1)
    lse_off = (lse[0].double() - sums).abs()
    bound = F32 / 2 * (s.amax(-1).abs() + sums.abs()) + (p * e).sum(-1) + (n / 16 + 16) * F32
    assert (lse_off <= bound).all(), (lse_off - bound).max().item()
    return out, lse


def masked(n, hq, hk, d, dtype, low, dead, seed=0):
    """Queries and keys of small scores, the keys in `dead` at `low` below them by one element.  A dead key's other
    elements are 0: its scores are one number."""
    q, k = small(n, hq, d, seed), small(n, hk, d, seed + 1)
    root = 2.0 ** (math.frexp(low)[1] // 2)
    q[..., 0] = root
    for a, b in dead:
        k[:, a:b] = 0
        k[:, a:b, :, 0] = -low / root
    return q.to(dtype), k.to(dtype), values(n, hk, d, dtype, seed + 2)


# whole blocks of keys that nobody sees: the last of a row's, its first, the first of all, all up to some row
DEAD = {"own": [(128, 300)], "first": [(0, 130)], "between": [(100, 260), (300, 511)], "all": [(0, 600)], "odd": [(1, 2), (131, 257)]}


@pytest.mark.parametrize("dtype, low", [(BF, 1e4), (BF, 3e8), (BF, 2.0 ** 30), (BF, 1e10), (BF, 1e30), (HALF, 1e4), (HALF, 3e8), (HALF, 2.0 ** 29)])
@pytest.mark.parametrize("name", DEAD)
def test_keys_masked_by_low_values(tb, name, dtype, low):
    q, k, v = masked(600, 2, 1, 64, dtype, low, DEAD[name])
    check_forward(tb, q, k, v, 0.25)


def large(n, hq, hk, d, dtype, size, seed=0):
    """All scores next to `size` (a power of two, either sign), a few steps of 2^-21 of it apart."""
    q, k = zeros(n, hq, d, torch.float32), zeros(n, hk, d, torch.float32)
    step = abs(size) * 4 * F32
    root = 2.0 ** (math.frexp(abs(size))[1] // 2)
    g = torch.Generator(device="cuda").manual_seed(seed)
    q[..., 0], k[..., 0] = root, size / root
    q[..., 1] = 2.0 ** (math.frexp(step)[1] // 2)
    k[..., 1] = torch.randint(-3, 4, (1, n, hk), generator=g, device="cuda") * (step / q[0, 0, 0, 1])
    return q.to(dtype), k.to(dtype), values(n, hk, d, dtype, seed + 1)


@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("dtype, power", [(BF, 12), (BF, 20), (BF, 21), (BF, 25), (BF, 29), (BF, 33), (BF, 60), (BF, 100),
                                          (HALF, 12), (HALF, 20), (HALF, 23), (HALF, 26), (HALF, 29)])
@pytest.mark.parametrize("scale", [0.25, 0.3, 0.088388346])
def test_rows_of_scores_far_from_zero(tb, dtype, power, sign, scale):
    q, k, v = large(300, 2, 1, 64, dtype, sign * 2.0 ** power, seed=power)
    check_forward(tb, q, k, v, scale)


@pytest.mark.parametrize("d", [64, 128])
def test_scores_that_grow_far_from_zero(tb, d):
    """Each block's scores lie above those of the blocks behind it: the maximum moves in every block, by little and by
    far, from rows near zero to rows far from it and back."""
    n, steps = 1100, [0, -2.0 ** 12, -2.0 ** 22, -2.0 ** 23, 2.0 ** 24, 2.0 ** 18, 1.0, -2.0 ** 30, 2.0 ** 29]
    q, k, v = zeros(n, 2, d, BF), zeros(n, 1, d, BF), values(n, 1, d, BF, 3)
    q[..., 0] = 1.0
    for i in range(n):
        k[:, i, :, 0] = steps[8 - i // 128]
    check_forward(tb, q, k, v, 0.5)


@pytest.mark.parametrize("dead", [[(128, 300)], [(5, 400)]])
def test_scores_below_all_numbers(tb, dead):
    """Masked keys whose scores overflow to -inf, among them all of a row's own block; real ones of low scores before."""
    q, k, v = masked(400, 2, 1, 64, BF, 2.0 ** 200, dead)
    k[:, :100, :, 9], q[..., 9] = -256.0, 16.0
    check_forward(tb, q, k, v, 0.25)
