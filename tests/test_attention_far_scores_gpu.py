"""Attention whose scores lie far from zero: keys masked by low values, rows of large scores only, and scores beyond
fp32's range, and their gradients, against the formula in 64 bits.

Every score here is a sum of products that fp32 holds exactly, whatever their order: multiples of the last place of
the largest.  So P differs from the formula's by what is done behind the scores: a row's maximum is taken off (exact
between neighbours), the difference times scale * log2(e) has three roundings of itself, the power 2 ulp.  A log
sum is a score, rounded to fp32, and the logarithm of a sum, added with one rounding.  The gradient's P comes from
a score and a log sum as it is given: each is off by half a step of fp32, the score by nothing where scale is a power of
two and the log sum is so large that it is taken off the score itself.
"""
import math

import pytest
import torch

import attention_reference as ref

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


def check_backward(tb, dout, q, k, v, scale):
    scale = torch.tensor(scale, dtype=torch.float32).item()
    out, lse = forward(tb, q, k, v, scale)
    n, hq, hk, d = q.shape[1], q.shape[2], k.shape[2], q.shape[3]
    grads = [torch.full_like(x, -7.0) for x in (q, k, v)]
    ws = torch.full((tb.tb_attention_bwd_workspace_size(1, n, hq, hk, d, q.dtype),), 0xFF, dtype=torch.uint8, device="cuda")
    tb.tb_attention_bwd(dout, q, k, v, out, lse, *grads, ws, scale=scale)
    assert tb.tb_device_error() == 0
    half, group = torch.finfo(q.dtype).eps / 2, hq // hk
    s, sums = scores(q, k, scale), lse[0].double()[..., None]
    p = torch.exp(s - sums)
    e = F32 / 2 * (s.abs() + sums.abs())
    if math.frexp(scale)[0] == 0.5:
        e = torch.where(sums.abs() > 1024, 0.0, e)
    e = torch.expm1(e.nan_to_num(0.0, 0.0, 0.0) + 4 * F32 * (1 + (s - sums).abs().nan_to_num(0.0, 0.0, 0.0)).clamp(max=400))
    qq, kk, vv, up, oo = (x[0].double() for x in (q, k, v, dout, out))
    kk, vv = kk.repeat_interleave(group, 1), vv.repeat_interleave(group, 1)
    dp, delta = torch.einsum("ihd,jhd->hij", up, vv), torch.einsum("ihd,ihd->hi", up, oo)[..., None]
    ds = p * (dp - delta)
    dp_off = (d / 16 + 16) * F32 * torch.einsum("ihd,jhd->hij", up.abs(), vv.abs()) \
        + (d / 8 + 8) * F32 * torch.einsum("ihd,ihd->hi", up.abs(), oo.abs())[..., None]
    # a power below 2^-126 is 0; fp16: below the normal numbers of what P and dS are held times
    floor_p, floor_s = 2.0 ** -126, 2.0 ** -126 * (dp - delta).abs()
    if q.dtype == HALF:
        most = up.norm(dim=-1).max().item() * vv.norm(dim=-1).max().item()
        floor_p, floor_s = 2.0 ** -39, 2 * most * 2.0 ** -37
    open_ = torch.ones(n, n, dtype=torch.bool, device="cuda").tril()
    p_off = torch.where(p > 0, p * (e + half), 0.0) + floor_p * open_
    ds_off = torch.where(p > 0, ds.abs() * (e + half + 4 * F32) + p * dp_off, 0.0) + floor_s * open_
    add = (n * group / 16 + 32) * F32
    over = lambda x: x.unflatten(1, (hk, group)).sum(2)
    for got, x, off, rows, eq, what in ((grads[0], ds * scale, ds_off * scale, kk, "hij,jhd->ihd", "dq"),
                                        (grads[1], ds * scale, ds_off * scale, qq, "hij,ihd->jhd", "dk"), (grads[2], p, p_off, up, "hij,ihd->jhd", "dv")):
        want, slack = torch.einsum(eq, x, rows), torch.einsum(eq, off + add * x.abs(), rows.abs())
        if what != "dq":
            want, slack = over(want), over(slack)
        ref.near(got[0], want, slack, what)


def slopes(q, seed=9):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(q.shape, generator=g, device="cuda") * 0.01).to(q.dtype)


@pytest.mark.parametrize("dtype, low", [(BF, 1e4), (BF, 3e8), (BF, 1e10), (BF, 1e30), (HALF, 1e4), (HALF, 3e8), (HALF, 2.0 ** 29)])
@pytest.mark.parametrize("name", DEAD)
def test_gradient_of_keys_masked_by_low_values(tb, name, dtype, low):
    q, k, v = masked(600, 2, 1, 64, dtype, low, DEAD[name])
    check_backward(tb, slopes(q), q, k, v, 0.25)


# (with other scales than powers of two the scores' own rounding leaves nothing of P beyond 2^24)
@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("dtype, power, scale", [(BF, 8, 0.3), (BF, 12, 0.25), (BF, 13, 0.3), (BF, 16, 0.088388346), (BF, 20, 0.25), (BF, 22, 0.3),
                                                 (BF, 24, 0.25), (BF, 27, 0.25), (BF, 33, 0.25), (BF, 60, 0.25), (HALF, 12, 0.3), (HALF, 16, 0.25),
                                                 (HALF, 20, 0.25), (HALF, 22, 0.3), (HALF, 26, 0.25), (HALF, 29, 0.25)])
def test_gradient_of_rows_of_scores_far_from_zero(tb, dtype, power, scale, sign):
    q, k, v = large(300, 2, 1, 64, dtype, sign * 2.0 ** power, seed=power)
    check_backward(tb, slopes(q), q, k, v, scale)


@pytest.mark.parametrize("offsets", [None, [0, 1, 130, 400]])
@pytest.mark.parametrize("dtype", [BF, HALF])
@pytest.mark.parametrize("score", [2e3, 1e4, 5e4, 2e5, 1e6, 1e7, 1e8])
def test_one_large_key(tb, score, dtype, offsets):
    """Every row's one large key is its sequence's first: P is 1 and 0, out the key's v and dv the sum of dout, at
    any scale and whatever fp32 makes of the score."""
    n, d = 400, 64
    starts = offsets or [0, n]
    q, k, v = zeros(n, 2, d, dtype), zeros(n, 1, d, dtype), values(n, 1, d, dtype, 1)
    root = 2.0 ** (math.frexp(score)[1] // 2)
    q[..., 0] = root
    k[:, starts[:-1], :, 0] = score / root / 0.3
    dout, at = slopes(q), None if offsets is None else torch.tensor(offsets, device="cuda")
    out, lse = torch.zeros_like(q), torch.zeros(1, 2, n, device="cuda")
    tb.tb_attention(q, k, v, out, lse, offsets=at, scale=0.3)
    grads = [torch.zeros_like(x) for x in (q, k, v)]
    ws = torch.empty(tb.tb_attention_bwd_workspace_size(1, n, 2, 1, d, dtype), dtype=torch.uint8, device="cuda")
    tb.tb_attention_bwd(dout, q, k, v, out, lse, *grads, ws, offsets=at, scale=0.3)
    assert tb.tb_device_error() == 0
    for a, b in zip(starts, starts[1:]):
        assert torch.equal(out[0, a:b], v[0, a].expand(b - a, 2, d))
        want, size = dout[0, a:b].double().sum((0, 1)), dout[0, a:b].double().abs().sum((0, 1))
        ref.near(grads[2][0, a, 0], want, size * (2 * (b - a) / 16 + 32) * F32, "dv")
        assert (grads[2][0, a + 1:b] == 0).all()
        # dS of a key's own v is dout . v, formed twice in fp32
        dp = torch.einsum("ihd,d->ih", dout[0, a:b].double().abs(), v[0, a, 0].double().abs()) * (d / 8 + 24) * F32
        dp = dp + (2.0 ** -24 * dp.max() if dtype == HALF else 0.0)
        ref.near(grads[0][0, a:b, :, 0], torch.zeros(b - a, 2, dtype=torch.float64, device="cuda"), 0.3 * dp * k[0, a, 0, 0].double().abs(), "dq")


@pytest.mark.parametrize("hq, hk, d", [(16, 1, 64), (12, 2, 128), (8, 8, 72)])
@pytest.mark.parametrize("dtype", [BF, HALF])
def test_gradient_of_grouped_heads(tb, dtype, hq, hk, d):
    """The same where several pieces of work share a key head, each head's scores at a distance of its own from zero."""
    n = 700
    q, k, v = large(n, hq, hk, d, torch.float32, 2.0 ** 20, seed=d)
    q *= 2.0 ** (torch.arange(hq, device="cuda") % 7 - 6)[:, None]
    q, k, v = q.to(dtype), k.to(dtype), v.to(dtype)
    check_backward(tb, slopes(q), q, k, v, 0.25)


@pytest.mark.parametrize("dtype", [BF, HALF])
def test_batch_entries_and_sequences_do_not_mix(tb, dtype):
    """Sequences of near and far scores beside each other: each has the bits that it has alone.  (Of the packed row two pieces
    of work share a key head, whose sums are joined: dk and dv are the same terms in another order, both sums off by at
    most (m / 16 + 32) 2^-23 of their m terms' magnitudes, and rounded; |dS| is at most 2 |dout| max |v|.)"""
    n, d = 300, 64
    parts = [large(n, 4, 2, d, dtype, s, seed=i) for i, s in enumerate((1.0, 2.0 ** 22, 64.0, -2.0 ** 14))]
    alone = []

    def grads(q, k, v, dout, offsets=None):
        out, lse = torch.empty_like(q), torch.empty(q.shape[0], 4, q.shape[1], device="cuda")
        tb.tb_attention(q, k, v, out, lse, offsets=offsets)
        got = [torch.empty_like(x) for x in (q, k, v)]
        ws = torch.empty(tb.tb_attention_bwd_workspace_size(q.shape[0], q.shape[1], 4, 2, d, dtype), dtype=torch.uint8, device="cuda")
        tb.tb_attention_bwd(dout, q, k, v, out, lse, *got, ws, offsets=offsets)
        return [out, *got]

    # (one row of dout and of v in each that is as large: fp16's power of two goes by all sequences)
    for i, (q, k, v) in enumerate(parts):
        dout = slopes(q, seed=i)
        dout[:, 0], v[:, 0] = 1.0, 4.0
        parts[i] = (q, k, v, dout)
        alone.append(grads(q, k, v, dout))
    batch = grads(*(torch.cat([p[j] for p in parts]) for j in range(4)))
    packed = grads(*(torch.cat([p[j] for p in parts], 1) for j in range(4)), offsets=torch.arange(0, 4 * n + 1, n, device="cuda"))
    assert tb.tb_device_error() == 0
    for j in range(4):
        for i in range(4):
            assert torch.equal(batch[j][i:i + 1], alone[i][j]), (i, j)
            mine = packed[j][:, i * n:(i + 1) * n]
            if j < 2:
                assert torch.equal(mine, alone[i][j]), (i, j)
                continue
            q, _, v, dout = (x[0].double() for x in parts[i])
            terms = dout.abs().unflatten(1, (2, 2)).sum((0, 2)) if j == 3 else \
                2 * v.norm(dim=-1).max() * d ** -0.5 * (dout.norm(dim=-1, keepdim=True) * q.abs()).unflatten(1, (2, 2)).sum((0, 2))
            slack, size = (2 * n / 16 + 32) * F32 * terms, torch.maximum(mine.double().abs(), alone[i][j].double().abs())
            bound = 2 * slack + torch.finfo(dtype).eps * (size + slack) + torch.finfo(dtype).smallest_normal * torch.finfo(dtype).eps
            assert ((mine.double() - alone[i][j].double()).abs() <= bound).all(), (i, j)
