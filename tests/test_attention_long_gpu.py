"""Attention and its gradient of long sequences: whole against the formula in 64 bits up to 16,384 tokens, and at some
rows and columns of 200,000, with the bounds of attention_reference.py."""
import math

import pytest
import torch

import attention_reference as ref
import test_attention_bwd_gpu as bwd
import test_attention_gpu as fwd

pytestmark = pytest.mark.gpu
BF, HALF = torch.bfloat16, torch.float16
F32 = ref.F32


@pytest.fixture(scope="module")
def tb():
    import ln_backward_gb300
    return ln_backward_gb300


@pytest.mark.parametrize("s, hq, hk, d, dtype, layout", [(4100, 3, 1, 128, BF, "joint"), (8191, 2, 2, 128, HALF, "bhsd"), (16384, 2, 1, 64, HALF, "bhsd"),
                                                         (9000, 2, 1, 80, BF, "bshd")])
def test_whole(tb, s, hq, hk, d, dtype, layout):
    fwd.check(tb, *fwd.inputs(1, s, hq, hk, d, dtype, layout, seed=s))
    bwd.check(tb, bwd.problem(tb, 1, s, hq, hk, d, dtype, layout, seed=s), layout=layout)


def test_packed_behind_a_long_one(tb):
    offsets = [0, 7000, 7001, 7300, 9300, 9428]
    fwd.check(tb, *fwd.inputs(1, 9500, 4, 2, 128, BF, seed=1), offsets)
    bwd.check(tb, bwd.problem(tb, 1, 9500, 4, 2, 128, BF, seed=1, offsets=offsets), offsets)


@pytest.mark.parametrize("d, dtype", [(64, BF), (128, BF), (64, HALF)])
def test_some_rows_and_columns(tb, d, dtype):
    n, scale, half = 200_000, d ** -0.5, torch.finfo(dtype).eps / 2
    given = bwd.problem(tb, 1, n, 1, 1, d, dtype, "bshd", seed=d)
    dq, dk, dv = (x[0, :, 0] for x in bwd.run(tb, *given, layout="bshd"))
    dout, q, k, v, out = (x[0, :, 0].double() for x in given[:5])
    got, sums = given[4][0, :, 0], given[5][0, 0]
    g = torch.Generator().manual_seed(d)
    at = torch.cat((torch.tensor([0, 1, 127, 128, 511, 512, n // 2, n - 129, n - 1]), torch.randint(0, n, (40,), generator=g))).cuda()
    every = torch.arange(n, device="cuda")
    delta, delta_size = (dout * out).sum(-1), (dout * out).abs().sum(-1)
    lse = sums.double()
    # fp16 holds P times 2^14 and dS times a power of two by the largest norms, and has steps of 2^-25 below its numbers
    most = dout.norm(dim=-1).max().item() * v.norm(dim=-1).max().item()
    floor_p, floor_s = (2.0 ** -39, 2 * most * 2.0 ** -37) if dtype == HALF else (0.0, 0.0)

    def pieces(rows, cols, open_):
        """P, dS and the bounds of what the kernels' may be off, of the given queries and keys."""
        s = q[rows] @ k[cols].T * scale
        e = (d / 16 + 16) * F32 * scale * (q[rows].abs() @ k[cols].T.abs()) + 8 * F32 * (1 + s.abs())
        p = torch.exp(s - lse[rows, None]).masked_fill(~open_, 0.0)
        e = e + 4 * F32 * lse[rows, None].abs() + 8 * F32 * (1 + (s - lse[rows, None]).abs())
        dp = dout[rows] @ v[cols].T - delta[rows, None]
        dp_off = (d / 16 + 16) * F32 * (dout[rows].abs() @ v[cols].T.abs()) + (d / 8 + 8) * F32 * delta_size[rows, None]
        ds = p * dp
        return s, e, p, p * (e + half) + floor_p * open_, ds, ds.abs() * (e + half + 4 * F32) + p * dp_off + floor_s * open_

    add = (n / 16 + 32) * F32
    s, _, p, _, ds, ds_off = pieces(at, slice(None), every[None] <= at[:, None])
    s.masked_fill_(every[None] > at[:, None], -math.inf)
    # (the row's exact log sum, not the kernel's)
    exact = torch.logsumexp(s, -1)
    e = (d / 16 + 16) * F32 * scale * (q[at].abs() @ k.T.abs()).amax(-1) + 8 * F32 * (1 + (q[at] @ k.T * scale).abs().amax(-1))
    ref.near(sums[at], exact, e + (n / 128 + 16) * F32 + 4 * F32 * exact.abs(), "lse")
    share = torch.softmax(s, -1)
    size = share @ v.abs()
    ref.near(got[at], share @ v, size * (2 * e[:, None] + add + half) + torch.finfo(dtype).smallest_normal * half * v.abs().sum(0), "out")
    ref.near(dq[at], ds @ k * scale, (ds_off + add * ds.abs()) @ k.abs() * scale, "dq")
    _, _, p, p_off, ds, ds_off = pieces(slice(None), at, every[:, None] >= at[None])
    ref.near(dv[at], p.T @ dout, (p_off + add * p).T @ dout.abs(), "dv")
    ref.near(dk[at], ds.T @ q * scale, (ds_off + add * ds.abs()).T @ q.abs() * scale, "dk")
