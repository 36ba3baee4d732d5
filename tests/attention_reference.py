"""Causal attention over packed sequences and its gradient in 64 bits, and how far fp32 arithmetic with 16-bit
operands of the second products may be off.

Bounds.  A 16-bit rounding is off by eps/2 of the value (eps = 2^-7 for bf16, 2^-10 for fp16).  Tensor
cores add 16 products at a time to an accumulator that truncates: a sum of n terms is off by at most
(n / 16 + 16) 2^-23 of the sum of their magnitudes.  A score's error is its exponential's relative one; the
exponent's own arithmetic adds a rounding of the score and of what is subtracted, and 2 ulp for the power.
"""
import math

import torch

F32 = 2.0 ** -23


def spans(batch, seq, offsets):
    """(batch entry, first, end) of every sequence."""
    if offsets is None:
        return [(b, 0, seq) for b in range(batch)]
    o = [int(x) for x in offsets]
    return [(0, a, b) for a, b in zip(o, o[1:])]


def _scores(q, k, scale):
    """Scores of one sequence and one key head, [group, n, n], those behind the query at -inf, and the bound of their error."""
    n, d = k.shape
    s = torch.einsum("ihd,jd->hij", q, k) * scale
    hidden = torch.ones(n, n, dtype=torch.bool, device=k.device).triu(1)
    off = (d / 16 + 16) * F32 * scale * torch.einsum("ihd,jd->hij", q.abs(), k.abs()) + 8 * F32 * (1 + s.abs())
    s.masked_fill_(hidden, -math.inf)
    off.masked_fill_(hidden, 0.0)
    return s, off


def forward(q, k, v, scale, offsets=None):
    """out, lse and the bounds of what each may be off before its rounding; NaN where no sequence has the token."""
    half = torch.finfo(q.dtype).eps / 2
    b, seq, hq, d = q.shape
    group = hq // k.shape[2]
    out = torch.full((b, seq, hq, d), math.nan, dtype=torch.float64, device=q.device)
    lse = torch.full((b, hq, seq), math.nan, dtype=torch.float64, device=q.device)
    out_off, lse_off = torch.zeros_like(out), torch.zeros_like(lse)
    for row, lo, hi in spans(b, seq, offsets):
        n = hi - lo
        for h in range(k.shape[2] if n else 0):
            mine = slice(h * group, (h + 1) * group)
            kk, vv = k[row, lo:hi, h].double(), v[row, lo:hi, h].double()
            s, off = _scores(q[row, lo:hi, mine].double(), kk, scale)
            p = torch.softmax(s, -1)
            e = off.amax(-1)                                     # [group, n]
            out[row, lo:hi, mine] = torch.einsum("hij,jd->ihd", p, vv)
            size = torch.einsum("hij,jd->ihd", p, vv.abs())
            out_off[row, lo:hi, mine] = size * ((2 * e + (n / 16 + 32) * F32).T[..., None] + half)
            # a 16-bit P below the type's normal numbers (it is at most 2^8 and the largest at least 1)
            out_off[row, lo:hi, mine] += torch.finfo(q.dtype).smallest_normal * half * vv.abs().sum(0)
            lse[row, mine, lo:hi] = torch.logsumexp(s, -1)
            lse_off[row, mine, lo:hi] = e + (n / 128 + 16) * F32 + 4 * F32 * lse[row, mine, lo:hi].abs()
    return out, lse, out_off, lse_off


def backward(dout, q, k, v, out, lse, scale, offsets=None):
    """dq, dk, dv of the formula, with out and lse as they are given, and the bounds of what each may be off before
    its rounding; NaN where no sequence has the token."""
    half = torch.finfo(q.dtype).eps / 2
    b, seq, hq, d = q.shape
    group = hq // k.shape[2]
    inside = [(row, lo, hi) for row, lo, hi in spans(b, seq, offsets) if hi > lo]
    res = [torch.full(x.shape, math.nan, dtype=torch.float64, device=q.device) for x in (q, k, v)]
    off = [torch.zeros_like(x) for x in res]
    floor_p = floor_s = 0.0
    if q.dtype == torch.float16 and inside:   # below the normal numbers of what P and dS are held times
        most = max(dout[r, a:z].double().norm(dim=-1).max().item() for r, a, z in inside) * \
            max(v[r, a:z].double().norm(dim=-1).max().item() for r, a, z in inside)
        floor_p, floor_s = 2.0 ** -14 * 2.0 ** -25, 2 * most * 2.0 ** -12 * 2.0 ** -25
    for row, lo, hi in inside:
        n = hi - lo
        for h in range(k.shape[2]):
            mine = slice(h * group, (h + 1) * group)
            qq, kk, vv = q[row, lo:hi, mine].double(), k[row, lo:hi, h].double(), v[row, lo:hi, h].double()
            up, oo = dout[row, lo:hi, mine].double(), out[row, lo:hi, mine].double()
            s, e = _scores(qq, kk, scale)
            sums = lse[row, mine, lo:hi].double()[..., None]
            p = torch.exp(s - sums)
            e = e + 4 * F32 * sums.abs() + 8 * F32 * (1 + (s - sums).abs().nan_to_num(0.0, 0.0, 0.0))
            dp = torch.einsum("ihd,jd->hij", up, vv)
            delta = torch.einsum("ihd,ihd->hi", up, oo)[..., None]
            ds = p * (dp - delta)
            dp_off = (d / 16 + 16) * F32 * torch.einsum("ihd,jd->hij", up.abs(), vv.abs()) \
                + (d / 8 + 8) * F32 * torch.einsum("ihd,ihd->hi", up.abs(), oo.abs())[..., None]
            open_ = torch.ones(n, n, dtype=torch.bool, device=q.device).tril()
            p_off = p * (e + half) + floor_p * open_
            ds_off = ds.abs() * (e + half + 4 * F32) + p * dp_off + floor_s * open_
            add = (n * group / 16 + 32) * F32
            for i, (x, x_off, rows, eq) in enumerate(((ds * scale, ds_off * scale, kk, "hij,jd->ihd"),
                                                      (ds * scale, ds_off * scale, qq, "hij,ihd->jd"),
                                                      (p, p_off, up, "hij,ihd->jd"))):
                at = (row, slice(lo, hi), mine if i == 0 else h)
                res[i][at] = torch.einsum(eq, x, rows)
                off[i][at] = torch.einsum(eq, x_off + add * x.abs(), rows.abs())
    return res, off


def near(got, want, slack, what):
    """got is want's rounding to its type, give or take `slack` before the rounding; NaN in want: not looked at."""
    live = ~want.isnan()
    got, want, slack = got[live], want[live], slack[live]
    half = torch.finfo(got.dtype).eps / 2
    off = (got.double() - want).abs()
    bad = ~(off <= half * (want.abs() + slack) + slack + torch.finfo(got.dtype).smallest_normal * half)
    assert not bad.any(), f"{what}: {bad.sum().item()} of {off.numel()} over the bound, at most by {off[bad].max().item()}"
