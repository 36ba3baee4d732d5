"""Rotary positions and the per-head RMS norm in 64 bits, and how far a kernel that computes
in fp32 and rounds once may be from them.

Error terms, relative to the values they multiply (u = 2^-24, one fp32 rounding):

* a sine or cosine: 16-bit calls use the hardware's, off by at most 2^-21.19 on [-pi, pi], at
  an angle rounded twice (2 pi u); fp32 calls use one accurate to 2 ulp at an angle rounded
  once.  With the two products and the sum of the rotation: below 2^-20 of |a| + |b|.
* 1/rms: the squares of a head are added by at most 32 + 5 steps, halved by the root, then
  rsqrt (2 ulp) and the mean's rounding: below 2^-19.
* a mean of dxhat * xhat: chains of at most 32 + 5 additions and 4 products: below 2^-18 of
  the mean of the absolute terms.
* dgamma: every chain is shorter than its number of terms.
"""
import torch

SIN, RMS, MEAN, PRODUCTS = 2.0 ** -20, 2.0 ** -19, 2.0 ** -18, 2.0 ** -22
U = 2.0 ** -24
SMALLEST = {torch.float32: 2.0 ** -149, torch.bfloat16: 2.0 ** -133, torch.float16: 2.0 ** -24}


def frequencies(rot, base=10000.0, device="cuda"):
    """(radians per position in float64, the table in 2^-64 turn): exact quotients of whole
    numbers, so that both describe the same frequency."""
    turns = [int(round(base ** (-2.0 * i / rot) / 6.283185307179586 * 2.0 ** 64)) for i in range(rot // 2)]
    signed = [t - (1 << 64) if t >= 1 << 63 else t for t in turns]
    return turns, torch.tensor(signed, dtype=torch.int64, device=device)


def angles(positions, turns):
    """Angle of every (position, frequency), reduced to one turn in whole numbers."""
    pos = positions.reshape(-1).tolist()
    flat = [[((p * t) & ((1 << 64) - 1)) / 2.0 ** 64 * 6.283185307179586 for t in turns] for p in pos]
    a = torch.tensor(flat, dtype=torch.float64).reshape(*positions.shape, len(turns))
    return a.to(positions.device)


def split(x, rot, interleaved):
    r = x[..., :rot]
    return (r[..., 0::2], r[..., 1::2]) if interleaved else (r[..., :rot // 2], r[..., rot // 2:])


def join(a, b, rest, interleaved):
    r = torch.stack((a, b), -1).flatten(-2) if interleaved else torch.cat((a, b), -1)
    return torch.cat((r, rest), -1)


def rotate(x, angle, rot, interleaved, sign=1.0, magnitude=1.0):
    """x [batch, seq, heads, dim] in float64, angle [batch, seq, rot / 2]."""
    c = angle.cos()[:, :, None] * magnitude
    s = angle.sin()[:, :, None] * (magnitude * sign)
    a, b = split(x, rot, interleaved)
    return join(a * c - b * s, a * s + b * c, x[..., rot:], interleaved)


def pair_sums(x, rot, interleaved, magnitude=1.0):
    """|a| + |b| at both places of a pair; nothing behind the rotated part."""
    a, b = split(x.abs(), rot, interleaved)
    t = (a + b) * abs(magnitude)
    return join(t, t, torch.zeros_like(x[..., rot:]), interleaved)


def normed(x, gamma, eps):
    inv = (x.square().mean(-1) + eps).rsqrt()
    return x * inv[..., None] * gamma, inv


def norm_grad(dy, x, inv, gamma, angle, rot, interleaved, magnitude=1.0):
    """(dx, dgamma, bound on dx's error, bound on dgamma's) for a call whose inv_rms is exact."""
    dn = rotate(dy, angle, rot, interleaved, -1.0, magnitude)
    a = pair_sums(dy, rot, interleaved, magnitude) * SIN
    r = inv[..., None]
    xhat = x * r
    m = (dn * gamma * xhat).mean(-1, keepdim=True)
    dx = r * (dn * gamma - xhat * m)
    err_m = ((gamma * xhat).abs() * a + (dn * gamma * xhat).abs() * MEAN).mean(-1, keepdim=True)
    err = r * (gamma.abs() * a + xhat.abs() * err_m + ((dn * gamma).abs() + (xhat * m).abs()) * PRODUCTS)
    n = x.shape[0] * x.shape[1] * x.shape[2]
    dg = (dn * xhat).sum((0, 1, 2))
    dg_err = (xhat.abs() * a + (dn * xhat).abs() * (n + 64) * U).sum((0, 1, 2))
    return dx, dg, err, dg_err


def check(got, ref, err, what=""):
    """got is a rounding to its type of a value within err of ref."""
    t = got.dtype
    room = err + (ref.abs() + err) * (torch.finfo(t).eps / 2) + SMALLEST[t]
    bad = ~((got.double() - ref).abs() <= room)
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.numel()} off; worst "
                           f"{((got.double() - ref).abs() / room).max().item():.3g} of the bound")
