"""Rotary frequencies, and what the rotary entry points refuse, without a GPU: every check
below returns before any CUDA call and no pointer is dereferenced."""
import ctypes
import math

import pytest
import torch

OK, INVALID, DTYPE, MISALIGNED, ALIAS, WORKSPACE = 0, 1, 2, 3, 4, 5
F32, F16, BF16 = 0, 1, 2


@pytest.fixture(scope="module")
def tb():
    import __graft_entry__
    __graft_entry__.build()
    import ln_backward_gb300
    return ln_backward_gb300


# ----------------------------------------------------------------------------- frequencies
def radians(table):
    return [(t & ((1 << 64) - 1)) / 2.0 ** 64 * 2 * math.pi for t in table.tolist()]


def plain(rot, base, kind, factor, ctx, fast, slow):
    w = [base ** (-2.0 * i / rot) for i in range(rot // 2)]
    if kind == "linear":
        return [x / factor for x in w]
    if kind == "ntk":
        b = base * factor ** (rot / (rot - 2))
        return [b ** (-2.0 * i / rot) for i in range(rot // 2)]
    if kind == "yarn":
        def at(n):
            return rot * math.log(ctx / (n * 2 * math.pi)) / (2 * math.log(base))
        lo, hi = max(math.floor(at(fast)), 0), min(math.ceil(at(slow)), rot - 1)
        ramp = [min(max((i - lo) / (hi - lo), 0), 1) for i in range(rot // 2)]
        return [x / factor * r + x * (1 - r) for x, r in zip(w, ramp)]
    if kind == "wavelength":
        out = []
        for x in w:
            wavelength = 2 * math.pi / x
            if wavelength < ctx / fast:
                out.append(x)
            elif wavelength > ctx / slow:
                out.append(x / factor)
            else:
                t = (ctx / wavelength - slow) / (fast - slow)
                out.append((1 - t) * x / factor + t * x)
        return out
    return w


@pytest.mark.parametrize("kind, kw", [
    ("none", {}), ("linear", dict(factor=4.0)), ("ntk", dict(factor=8.0)),
    ("yarn", dict(factor=16.0, original_context=4096.0)),
    ("wavelength", dict(factor=8.0, original_context=8192.0, fast=4.0, slow=1.0))])
@pytest.mark.parametrize("rot, base", [(128, 10000.0), (64, 500000.0), (20, 10000.0)])
def test_frequencies(tb, kind, kw, rot, base):
    table, mag = tb.tb_rope_freqs(rot, base, kind, device="cpu", **kw)
    want = plain(rot, base, kind, kw.get("factor", 1.0), kw.get("original_context", 1.0),
                 kw.get("fast", 32.0), kw.get("slow", 1.0))
    assert table.dtype == torch.int64 and table.numel() == rot // 2
    for got, w in zip(radians(table), want):
        # both are computed in double: pow and a quotient, and the last part of a turn
        assert abs(got - w) <= 1e-13 * w + 2.0 ** -62
    assert mag == pytest.approx(0.1 * math.log(16) + 1 if kind == "yarn" else 1.0, rel=1e-6)


@pytest.mark.parametrize("kind", ["yarn", "wavelength"])
@pytest.mark.parametrize("ctx, divided", [(2.0, True), (3e8, False)])
def test_blends_that_no_pair_lies_in(tb, kind, ctx, divided):
    """Every pair makes fewer than `slow` turns over a context of 2, more than `fast` over 3e8."""
    rot, base, factor = 16, 100.0, 4.0
    table, _ = tb.tb_rope_freqs(rot, base, kind, factor=factor, original_context=ctx, device="cpu")
    for i, got in enumerate(radians(table)):
        w = base ** (-2.0 * i / rot) / (factor if divided else 1.0)
        assert abs(got - w) <= 1e-13 * w + 2.0 ** -62


def test_far_positions_keep_their_angle(tb):
    """pos * freq modulo 2^64 against whole-number arithmetic on the exact product."""
    table, _ = tb.tb_rope_freqs(64, device="cpu")
    for pos in (131071, 2 ** 31 + 3, -7):
        wrapped = (table * pos)                      # int64 wraps
        for t, w in zip(table.tolist(), wrapped.tolist()):
            assert (t * pos - w) % (1 << 64) == 0


def test_frequency_refusals(tb):
    f = tb._binding.lib.tb_rope_freqs
    S = tb._binding.tb_rope_scaling
    buf, mag = (ctypes.c_uint64 * 64)(), ctypes.c_float()

    def go(rot=64, base=1e4, how=None, out=buf, m=ctypes.byref(mag)):
        return f(rot, base, ctypes.byref(how) if how else None, out, m)

    assert go() == OK and go(rot=0, out=None) == OK
    assert go(rot=63) == INVALID and go(rot=-2) == INVALID and go(rot=1026) == INVALID
    assert go(base=0.0) == INVALID and go(base=float("nan")) == INVALID and go(base=float("inf")) == INVALID
    assert go(out=None) == INVALID and go(m=None) == INVALID
    assert go(how=S(5, 2.0, 0, 0, 0)) == INVALID and go(how=S(-1, 2.0, 0, 0, 0)) == INVALID
    assert go(how=S(1, 0.5, 0, 0, 0)) == INVALID                     # factor below 1
    assert go(how=S(3, 4.0, 0.0, 32, 1)) == INVALID                  # no original context
    assert go(how=S(4, 4.0, 8192.0, 1, 4)) == INVALID                # fast <= slow
    assert go(how=S(4, 4.0, 8192.0, 4, 0)) == INVALID
    assert go(base=1.0, how=S(3, 4.0, 4096.0, 32, 1)) == INVALID     # log(base) = 0
    with pytest.raises(ValueError, match="scaling"):
        tb.tb_rope_freqs(64, scaling="cubic", device="cpu")


# ----------------------------------------------------------------------------- refusals of the C entry points
class Call:
    """A valid tb_rope / tb_qk_norm_rope_bwd call at fake, disjoint addresses, to be spoilt."""

    def __init__(self, tb):
        self.tb = tb
        self.H, self.A = tb._binding.tb_heads, tb._binding.tb_rope_angles
        self.batch, self.seq, self.dim, self.dtype = 2, 8, 64, BF16
        self.t = {n: self.H((i + 1) << 24, 8 * 4 * 64, 4 * 64, 64, 4)
                  for i, n in enumerate(("q", "k", "qo", "ko", "dqo", "dko"))}
        self.ang = self.A(0x9000000, 0xA000000, 8, 0, 64, 0, 1.0)
        self.gamma = [0xB000000, 0xB100000]
        self.inv = [0xC000000, 0xC100000]
        self.dg = [0xD000000, 0xD100000]
        self.eps, self.ws, self.ws_bytes = 1e-6, 0xE000000, 0

    def ref(self, n):
        t = self.t[n]
        return ctypes.byref(t) if t is not None else None

    def rope(self, fn="tb_rope"):
        return getattr(self.tb._binding.lib, fn)(
            self.ref("q"), self.ref("k"), self.ref("qo"), self.ref("ko"), self.batch, self.seq,
            self.dim, ctypes.byref(self.ang) if self.ang else None, self.dtype, None)

    def norm(self):
        return self.tb._binding.lib.tb_qk_norm_rope(
            self.ref("q"), self.ref("k"), *self.gamma, self.eps, self.ref("qo"), self.ref("ko"),
            *self.inv, self.batch, self.seq, self.dim, ctypes.byref(self.ang), self.dtype, None)

    def bwd(self):
        return self.tb._binding.lib.tb_qk_norm_rope_bwd(
            self.ref("dqo"), self.ref("dko"), self.ref("q"), self.ref("k"), *self.inv, *self.gamma,
            self.ref("qo"), self.ref("ko"), *self.dg, self.batch, self.seq, self.dim,
            ctypes.byref(self.ang), self.dtype, self.ws, self.ws_bytes, None)


def spoilt(tb, **how):
    c = Call(tb)
    for k, v in how.items():
        if "__" in k:
            t, f = k.split("__")
            setattr(c.ang if t == "ang" else c.t[t], f, v)
        elif k in c.t:
            c.t[k] = v
        else:
            setattr(c, k, v)
    return c


def test_empty_calls_need_no_gpu(tb):
    for fn in ("tb_rope", "tb_rope_bwd"):
        assert spoilt(tb, batch=0).rope(fn) == OK and spoilt(tb, seq=0).rope(fn) == OK
    assert spoilt(tb, seq=0).norm() == OK
    c = spoilt(tb, q__heads=0, qo__heads=0, k__heads=0, ko__heads=0)
    assert c.rope() == OK


@pytest.mark.parametrize("how, want", [
    (dict(batch=-1), INVALID), (dict(seq=-1), INVALID), (dict(dim=0), INVALID), (dict(dim=1025), INVALID),
    (dict(dtype=7), DTYPE), (dict(ang=None), INVALID), (dict(q=None), INVALID), (dict(qo=None), INVALID),
    (dict(k=None), INVALID), (dict(ko=None), INVALID), (dict(qo__heads=3), INVALID),
    (dict(q__heads=-1, qo__heads=-1), INVALID), (dict(q__stride_seq=-64), INVALID),
    (dict(q__heads=(1 << 20) + 1, qo__heads=(1 << 20) + 1), INVALID),
    (dict(q__data=None), INVALID), (dict(qo__data=None), INVALID), (dict(q__data=0x1000001), MISALIGNED),
    (dict(q__data=0x1000002, dtype=F32), MISALIGNED), (dict(q__stride_batch=1 << 61), INVALID),
    (dict(ang__rotary_dim=63), INVALID), (dict(ang__rotary_dim=66), INVALID), (dict(ang__rotary_dim=-2), INVALID),
    (dict(ang__layout=2), INVALID), (dict(ang__magnitude=float("nan")), INVALID),
    (dict(ang__freqs=None), INVALID), (dict(ang__freqs=0x9000004), MISALIGNED),
    (dict(ang__positions=0xA000004), MISALIGNED), (dict(ang__positions_stride=7), INVALID),
    (dict(ang__positions_stride=-8), INVALID),
    (dict(qo__data=(1 << 24) + 128), ALIAS),          # not the same rows, but their elements
    (dict(qo__data=2 << 24), ALIAS),                  # q_out over k
    (dict(ko__data=3 << 24), ALIAS),                  # both outputs in one place
    (dict(qo__stride_seq=128), ALIAS),                # an output whose rows overlap
    (dict(qo__stride_batch=0), ALIAS),
    (dict(qo__data=1 << 24, qo__stride_head=128, qo__stride_seq=512, qo__stride_batch=4096), ALIAS),
    (dict(qo__data=0x9000000 - 64), ALIAS),           # over the frequencies
    (dict(qo__data=0xA000000), ALIAS),                # over the positions
])
def test_rope_refusals(tb, how, want):
    assert spoilt(tb, **how).rope() == want
    assert spoilt(tb, **how).rope("tb_rope_bwd") == want
    if "ang" not in how:
        assert spoilt(tb, **how).norm() == want


def test_positions_too_far_apart_are_refused(tb):
    """Strides whose product with the batch leaves 64 bits, which a sum of them would wrap around."""
    for stride in (1 << 60, (1 << 63) - 1):
        assert spoilt(tb, ang__positions_stride=stride).rope() == INVALID
        assert spoilt(tb, ang__positions_stride=stride, batch=3).norm() == INVALID
    # without entries the stride is never used
    assert spoilt(tb, ang__positions_stride=1 << 60, batch=1, seq=0).rope() == OK


def test_slices_of_one_buffer_are_told_apart(tb):
    """Outputs among the heads of the buffer that holds the inputs: refused where an element is
    shared, although no row is the same.  (That disjoint slices pass is tested on the GPU,
    where the call goes on to run.)"""
    base, row = 1 << 24, 12 * 64                       # 4 query, 4 key, 4 value heads
    ok = dict(stride_batch=8 * row, stride_seq=row, stride_head=64)

    def heads(c, data, n=4):
        return c.H(data, ok["stride_batch"], ok["stride_seq"], ok["stride_head"], n)

    c = Call(tb)
    c.dtype = BF16
    c.t["q"], c.t["k"] = heads(c, base), heads(c, base + 2 * 256)
    # q_out one head into the keys
    c.t["qo"], c.t["ko"] = heads(c, base + 2 * 64), heads(c, base + 2 * 512)
    assert c.rope() == ALIAS
    # q_out over the last value head of the previous token and the first query head
    c.t["qo"] = heads(c, base + 2 * (row - 64))
    assert c.rope() == ALIAS


@pytest.mark.parametrize("how, want", [
    (dict(eps=-1.0), INVALID), (dict(eps=float("nan")), INVALID), (dict(gamma=[None, 0xB100000]), INVALID),
    (dict(gamma=[0xB000000, None]), INVALID), (dict(gamma=[0xB000002, 0xB100000]), MISALIGNED),
    (dict(inv=[0xC000002, 0xC100000]), MISALIGNED), (dict(inv=[0xC000000, 0xC000000]), ALIAS),
    (dict(inv=[0xB000000, 0xC100000]), ALIAS), (dict(inv=[3 << 24, 0xC100000]), ALIAS),
    (dict(inv=[(1 << 24) + 4, 0xC100000]), ALIAS)])
def test_norm_refusals(tb, how, want):
    assert spoilt(tb, **how).norm() == want


@pytest.mark.parametrize("how, want", [
    (dict(dqo=None), INVALID), (dict(dko=None), INVALID), (dict(dqo__heads=2), INVALID),
    (dict(inv=[None, 0xC100000]), INVALID), (dict(inv=[0xC000000, None]), INVALID),
    (dict(dg=[None, 0xD100000]), INVALID), (dict(dg=[0xD000001, 0xD100000]), MISALIGNED),
    (dict(gamma=[None, 0xB100000]), INVALID)])
def test_norm_gradient_refusals(tb, how, want):
    assert spoilt(tb, **how).bwd() == want


def test_workspace_query_refusals(tb):
    f, n = tb._binding.lib.tb_qk_norm_rope_bwd_workspace_size, ctypes.c_size_t(9)
    assert f(2, 8, 4, 4, 64, BF16, None) == INVALID
    assert f(-1, 8, 4, 4, 64, BF16, ctypes.byref(n)) == INVALID
    assert f(2, 8, 4, 4, 2000, BF16, ctypes.byref(n)) == INVALID
    assert f(2, 8, 4, 4, 64, 9, ctypes.byref(n)) == DTYPE
    assert f(0, 8, 4, 4, 64, BF16, ctypes.byref(n)) == OK and n.value == 0


# ----------------------------------------------------------------------------- the binding
def test_binding_refusals(tb):
    q, k = torch.zeros(2, 3, 4, 64), torch.zeros(2, 3, 2, 64)
    fr = torch.zeros(32, dtype=torch.int64)
    with pytest.raises(ValueError, match="q must be"):
        tb.tb_rope(q[0], k, q, k, fr)
    with pytest.raises(ValueError, match="together"):
        tb.tb_rope(q, None, q, k, fr)
    with pytest.raises(ValueError, match="k must be"):
        tb.tb_rope(q, k[:, :2], q, k, fr)
    with pytest.raises(ValueError, match="k must be torch.float32"):
        tb.tb_rope(q, k.half(), q, k, fr)
    with pytest.raises(ValueError, match="contiguous"):
        tb.tb_rope(torch.zeros(2, 3, 4, 128)[..., ::2], k, q, k, fr)
    with pytest.raises(ValueError, match="CUDA"):
        tb.tb_rope(q, k, q, k, fr)
    with pytest.raises(ValueError, match="CUDA"):
        tb.tb_qk_norm_rope(q, k, torch.ones(64), torch.ones(64), q, k)


# pi to 60 places (public constant), for angles formed apart from the library's binary fractions
PI = "3.14159265358979323846264338327950288419716939937510582097494"


@pytest.mark.parametrize("rot, base", [(64, 10000), (128, 500000), (6, 100)])
def test_far_positions_against_long_decimals(tb, rot, base):
    """The angle of a far position, as the kernels form it from the table, against one formed in 60
    decimal places from base^(-2i/rot) itself."""
    from decimal import Decimal, localcontext
    with localcontext() as ctx:
        ctx.prec = 60
        table, _ = tb.tb_rope_freqs(rot, float(base), device="cpu")
        for pos in (1, 131071, 2 ** 31 + 3, -131071, 2 ** 40 + 1):
            for i, entry in enumerate(table.tolist()):
                phase = (pos * entry) & ((1 << 64) - 1)              # what 64-bit arithmetic leaves
                got = Decimal(phase) / Decimal(1 << 64)              # of a turn
                w = Decimal(base) ** (Decimal(-2 * i) / rot) / (2 * Decimal(PI))
                want = w * pos % 1
                off = abs(got - want) % 1
                off = min(off, 1 - off)
                # the table: pow and a product or two in double, then half of 2^-64 a position
                assert off <= abs(pos) * (w * 4 * Decimal(2) ** -53 + Decimal(2) ** -65)
