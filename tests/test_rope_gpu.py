"""Rotary positions and the per-head RMS norm of queries and keys against 64-bit arithmetic,
over head sizes, layouts, strides and types, on the vectorised and the general kernels."""
import pytest
import torch

import rope_reference as ref

pytestmark = pytest.mark.gpu
BF, HF, FP = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module")
def tb():
    import ln_backward_gb300
    return ln_backward_gb300


def make(shape, dtype, layout, seed, shift=0):
    """Queries, keys [batch, seq, heads, dim] as views in a layout; `shift` elements move the
    buffer off its alignment. Also the buffers, to see what lies outside the views."""
    b, s, hq, hk, d = shape
    g = torch.Generator(device="cuda").manual_seed(seed)

    def buf(n):
        return torch.randn(n + shift, generator=g, device="cuda").to(dtype)[shift:]

    if layout == "qkv":
        flat = buf(b * s * (hq + 2 * hk) * d)
        x = flat.view(b, s, hq + 2 * hk, d)
        return x[:, :, :hq], x[:, :, hq:hq + hk], [flat]
    fq, fk = buf(b * s * hq * d), buf(b * s * hk * d)
    if layout == "bhsd":
        return fq.view(b, hq, s, d).transpose(1, 2), fk.view(b, hk, s, d).transpose(1, 2), [fq, fk]
    if layout == "sbhd":
        return fq.view(s, b, hq, d).transpose(0, 1), fk.view(s, b, hk, d).transpose(0, 1), [fq, fk]
    return fq.view(b, s, hq, d), fk.view(b, s, hk, d), [fq, fk]


# (batch, seq, heads_q, heads_k, head_dim), rotary_dim: vector widths of 16, 8 and 4 bytes, two
# units a lane, idle lanes, one head, heads that do not fill a warp or share it with other tokens'
# (up to 32 of them), the general kernel
SIZES = [((2, 7, 4, 2, 128), 128), ((1, 1, 32, 8, 128), 128), ((3, 5, 5, 1, 64), 64),
         ((2, 9, 3, 3, 80), 40), ((2, 4, 6, 2, 96), 24), ((1, 33, 2, 1, 256), 64),
         ((2, 3, 2, 2, 192), 96), ((1, 6, 2, 1, 212), 106), ((1, 5, 3, 1, 33), 32),
         ((2, 3, 1, 1, 1024), 512), ((1, 4, 2, 1, 2), 2), ((1, 3, 2, 2, 1), 0), ((1, 2, 9, 9, 16), 8),
         ((1, 300, 12, 4, 64), 32), ((5, 1, 7, 7, 128), 0), ((1, 3, 40, 3, 520), 130),
         ((3, 37, 2, 1, 64), 64), ((2, 41, 3, 2, 48), 32), ((2, 19, 4, 1, 16), 16), ((1, 53, 2, 1, 66), 16)]


def _case(shape, rot, seed):
    b, s = shape[:2]
    g = torch.Generator(device="cuda").manual_seed(seed)
    turns, freqs = ref.frequencies(rot) if rot else ([], None)
    pos = torch.randint(-5, 200000, (b, s), generator=g, device="cuda")
    gam = [1 + 0.1 * torch.randn(shape[4], generator=g, device="cuda") for _ in range(2)]
    return turns, freqs, pos, ref.angles(pos, turns) if rot else pos.double()[..., None][..., :0], gam


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype", [BF, HF, FP])
@pytest.mark.parametrize("shape, rot", [(s, r) for s, r in SIZES if r])
def test_rotation_and_its_gradient(tb, shape, rot, dtype, interleaved):
    turns, freqs, pos, angle, _ = _case(shape, rot, 1)
    for k, layout in enumerate(("qkv", "bhsd", "bshd", "sbhd")):
        xq, xk, _ = make(shape, dtype, layout, 10 + k)
        yq, yk, bufs = make(shape, dtype, ("bhsd", "qkv", "sbhd", "bshd")[k], 20 + k)
        before = [f.clone() for f in bufs]
        for fn, sign in ((tb.tb_rope, 1.0), (tb.tb_rope_bwd, -1.0)):
            fn(xq, xk, yq, yk, freqs, positions=pos, interleaved=interleaved, magnitude=1.25)
            for x, y in ((xq, yq), (xk, yk)):
                x64 = x.double()
                ref.check(y, ref.rotate(x64, angle, rot, interleaved, sign, 1.25),
                          ref.pair_sums(x64, rot, interleaved, 1.25) * ref.SIN, f"{layout} {fn.__name__}")
        if k == 1:    # the values behind q and k in the joint buffer are as they were
            b, s, hq, hk, d = shape
            rest = bufs[0].view(b, s, hq + 2 * hk, d)[:, :, hq + hk:]
            assert torch.equal(rest, before[0].view(b, s, hq + 2 * hk, d)[:, :, hq + hk:])


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype", [BF, HF, FP])
@pytest.mark.parametrize("shape, rot", SIZES)
def test_norm_and_rotation(tb, shape, rot, dtype, interleaved):
    turns, freqs, pos, angle, gam = _case(shape, rot, 2)
    for k, layout in enumerate(("qkv", "bhsd")):
        xq, xk, _ = make(shape, dtype, layout, 30 + k)
        yq, yk, _ = make(shape, dtype, ("bshd", "qkv")[k], 40 + k)
        inv = [torch.full(x.shape[:3], -1.0, device="cuda") for x in (xq, xk)]
        tb.tb_qk_norm_rope(xq, xk, *gam, yq, yk, *inv, eps=1e-5, freqs=freqs, positions=pos,
                           interleaved=interleaved)
        for x, y, g, r in ((xq, yq, gam[0], inv[0]), (xk, yk, gam[1], inv[1])):
            n, want = ref.normed(x.double(), g.double(), 1e-5)
            assert ((r.double() - want).abs() <= want * (ref.RMS + ref.U)).all()
            err = (ref.pair_sums(n, rot, interleaved) + n.abs()) * (ref.SIN + ref.RMS + ref.PRODUCTS)
            ref.check(y, ref.rotate(n, angle, rot, interleaved), err, layout)
        # the serving form (nothing saved) gives the same bits
        zq, zk = torch.empty_like(yq), torch.empty_like(yk)
        tb.tb_qk_norm_rope(xq, xk, *gam, zq, zk, eps=1e-5, freqs=freqs, positions=pos,
                           interleaved=interleaved)
        ref.check(zq, yq.double(), torch.zeros_like(yq, dtype=torch.float64))
        assert torch.equal(zk.float(), yk.float())


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype", [BF, HF, FP])
@pytest.mark.parametrize("shape, rot", SIZES)
def test_norm_gradient(tb, shape, rot, dtype, interleaved):
    b, s, hq, hk, d = shape
    turns, freqs, pos, angle, gam = _case(shape, rot, 3)
    ws = torch.empty(tb.tb_qk_norm_rope_bwd_workspace_size(b, s, hq, hk, d, dtype), dtype=torch.uint8,
                     device="cuda")
    for k, layout in enumerate(("qkv", "bhsd")):
        xq, xk, _ = make(shape, dtype, layout, 50 + k)
        gq, gk, _ = make(shape, dtype, ("bhsd", "bshd")[k], 60 + k)
        dq, dk, _ = make(shape, dtype, ("qkv", "qkv")[k], 70 + k)
        inv = [ref.normed(x.double(), 1.0, 1e-5)[1].float() for x in (xq, xk)]
        dg = [torch.full((d,), 7.0, device="cuda") for _ in range(2)]
        args = (gq, gk, xq, xk, *inv, *gam, dq, dk, *dg)
        tb.tb_qk_norm_rope_bwd(*args, freqs=freqs, positions=pos, interleaved=interleaved, workspace=ws)
        for dy, x, r, g, dx, got in ((gq, xq, inv[0], gam[0], dq, dg[0]), (gk, xk, inv[1], gam[1], dk, dg[1])):
            want, want_g, err, err_g = ref.norm_grad(dy.double(), x.double(), r.double(), g.double(), angle,
                                                     rot, interleaved)
            ref.check(dx, want, err, f"{layout} dx")
            ref.check(got, want_g, err_g, f"{layout} dgamma")
        first = [t.clone() for t in (dq, dk, *dg)]
        ws.fill_(255)
        tb.tb_qk_norm_rope_bwd(*args, freqs=freqs, positions=pos, interleaved=interleaved, workspace=ws)
        for t, f in zip((dq, dk, *dg), first):
            assert torch.equal(t, f)


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("shift", [1, 2, 3, 4])
def test_any_alignment(tb, dtype, shift):
    """Buffers off the vectors' alignment take narrower vectors or the general kernel."""
    shape, rot = (2, 5, 4, 2, 128), 64
    b, s, hq, hk, d = shape
    turns, freqs, pos, angle, gam = _case(shape, rot, 4)
    xq, xk, _ = make(shape, dtype, "qkv", 1, shift)
    yq, yk, _ = make(shape, dtype, "bhsd", 2)
    tb.tb_rope(xq, xk, yq, yk, freqs, positions=pos)
    ref.check(yq, ref.rotate(xq.double(), angle, rot, False), ref.pair_sums(xq.double(), rot, False) * ref.SIN)
    gq, gk, _ = make(shape, dtype, "bshd", 3, shift)
    inv = [ref.normed(x.double(), 1.0, 1e-6)[1].float() for x in (xq, xk)]
    dg = [torch.empty(d, device="cuda") for _ in range(2)]
    ws = torch.empty(tb.tb_qk_norm_rope_bwd_workspace_size(b, s, hq, hk, d, dtype), dtype=torch.uint8, device="cuda")
    tb.tb_qk_norm_rope_bwd(gq, gk, xq, xk, *inv, *gam, yq, yk, *dg, freqs=freqs, positions=pos, workspace=ws)
    want, want_g, err, err_g = ref.norm_grad(gk.double(), xk.double(), inv[1].double(), gam[1].double(), angle, rot, False)
    ref.check(yk, want, err)
    ref.check(dg[1], want_g, err_g)


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("dim, rot", [(128, 128), (33, 18)])
def test_in_place_equals_out_of_place(tb, dtype, dim, rot):
    shape = (2, 6, 4, 2, dim)
    b, s, hq, hk, d = shape
    turns, freqs, pos, angle, gam = _case(shape, rot, 5)
    for bwd in (tb.tb_rope, tb.tb_rope_bwd):
        xq, xk, _ = make(shape, dtype, "qkv", 6)
        yq, yk, _ = make(shape, dtype, "bshd", 7)
        bwd(xq, xk, yq, yk, freqs, positions=pos)
        bwd(xq, xk, xq, xk, freqs, positions=pos)
        assert torch.equal(xq, yq) and torch.equal(xk, yk)
    xq, xk, _ = make(shape, dtype, "qkv", 8)
    tb.tb_qk_norm_rope(xq, xk, *gam, yq, yk, freqs=freqs, positions=pos)
    tb.tb_qk_norm_rope(xq, xk, *gam, xq, xk, freqs=freqs, positions=pos)
    assert torch.equal(xq, yq) and torch.equal(xk, yk)
    ws = torch.empty(tb.tb_qk_norm_rope_bwd_workspace_size(*shape, dtype), dtype=torch.uint8, device="cuda")
    for over in ("dy", "x"):
        xq, xk, _ = make(shape, dtype, "qkv", 9)
        gq, gk, _ = make(shape, dtype, "bhsd", 10)
        inv = [ref.normed(x.double(), 1.0, 1e-6)[1].float() for x in (xq, xk)]
        dg = [torch.empty(d, device="cuda") for _ in range(4)]
        kw = dict(freqs=freqs, positions=pos, workspace=ws)
        tb.tb_qk_norm_rope_bwd(gq, gk, xq, xk, *inv, *gam, yq, yk, *dg[:2], **kw)
        tb.tb_qk_norm_rope_bwd(gq, gk, xq, xk, *inv, *gam, *((gq, gk) if over == "dy" else (xq, xk)), *dg[2:], **kw)
        got = (gq, gk) if over == "dy" else (xq, xk)
        assert torch.equal(got[0], yq) and torch.equal(got[1], yk)
        assert torch.equal(dg[0], dg[2]) and torch.equal(dg[1], dg[3])


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("shape, rot, interleaved", [((2, 4001, 8, 2, 128), 128, False), ((3, 2003, 7, 3, 80), 32, True),
                                                     ((1, 9001, 1, 1, 64), 64, True)])
def test_gradient_in_place_over_many_tokens(tb, shape, rot, interleaved, dtype):
    """Warps that take several tokens ask for the next one's heads before they write the last one's."""
    b, s, hq, hk, d = shape
    turns, freqs, pos, angle, gam = _case(shape, rot, 21)
    ws = torch.empty(tb.tb_qk_norm_rope_bwd_workspace_size(*shape, dtype), dtype=torch.uint8, device="cuda")
    kw = dict(freqs=freqs, positions=pos, interleaved=interleaved, workspace=ws)
    xq, xk, _ = make(shape, dtype, "qkv", 22)
    gq, gk, _ = make(shape, dtype, "bshd", 23)
    inv = [ref.normed(x.double(), 1.0, 1e-6)[1].float() for x in (xq, xk)]
    dq, dk, _ = make(shape, dtype, "bhsd", 24)
    dg = [torch.empty(d, device="cuda") for _ in range(6)]
    tb.tb_qk_norm_rope_bwd(gq, gk, xq, xk, *inv, *gam, dq, dk, *dg[:2], **kw)
    want, want_g, err, err_g = ref.norm_grad(gq.double(), xq.double(), inv[0].double(), gam[0].double(), angle, rot, interleaved)
    ref.check(dq, want, err)
    ref.check(dg[0], want_g, err_g)
    g2, x2, = [t.clone() for t in (gq, gk)], [t.clone() for t in (xq, xk)]
    tb.tb_qk_norm_rope_bwd(*g2, xq, xk, *inv, *gam, *g2, *dg[2:4], **kw)
    tb.tb_qk_norm_rope_bwd(gq, gk, *x2, *inv, *gam, *x2, *dg[4:], **kw)
    for got in (g2, x2):
        assert torch.equal(got[0], dq) and torch.equal(got[1], dk)
    for i in (2, 4):
        assert torch.equal(dg[i], dg[0]) and torch.equal(dg[i + 1], dg[1])


def test_queries_alone_positions_and_offsets(tb):
    shape, rot = (3, 8, 4, 2, 64), 64
    turns, freqs = ref.frequencies(rot)
    xq, xk, _ = make(shape, FP, "bshd", 11)
    y, z = torch.empty_like(xq), torch.empty_like(xq)
    tb.tb_rope(xq, None, y, None, freqs, offset=5)                      # 5, 6, ...
    rows = torch.arange(8, device="cuda")
    tb.tb_rope(xq, None, z, None, freqs, positions=rows + 5)            # one row for all
    assert torch.equal(y, z)
    tb.tb_rope(xq, None, z, None, freqs, positions=(rows + 9).expand(3, 8), offset=-4)
    assert torch.equal(y, z)
    far = torch.tensor([[2**40], [-2**33 - 1], [2**31 + 7]], device="cuda")
    x1 = xq[:, :1]
    y1 = torch.empty_like(x1)
    tb.tb_rope(x1, None, y1, None, freqs, positions=far)
    ref.check(y1, ref.rotate(x1.double(), ref.angles(far, turns), rot, False),
              ref.pair_sums(x1.double(), rot, False) * ref.SIN)
    wide = torch.zeros(3, 20, dtype=torch.int64, device="cuda")          # a longer row of positions
    wide[:, 4:12] = rows + 5
    tb.tb_rope(xq, None, z, None, freqs, positions=wide[:, 4:12])
    assert torch.equal(y, z)


def test_repeated_input_and_empty_calls(tb):
    shape, rot = (2, 3, 4, 1, 64), 64
    turns, freqs, pos, angle, gam = _case(shape, rot, 12)
    one = torch.randn(1, 1, 1, 64, device="cuda", dtype=BF).expand(2, 3, 4, 64)   # strides of zero
    y = torch.empty(2, 3, 4, 64, device="cuda", dtype=BF)
    tb.tb_rope(one, None, y, None, freqs, positions=pos)
    ref.check(y, ref.rotate(one.double(), angle, rot, False), ref.pair_sums(one.double(), rot, False) * ref.SIN)
    e = torch.empty(2, 0, 4, 64, device="cuda", dtype=BF)
    tb.tb_rope(e, None, e, None, freqs)
    none = torch.empty(2, 3, 0, 64, device="cuda", dtype=BF)
    tb.tb_rope(y, none, y, none, freqs, positions=pos)                  # no key heads
    dg = [torch.full((64,), 3.0, device="cuda") for _ in range(2)]
    st = torch.empty(2, 0, 4, device="cuda")
    tb.tb_qk_norm_rope_bwd(e, e, e, e, st, st, *gam, e, e, *dg, freqs=freqs)
    assert not dg[0].any() and not dg[1].any()                          # sums over nothing
    ws = torch.empty(tb.tb_qk_norm_rope_bwd_workspace_size(2, 3, 4, 0, 64, BF), dtype=torch.uint8, device="cuda")
    dg[1].fill_(3.0)
    x = torch.randn(2, 3, 4, 64, device="cuda").to(BF)
    inv = ref.normed(x.double(), 1.0, 1e-6)[1].float()
    dx = torch.empty_like(x)
    tb.tb_qk_norm_rope_bwd(y, none, x, none, inv, inv[:, :, :0].contiguous(), *gam, dx, none, *dg, freqs=freqs,
                           positions=pos, workspace=ws)
    assert not dg[1].any() and dg[0].any()


def test_values_at_the_edge(tb):
    """A NaN or infinity stays in its head; a head of zeros gives zeros; huge values overflow
    as the fp32 formula does."""
    shape, rot = (1, 4, 4, 1, 128), 128
    turns, freqs, pos, angle, gam = _case(shape, rot, 13)
    x = torch.randn(1, 4, 4, 128, device="cuda").to(BF)
    x[0, 0, 0, 3] = float("nan")
    x[0, 1, 1, 100] = float("inf")
    x[0, 2, 2] = 0
    y, inv = torch.empty_like(x), torch.empty(1, 4, 4, device="cuda")
    tb.tb_qk_norm_rope(x, None, gam[0], None, y, None, inv, eps=1e-6, freqs=freqs, positions=pos)
    assert y[0, 0, 0].isnan().all() and not y[0, 0, 1:].isnan().any()
    assert inv[0, 1, 1] == 0 and y[0, 1, 1].isnan().sum() == 2 and not y[0, 1, 0].isnan().any()
    assert not y[0, 2, 2].any() and abs(inv[0, 2, 2].item() - 1000.0) < 0.01
    assert y[0, 3].isfinite().all()
    tb.tb_rope(x, None, y, None, freqs, positions=pos)
    assert y[0, 0, 0].isnan().sum() == 2 and y[0, 0, 1:].isfinite().all()


def test_gradient_against_differences(tb):
    """<dx, v> and <dgamma, w> against central differences of the 64-bit forward."""
    shape, rot = (2, 5, 3, 1, 64), 32
    b, s, hq, hk, d = shape
    turns, freqs, pos, angle, gam = _case(shape, rot, 14)
    for inter in (False, True):
        x, _, _ = make(shape, FP, "bshd", 15)
        dy, _, _ = make(shape, FP, "bshd", 16)
        v, _, _ = make(shape, FP, "bshd", 17)
        w = torch.randn(d, device="cuda")

        def f(xx, gg):
            return (ref.rotate(ref.normed(xx, gg, 1e-5)[0], angle, rot, inter) * dy.double()).sum()

        inv = torch.empty(b, s, hq, device="cuda")
        dx, dg, y = torch.empty_like(x), torch.empty(d, device="cuda"), torch.empty_like(x)
        ws = torch.empty(tb.tb_qk_norm_rope_bwd_workspace_size(b, s, hq, 0, d, FP), dtype=torch.uint8, device="cuda")
        tb.tb_qk_norm_rope(x, None, gam[0], None, y, None, inv, eps=1e-5, freqs=freqs, positions=pos, interleaved=inter)
        tb.tb_qk_norm_rope_bwd(dy, None, x, None, inv, None, gam[0], None, dx, None, dg, None, freqs=freqs,
                               positions=pos, interleaved=inter, workspace=ws)
        h, g64 = 1e-5, gam[0].double()
        num = (f(x.double() + h * v.double(), g64) - f(x.double() - h * v.double(), g64)) / (2 * h)
        got = (dx.double() * v.double()).sum()
        # fp32 errors of the gradient (below 2^-17 of its terms) and the difference's h^2
        scale = (dx.double() * v.double()).abs().sum()
        assert (got - num).abs() <= scale * (2.0 ** -17 + 1e-6)
        num = (f(x.double(), g64 + h * w.double()) - f(x.double(), g64 - h * w.double())) / (2 * h)
        got, scale = (dg.double() * w.double()).sum(), (dg.double() * w.double()).abs().sum()
        assert (got - num).abs() <= scale * (2.0 ** -17 + 1e-6)


def test_graph_replay_and_side_stream(tb):
    shape, rot = (2, 64, 8, 2, 128), 128
    b, s, hq, hk, d = shape
    turns, freqs, pos, angle, gam = _case(shape, rot, 18)
    xq, xk, _ = make(shape, BF, "qkv", 19)
    gq, gk, _ = make(shape, BF, "bshd", 20)

    def outputs():
        return [torch.empty(b, s, h, d, dtype=BF, device="cuda") for h in (hq, hk, hq, hk)] + \
               [torch.empty(b, s, h, device="cuda") for h in (hq, hk)] + [torch.empty(d, device="cuda") for _ in range(2)]

    def calls(o, ws):
        yq, yk, dq, dk, rq, rk, dgq, dgk = o
        kw = dict(freqs=freqs, positions=pos)
        tb.tb_qk_norm_rope(xq, xk, *gam, yq, yk, rq, rk, **kw)
        tb.tb_qk_norm_rope_bwd(gq, gk, xq, xk, rq, rk, *gam, dq, dk, dgq, dgk, workspace=ws, **kw)
        tb.tb_rope(yq, yk, yq, yk, **kw)

    size = tb.tb_qk_norm_rope_bwd_workspace_size(*shape, BF)
    ws = torch.empty(size, dtype=torch.uint8, device="cuda")
    eager, cap, side = outputs(), outputs(), outputs()
    calls(eager, ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        calls(cap, ws)
    for _ in range(3):
        graph.replay()
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    ws2 = torch.empty(size, dtype=torch.uint8, device="cuda")
    with torch.cuda.stream(st):
        calls(side, ws2)
    torch.cuda.synchronize()
    for e, c, o in zip(eager, cap, side):
        assert torch.equal(e, c) and torch.equal(e, o)
