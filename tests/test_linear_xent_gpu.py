"""Softmax cross entropy of a linear output layer, and its gradients, against 64 bits.

Bounds, with u = 2^-24 and the products of 16-bit values exact in fp32:

* a logit: D additions, each off by at most one unit (tensor cores may truncate, 2u):
  2u (D + 8) sum |h w|;
* log sum exp: the largest logit error, exp2 (2 ulp), its argument (|l - top| log2(e) u) and
  the additions of a row (at most V / 8 + 512 in a chain), and the final sum;
* G = p - onehot: p off by its argument's error, rounded once to the type (half its eps), or
  by half of fp16's last step (2^-24, under a scale of 2^14) where it is that small;
* for dW, H times dloss / max |dloss|: another rounding to the type;
* dH, dW: those errors through the product, and its own V (or rows) additions;

and one rounding of every 16-bit result.
"""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu
BF, HF = torch.bfloat16, torch.float16
U = 2.0 ** -24


@pytest.fixture(scope="module")
def tb():
    import ln_backward_gb300
    return ln_backward_gb300


def problem(n, d, v, dtype, seed=0, scale=0.5, ignored=0.2):
    g = torch.Generator(device="cuda").manual_seed(1000 * seed + n + d + v)
    H = torch.randn(n, d, generator=g, device="cuda").to(dtype)
    W = (torch.randn(v, d, generator=g, device="cuda") * (scale * d ** -0.5 * 4)).to(dtype)
    t = torch.randint(0, v, (n,), generator=g, device="cuda")
    t[0], t[-1] = v - 1, 0                                  # the borders of the vocabulary
    skip = torch.rand(n, generator=g, device="cuda") < ignored
    skip[0] = False
    t[skip] = -100
    dloss = torch.rand(n, generator=g, device="cuda") / n + 0.5 / n
    return H, W, t, dloss


def workspace(size):
    return torch.full((max(size, 16),), 255, dtype=torch.uint8, device="cuda")   # NaNs


def forward(tb, H, W, t, **kw):
    n, d, v = *H.shape, W.shape[0]
    loss, lse = torch.full((2, n), -7.0, device="cuda")
    tb.tb_linear_xent(H, W, t, loss, lse, workspace(tb.tb_linear_xent_workspace_size(n, d, v, H.dtype)), **kw)
    return loss, lse


def backward(tb, dloss, H, W, t, lse, want="HW", **kw):
    n, d, v = *H.shape, W.shape[0]
    dH = torch.full_like(H, 3.0) if "H" in want else None
    dW = torch.full_like(W, 3.0) if "W" in want else None
    tb.tb_linear_xent_bwd(dloss, H, W, t, lse, dH, dW,
                          workspace(tb.tb_linear_xent_bwd_workspace_size(n, d, v, H.dtype)), **kw)
    return dH, dW


def logits64(H, W):
    l = H.double() @ W.double().T
    err = (H.double().abs() @ W.double().abs().T).max() * (2 * U * (H.shape[1] + 8))
    return l, err


def check_forward(loss, lse, H, W, t, ignore=-100):
    l, err_l = logits64(H, W)
    want = torch.logsumexp(l, -1)
    span = (l.max() - l.min()).item()
    err = err_l + U * (8 + 2 * span + W.shape[0] / 8 + 512 + 4 * want.abs())
    assert ((lse.double() - want).abs() <= err).all(), ((lse.double() - want).abs() / err).max()
    keep = t != ignore
    row = torch.where(keep, want - l.gather(1, torch.where(keep, t, 0)[:, None])[:, 0], 0.0)
    assert ((loss.double() - row).abs() <= (err + err_l + U * row.abs()) * keep).all()


def check_backward(dH, dW, dloss, H, W, t, lse, ignore=-100):
    l, err_l = logits64(H, W)
    n, v = l.shape
    keep = t != ignore
    weight = torch.where(keep, dloss.double(), 0.0)
    p = (l - lse.double()[:, None]).exp()
    p_err = p * (err_l + U * (4 + 2 * (l - lse.double()[:, None]).abs() + 2 * lse.double().abs()[:, None]))
    p[torch.arange(n, device="cuda"), torch.where(keep, t, 0)] -= 1.0
    G, p_err = p * weight[:, None], p_err * weight.abs()[:, None]
    half = torch.finfo(H.dtype).eps / 2
    tiny = 2.0 ** -25 if H.dtype == HF else 0.0
    G_err = p_err + G.abs() * (half + 4 * U) + tiny * 2.0 ** -14 * weight.abs()[:, None]
    # a scaled H below fp16's normal numbers is off by half a step of the largest |dloss|
    W_err = G_err + G.abs() * (half + 2 * U)
    H_tiny = tiny * weight.abs().max()

    def check(got, A, A_err, B, terms, what, more=0.0):
        want = A @ B
        err = more + A_err @ B.abs() + (A.abs() @ B.abs()) * (2 * U * (terms + 16))
        room = err + (want.abs() + err) * half + (2.0 ** -25 if H.dtype == HF else 0.0)
        off = (got.double() - want).abs()
        assert (off <= room).all(), f"{what}: {(off / room).max().item():.3g} of the bound"

    if dH is not None:
        check(dH, G, G_err, W.double(), v, "dH")
    if dW is not None:
        check(dW, G.T, W_err.T, torch.where(keep[:, None], H.double(), 0.0), n, "dW",
              (p.abs().T @ keep.double()[:, None]) * H_tiny)


# one row, one column, one element; ragged in every direction; one element over a tile; row
# lengths that TMA cannot read as they are; contractions split over the vocabulary
SIZES = [(1, 8, 1), (1, 64, 10), (3, 1, 7), (5, 64, 257), (37, 72, 300), (256, 64, 256), (256, 128, 512),
         (257, 40, 1000), (300, 200, 2049), (130, 33, 515), (2, 13, 3), (64, 768, 5003), (700, 264, 700),
         (513, 520, 777), (37, 768, 50257)]


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("n, d, v", SIZES)
def test_loss(tb, n, d, v, dtype):
    H, W, t, _ = problem(n, d, v, dtype)
    check_forward(*forward(tb, H, W, t), H, W, t)


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("n, d, v", SIZES)
def test_gradients(tb, n, d, v, dtype):
    H, W, t, dloss = problem(n, d, v, dtype, 1)
    if dtype == HF:
        dloss = dloss * 1024                     # a loss scale
    lse = torch.logsumexp(H.double() @ W.double().T, -1).float()
    dH, dW = backward(tb, dloss, H, W, t, lse)
    check_backward(dH, dW, dloss, H, W, t, lse)
    assert not dH[t == -100].any()
    only_h, _ = backward(tb, dloss, H, W, t, lse, "H")
    _, only_w = backward(tb, dloss, H, W, t, lse, "W")
    assert torch.equal(only_h, dH) and torch.equal(only_w, dW)      # and every run is the same


# several pieces of the vocabulary (of 256 MiB of G), launches of the loss, and with 7,000 columns
# pieces whose dH is split as well; row lengths whose fp32 sums TMA can and cannot write
@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("n, d, v", [(40000, 24, 5000), (20000, 32, 7000), (20000, 33, 7000), (36000, 400, 4001)])
def test_pieces_of_the_vocabulary(tb, n, d, v, dtype):
    H, W, t, dloss = problem(n, d, v, dtype, 2)
    loss, lse = forward(tb, H, W, t)
    check_forward(loss, lse, H, W, t)
    if dtype == HF:
        dloss = dloss * 4096
    dH, dW = backward(tb, dloss, H, W, t, lse)
    check_backward(dH, dW, dloss, H, W, t, lse)
    again = backward(tb, dloss, H, W, t, lse)
    assert torch.equal(again[0], dH) and torch.equal(again[1], dW)


@pytest.mark.parametrize("dtype", [BF, HF])
def test_masks(tb, dtype):
    """No row counts; one row counts; ignore_index is a class; a dloss of zero."""
    n, d, v = 70, 72, 300
    H, W, t, dloss = problem(n, d, v, dtype, 3, ignored=0.0)
    none = torch.full_like(t, -100)
    loss, lse = forward(tb, H, W, none)
    check_forward(loss, lse, H, W, none)
    assert not loss.any()
    dH, dW = backward(tb, dloss, H, W, none, lse)
    assert not dH.any() and not dW.any()
    one = none.clone()
    one[17] = t[17]
    dH, dW = backward(tb, dloss, H, W, one, lse)
    check_backward(dH, dW, dloss, H, W, one, lse)
    t[5:9] = 7
    loss, lse = forward(tb, H, W, t, ignore_index=7)
    check_forward(loss, lse, H, W, t, ignore=7)
    dH, dW = backward(tb, dloss, H, W, t, lse, ignore_index=7)
    check_backward(dH, dW, dloss, H, W, t, lse, ignore=7)
    dloss[20:40] = 0
    dH, dW = backward(tb, dloss, H, W, t, lse, ignore_index=7)
    check_backward(dH, dW, dloss, H, W, t, lse, ignore=7)
    dloss.zero_()
    dH, dW = backward(tb, dloss, H, W, t, lse, ignore_index=7)
    assert not dH.any() and not dW.any()


@pytest.mark.parametrize("dtype", [BF, HF])
def test_what_an_ignored_row_holds_does_not_matter(tb, dtype):
    n, d, v = 300, 136, 900
    H, W, t, dloss = problem(n, d, v, dtype, 4)
    loss, lse = forward(tb, H, W, t)
    dH, dW = backward(tb, dloss, H, W, t, lse)
    skip = t == -100
    assert skip.any()
    H2, dloss2, lse2 = H.clone(), dloss.clone(), lse.clone()
    H2[skip] = float("nan")
    dloss2[skip] = float("inf")
    lse2[skip] = float("nan")
    loss2, l2 = forward(tb, H2, W, t)
    assert torch.equal(loss2, loss) and torch.equal(l2[~skip], lse[~skip])
    dH2, dW2 = backward(tb, dloss2, H2, W, t, lse2)
    assert torch.equal(dH2, dH) and torch.equal(dW2, dW)


@pytest.mark.parametrize("n, d, v", [(300, 136, 900), (40000, 24, 5000)])
@pytest.mark.parametrize("dtype", [BF, HF])
def test_what_a_row_of_weight_zero_holds_does_not_matter(tb, n, d, v, dtype):
    """Padding that has targets and a dloss of 0, in one piece of the vocabulary and in several."""
    H, W, t, dloss = problem(n, d, v, dtype, 12, ignored=0.0)
    pad = torch.arange(n, device="cuda") % 7 == 3
    dloss[pad] = 0.0
    dloss[3] = -0.0
    _, lse = forward(tb, H, W, t)
    dH, dW = backward(tb, dloss, H, W, t, lse)
    assert not dH[pad].any() and dW.isfinite().all()
    for value in (float("nan"), float("inf")):
        H2 = H.clone()
        H2[pad] = value
        _, lse2 = forward(tb, H2, W, t)
        dH2, dW2 = backward(tb, dloss, H2, W, t, lse2)
        assert torch.equal(dH2, dH) and torch.equal(dW2, dW)


def test_a_target_outside_the_vocabulary(tb):
    n, d, v = 40, 64, 200
    H, W, t, dloss = problem(n, d, v, BF, 5, ignored=0.0)
    loss, lse = forward(tb, H, W, t)
    assert tb.tb_device_error() == 0
    bad = t.clone()
    bad[3], bad[4], bad[5] = v, -1, 2 ** 40
    loss2, lse2 = forward(tb, H, W, bad)
    assert tb.tb_device_error() == 1 and tb.tb_device_error() == 0       # read and reset
    assert loss2[3:6].isnan().all() and torch.equal(lse2, lse)
    keep = torch.ones(n, dtype=torch.bool, device="cuda")
    keep[3:6] = False
    assert torch.equal(loss2[keep], loss[keep])
    dH, dW = backward(tb, dloss, H, W, bad, lse)
    skipped = torch.where(keep, t, -100)
    check_backward(dH, dW, dloss, H, W, skipped, lse)


@pytest.mark.parametrize("dtype", [BF, HF])
def test_infinities_and_large_logits(tb, dtype):
    n, d, v = 33, 64, 700
    H, W, t, dloss = problem(n, d, v, dtype, 6, ignored=0.0)
    H = H * 20                                            # logits of hundreds: differences decide
    loss, lse = forward(tb, H, W, t)
    check_forward(loss, lse, H, W, t)
    dH, dW = backward(tb, dloss, H, W, t, lse)
    check_backward(dH, dW, dloss, H, W, t, lse)
    H = H / 20
    H[1, 0], W[:, 0] = float("inf"), W[:, 0].abs() + 0.01   # a row of +inf logits
    H[2, 0] = -float("inf")                                 # a row of -inf
    H[3, 0] = float("nan")
    loss, lse = forward(tb, H, W, t)
    assert lse[1] == float("inf") and lse[2] == -float("inf") and lse[3].isnan()
    assert loss[1:4].isnan().all() and loss[4:].isfinite().all() and loss[0].isfinite()


@pytest.mark.parametrize("off", [1, 2, 4])
@pytest.mark.parametrize("d", [64, 24])
def test_results_off_their_alignment(tb, d, off):
    """dH and dW where TMA cannot write them; what lies around them stays."""
    n, v = 150, 600
    H, W, t, dloss = problem(n, d, v, BF, 7)
    _, lse = forward(tb, H, W, t)
    want = backward(tb, dloss, H, W, t, lse)
    bufs = [torch.full((k * d + 2 * off + 8,), 5.0, dtype=BF, device="cuda") for k in (n, v)]
    got = [b[off:off + k * d].view(k, d) for b, k in zip(bufs, (n, v))]
    ws = workspace(tb.tb_linear_xent_bwd_workspace_size(n, d, v, BF))
    tb.tb_linear_xent_bwd(dloss, H, W, t, lse, *got, ws)
    for b, g, w, k in zip(bufs, got, want, (n, v)):
        assert torch.equal(g, w)
        assert (b[:off] == 5).all() and (b[off + k * d:] == 5).all()


def test_no_rows(tb):
    W = torch.randn(50, 64, device="cuda").to(BF)
    H = torch.empty(0, 64, dtype=BF, device="cuda")
    t, e = torch.empty(0, dtype=torch.int64, device="cuda"), torch.empty(0, device="cuda")
    tb.tb_linear_xent(H, W, t, e, e.clone(), None)
    dW = torch.ones_like(W)
    tb.tb_linear_xent_bwd(e, H, W, t, e, H.clone(), dW, None)
    assert not dW.any()


# many rows against a small vocabulary: dW has few tiles and is split over the rows; sums that TMA can
# and cannot write, results off their alignment
@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("n, d, v, off", [(5000, 40, 600, 0), (4099, 52, 701, 0), (6000, 7, 3, 0), (3001, 264, 1, 0),
                                          (5000, 64, 300, 1), (5000, 64, 300, 2), (5000, 64, 300, 4)])
def test_contractions_over_many_rows(tb, n, d, v, off, dtype):
    H, W, t, dloss = problem(n, d, v, dtype, 13)
    if dtype == HF:
        dloss = dloss * 1024
    _, lse = forward(tb, H, W, t)
    buf = torch.full((v * d + 2 * off + 8,), 5.0, dtype=dtype, device="cuda")
    dW, dH = buf[off:off + v * d].view(v, d), torch.empty_like(H)
    ws = workspace(tb.tb_linear_xent_bwd_workspace_size(n, d, v, dtype))
    tb.tb_linear_xent_bwd(dloss, H, W, t, lse, dH, dW, ws)
    check_backward(dH, dW, dloss, H, W, t, lse)
    assert (buf[:off] == 5).all() and (buf[off + v * d:] == 5).all()
    again = torch.empty_like(W)
    tb.tb_linear_xent_bwd(dloss, H, W, t, lse, None, again, ws)
    assert torch.equal(again, dW)


def test_gradient_against_differences(tb):
    """<dH, a> and <dW, b> against central differences of the 64-bit loss."""
    n, d, v = 60, 96, 500
    H, W, t, dloss = problem(n, d, v, BF, 8)
    _, lse = forward(tb, H, W, t)
    dH, dW = backward(tb, dloss, H, W, t, lse)
    keep = t != -100
    col = torch.where(keep, t, 0)[:, None]

    def f(h, w):
        l = h @ w.T
        return ((torch.logsumexp(l, -1) - l.gather(1, col)[:, 0]) * keep * dloss.double()).sum()

    a, b = torch.randn(n, d, device="cuda").double(), torch.randn(v, d, device="cuda").double()
    H64, W64, h = H.double(), W.double(), 1e-5
    for grad, x, num in ((dH, a, f(H64 + h * a, W64) - f(H64 - h * a, W64)),
                         (dW, b, f(H64, W64 + h * b) - f(H64, W64 - h * b))):
        got, scale = (grad.double() * x).sum(), (grad.double() * x).abs().sum()
        # three roundings to bf16 (G, H's copy, the result) of every term, and h^2
        assert (got - num / (2 * h)).abs() <= scale * (3 * 2.0 ** -8 + 1e-6)


def test_graph_replay_streams_and_two_calls_at_once(tb):
    n, d, v = 300, 256, 3000
    H, W, t, dloss = problem(n, d, v, BF, 9)
    size = max(tb.tb_linear_xent_workspace_size(n, d, v, BF), tb.tb_linear_xent_bwd_workspace_size(n, d, v, BF))

    def outputs():
        return [torch.empty(n, device="cuda"), torch.empty(n, device="cuda"), torch.empty_like(H), torch.empty_like(W)]

    def calls(o, ws):
        tb.tb_linear_xent(H, W, t, o[0], o[1], ws)
        tb.tb_linear_xent_bwd(dloss, H, W, t, o[1], o[2], o[3], ws)

    eager, cap, side, side2 = outputs(), outputs(), outputs(), outputs()
    ws = [workspace(size) for _ in range(4)]
    calls(eager, ws[0])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        calls(cap, ws[1])
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(3):
        for st, o, w in zip(streams, (side, side2), ws[2:]):
            with torch.cuda.stream(st):
                calls(o, w)
    torch.cuda.synchronize()
    for o in (cap, side, side2):
        for x, y in zip(o, eager):
            assert torch.equal(x, y)
    assert tb.tb_device_error() == 0


def masked_problem(dtype, value, columns, n=70, d=72, v=700, seed=14):
    """Columns of the vocabulary masked by an additive term: the hidden states' first element is a
    constant, and `value` over it the masked columns' first weight."""
    H, W, t, dloss = problem(n, d, v, dtype, seed, ignored=0.0)
    H[:, 0] = 1.0 if dtype == BF else 16384.0
    W[:, 0] = 0.0
    W[columns, 0] = value / H[0, 0].item()
    t = torch.arange(n, device="cuda") % 64 + 640                       # 640 .. 699: never masked below
    t[t >= v] = v - 1
    return H, W, t, dloss


@pytest.mark.parametrize("dtype, values", [(BF, (-1e10, 2.0 ** 33 * -1.7, -1e30, -3.3e38)),
                                           (HF, (-2.0 ** 29, -1.7 * 2.0 ** 28, -1e9))])
@pytest.mark.parametrize("columns", [slice(0, 640), slice(32, 64), slice(3, 500)])
@pytest.mark.parametrize("d", [72, 600, 1304])                     # 16 and 8 epilogue warps, several chunks
def test_masks_of_low_values(tb, d, dtype, values, columns):
    """A masked column counts exp(-large) = 0 whatever the large value is: the same bits as with a
    mask of -10,000, in 32-column groups that hold nothing else as well."""
    H, W, t, dloss = masked_problem(dtype, -1e4, columns, d=d)
    loss, lse = forward(tb, H, W, t)
    keep = torch.ones(W.shape[0], dtype=torch.bool, device="cuda")
    keep[columns] = False
    check_forward(loss, lse, H, W[keep].contiguous(), t - int((~keep).sum()))
    dH, dW = backward(tb, dloss, H, W, t, lse)
    assert not dW[columns].any()
    for value in values:
        H, W, t, dloss = masked_problem(dtype, value, columns, d=d)
        got = forward(tb, H, W, t)
        assert torch.equal(got[0], loss) and torch.equal(got[1], lse), value
        dH2, dW2 = backward(tb, dloss, H, W, t, lse)
        assert torch.equal(dH2, dH) and torch.equal(dW2, dW), value


@pytest.mark.parametrize("dtype, values", [(BF, (-1e10, 2.0 ** 33 * 1.7, 1e30, -3.3e38, 3.3e38)),
                                           (HF, (-2.0 ** 29, 1.7 * 2.0 ** 28, 1e9))])
def test_rows_whose_logits_are_all_far_from_zero(tb, dtype, values):
    """lse is its largest logit to fp32's last places, and G = exp(l - lse) is what it says for
    that lse: at most 1, and 0 in columns that lie far below."""
    n, v = 70, 700
    for value in values:
        H, W, t, dloss = masked_problem(dtype, value, slice(0, v))
        l = (H[0, 0].double() * W[0, 0].double()).item()
        loss, lse = forward(tb, H, W, t)
        # the other terms of a logit and log(700) are below one of fp32's places, of which
        # truncated additions lose one each
        assert ((lse.double() - l).abs() <= abs(l) * 2.0 ** -20).all(), value
        assert (loss.abs() <= abs(l) * 2.0 ** -20).all(), value
        # one column above all others: p = 1 there, and where it is the target nothing is left
        H, W, t, dloss = masked_problem(dtype, abs(value), slice(0, 1))
        t[:35] = 0
        loss, lse = forward(tb, H, W, t)
        top = (H.double() @ W[0].double())
        assert ((lse.double() - top).abs() <= top.abs() * 2.0 ** -20).all(), value
        # what the logits of a second call are, the first's were: l - lse = 0 where l is the maximum
        dH, dW = backward(tb, dloss, H, W, t, lse)
        assert not dH[:35].any()
        G = torch.zeros(n, v, device="cuda", dtype=torch.float64)
        G[35:, 0] = 1.0
        G[torch.arange(35, n), t[35:]] -= 1.0
        want, size = (G @ W.double()) * dloss.double()[:, None], (G.abs() @ W.double().abs()) * dloss.double()[:, None]
        half = torch.finfo(dtype).eps / 2
        assert ((dH.double() - want).abs() <= size * (half + 2.0 ** -17) + 2.0 ** -25)[:, 1:].all(), value
        assert dW.isfinite().all()


def test_a_million_rows_of_one_sign(tb):
    """dW's sums over the rows: equal terms whose sum fp16 holds exactly. A tensor core's accumulator
    that takes all of them cuts off 1e-9 of the sum for every element, 1e-3 here, two half steps of
    fp16; the tiles are as many as the pairs of CTAs, so that nothing else splits the rows."""
    n, d, v = 1 << 20, 19 * 256, 1000
    H = torch.ones(n, d, dtype=HF, device="cuda")
    W = torch.zeros(v, d, dtype=HF, device="cuda")
    t = torch.zeros(n, dtype=torch.int64, device="cuda")
    lse = torch.full((n,), math.log(v), device="cuda")
    dloss = torch.full((n,), 1.0 / n, device="cuda")
    _, dW = backward(tb, dloss, H, W, t, lse, "W")
    # G = 2^14 / 1000 = 16.384 is held as 1049 / 64, a tenth of a step away and far from a tie
    want = torch.full((v,), 1049 / 64 / 2 ** 14, dtype=HF, device="cuda")
    assert want[1].item() == 1049 / 64 / 2 ** 14
    assert torch.equal(dW[1:], want[1:, None].expand(v - 1, d))
    # the target's: (1049 / 64 - 16384) / 2^14 rounded, in G to a step of 8 and in dW likewise
    assert ((dW[0].double() + 1 - 1 / v).abs() <= 2.0 ** -10).all()


# rows of a matrix whose D is not a multiple of 8 start on any element, and so does a slice of them
@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("n, d, v", [(1, 1, 1), (3, 1, 2), (37, 7, 300), (130, 33, 515), (41, 770, 1003), (5, 12, 9)])
@pytest.mark.parametrize("off_h, off_w", [(1, 0), (0, 1), (3, 6), (2, 5)])
def test_operands_that_start_on_any_element(tb, n, d, v, off_h, off_w, dtype):
    H, W, t, dloss = problem(n, d, v, dtype, 15)
    loss, lse = forward(tb, H, W, t)
    dH, dW = backward(tb, dloss, H, W, t, lse)
    moved = []
    for x, off in ((H, off_h), (W, off_w)):         # between NaNs, so that nothing else can be read unseen
        buf = torch.full((x.numel() + off + 9,), float("nan"), dtype=dtype, device="cuda")
        buf[off:off + x.numel()] = x.flatten()
        moved.append(buf[off:off + x.numel()].view_as(x))
    got = forward(tb, *moved, t)
    assert torch.equal(got[0], loss) and torch.equal(got[1], lse)
    dH2, dW2 = backward(tb, dloss, *moved, t, lse)
    assert torch.equal(dH2, dH) and torch.equal(dW2, dW)


@pytest.mark.parametrize("n, d, v", [(300, 136, 900), (5000, 40, 600)])
@pytest.mark.parametrize("dtype, powers", [(BF, 16), (BF, 90), (HF, 10), (HF, 24)])
def test_row_weights_of_many_sizes(tb, n, d, v, dtype, powers):
    """Signed weights spread over powers of two, some rows far below the largest: dH keeps its accuracy
    for every row; dW is off by a rounding of H times the weight over the largest, which fp16 holds to
    half a step of 2^-24 where that is small."""
    H, W, t, dloss = problem(n, d, v, dtype, 16)
    g = torch.Generator(device="cuda").manual_seed(17)
    dloss = torch.exp2(-powers * torch.rand(n, generator=g, device="cuda")) * (torch.randint(0, 2, (n,), generator=g, device="cuda") * 2 - 1)
    dloss[7] = 64.0
    _, lse = forward(tb, H, W, t)
    dH, dW = backward(tb, dloss, H, W, t, lse)
    check_backward(dH, dW, dloss, H, W, t, lse)
    # every weight times a power of two moves nothing but the exponent, where the type has room
    if dtype == BF:
        dH2, dW2 = backward(tb, dloss * 2.0 ** -20, H, W, t, lse)
        big = dH.abs() > 2.0 ** -80
        assert torch.equal(dH2[big], (dH.float() * 2.0 ** -20).to(BF)[big])
        assert torch.equal(dW2, (dW.float() * 2.0 ** -20).to(BF))


# logits of more contracted elements than one accumulator takes: chunks of equal and of unequal length,
# one element over, several launches of the loss, tiles narrower than a pair's
@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("n, d, v", [(1, 1281, 1), (37, 1288, 700), (300, 2048, 1000), (129, 4100, 515), (513, 1500, 777),
                                     (17000, 1344, 300), (41, 4096, 20011), (5, 16384, 33), (70, 1280, 300)])
def test_long_contractions(tb, n, d, v, dtype):
    H, W, t, dloss = problem(n, d, v, dtype, 18)
    loss, lse = forward(tb, H, W, t)
    check_forward(loss, lse, H, W, t)
    again = forward(tb, H, W, t)
    assert torch.equal(again[0], loss) and torch.equal(again[1], lse)
    if dtype == HF:
        dloss = dloss * 1024
    dH, dW = backward(tb, dloss, H, W, t, lse)
    check_backward(dH, dW, dloss, H, W, t, lse)


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("d", [1024, 1280, 4096, 16384, 65536, 65544])
def test_logits_whose_terms_have_one_sign(tb, d, dtype):
    """A chunk of 1,280 elements is 80 additions of 16, each cut off by less than 2^-23 of what the sum
    has reached, half of the chunk in the mean: 80 * 2^-24 of the logit. At most 52 chunks are added in
    fp32, off by half of 2^-23 of the sum so far each. In one accumulator, 65,536 elements are off by 6e-5."""
    n, v = 3, 300
    H = torch.ones(n, d, dtype=dtype, device="cuda")
    W = torch.zeros(v, d, dtype=dtype, device="cuda")
    W[5] = 851.7 / d
    logit = W[5, 0].double().item() * d
    t = torch.tensor([5, 0, 299], device="cuda")
    loss, lse = forward(tb, H, W, t)
    room = logit * (80 + 52 + 2) * 2.0 ** -24
    assert ((lse.double() - logit).abs() <= room).all(), (lse.double() - logit).abs().max().item() / logit
    assert loss[0].abs() <= logit * 2.0 ** -23 and ((loss[1:].double() - logit).abs() <= room).all()


@pytest.mark.parametrize("n, d, v", [(300, 136, 900), (700, 40, 5003), (2000, 64, 40)])
def test_light_rows_keep_their_bits_in_fp16(tb, n, d, v):
    """Vocabulary rows that only tokens of small weight touch: one token of weight 2^12 knows its target,
    all others weigh 2^-6 to 2^-2, a part in 2^14 to 2^18 of it, and their gradients are numbers that
    fp16 holds well. Each is a product of two roundings, of G and of the scaled H, as for equal weights."""
    H, W, t, _ = problem(n, d, v, HF, 19, ignored=0.0)
    g = torch.Generator(device="cuda").manual_seed(20)
    dloss = torch.exp2(-6 + 4 * torch.rand(n, generator=g, device="cuda"))
    dloss[0] = 4096.0
    H[:, 0], W[:, 0] = 0.0, 0.0                     # the heavy token's logits: 200 at its target, else 0
    H[0] = 0.0
    H[0, 0], W[v - 1, 0] = 200.0, 1.0
    t[0] = v - 1
    t[1:] = t[1:] % (v - 1)
    _, lse = forward(tb, H, W, t)
    dH, dW = backward(tb, dloss, H, W, t, lse)
    l, err_l = logits64(H[1:], W)
    p = (l - lse[1:].double()[:, None]).exp()
    G = p.clone()
    G[torch.arange(n - 1, device="cuda"), t[1:]] -= 1.0
    G *= dloss[1:].double()[:, None]
    half = torch.finfo(HF).eps / 2
    h = H[1:].double()
    want, size = (G.T @ h)[:v - 1], (G.abs().T @ h.abs())[:v - 1]
    # G's and H's rounding, the exponent's, the additions; G below fp16's normal numbers: half a step of
    # 2^-24 under at least 2^6; elements of H below 2^-6 of the largest, half a step of what carries them
    p_err = (p * (err_l + 8 * U * 20) + 2.0 ** -31) * dloss[1:].double()[:, None]
    room = size * (2 * half + half * half + 2 * U * (n + 16)) + (p_err.T @ h.abs())[:v - 1]
    room += (G.abs().T.sum(1, keepdim=True))[:v - 1] * 2.0 ** -13 * half
    room = room + (want.abs() + room) * half + 2.0 ** -25
    off = (dW[:v - 1].double() - want).abs()
    assert (off <= room).all(), (off / room).max().item()
    # and the light rows' dH
    want, size = G @ W.double(), G.abs() @ W.double().abs()
    room = size * (half + 2 * U * (v + 16)) + p_err @ W.double().abs()
    room = room + (want.abs() + room) * half + 2.0 ** -25
    assert ((dH[1:].double() - want).abs() <= room).all()
