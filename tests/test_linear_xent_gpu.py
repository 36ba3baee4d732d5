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
