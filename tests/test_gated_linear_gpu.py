"""The gated projections and their gradients on the GPU, against the formulas in 64 bits.

Tolerances.  Inputs are 16-bit and exact in the reference.  A value is rounded once to the type:
at most half a step, eps/2 of itself (eps = 2^-7 for bf16, 2^-10 for fp16).  fp32 sums of n terms
in accumulators that truncate are off by at most 2^-23 times the sum of the terms' magnitudes for
every term added to the accumulator; MMAs add 16 at a time, so n/16 + 16 such steps bound it, and
the activation's few fp32 operations another 16.  The gradients' products have one operand more that was
rounded to the type (dG, dU): eps/2 of each term's magnitude.
"""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu
F32 = 2.0 ** -23


@pytest.fixture(scope="module")
def tb():
    import ln_backward_gb300
    return ln_backward_gb300


ACT = {"silu": torch.nn.functional.silu, "gelu": torch.nn.functional.gelu,
       "gelu_tanh": lambda x: torch.nn.functional.gelu(x, approximate="tanh")}
SLOPE = {"silu": 1.1, "gelu": 1.13, "gelu_tanh": 1.13}      # the largest |act'|, rounded up


def inputs(n, d, f, dtype, seed=0, grad=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    make = lambda shape, std: (torch.randn(shape, generator=g, device="cuda") * std).to(dtype)
    return make((n, d), 1.0), make((f, d), d ** -0.5), make((f, d), d ** -0.5), make((n, f), grad)


def nan_like(*shape, dtype):
    return torch.full(shape, math.nan, dtype=dtype, device="cuda")


def workspace(nbytes):
    return torch.full((nbytes,), 0xFF, dtype=torch.uint8, device="cuda")


def forward(tb, X, Wg, Wu, act, keep=True):
    n, f = X.shape[0], Wg.shape[0]
    H, G, U = (nan_like(n, f, dtype=X.dtype) for _ in range(3))
    ws = workspace(tb.tb_gated_linear_workspace_size(n, X.shape[1], f, X.dtype))
    tb.tb_gated_linear(X, Wg, Wu, H, *((G, U) if keep else (None, None)), workspace=ws, activation=act)
    return H, G, U


def backward(tb, dH, X, Wg, Wu, G, U, act, dx=True, dw=True):
    n, d = X.shape
    f = Wg.shape[0]
    dX, dWg, dWu = nan_like(n, d, dtype=X.dtype), nan_like(f, d, dtype=X.dtype), nan_like(f, d, dtype=X.dtype)
    ws = workspace(tb.tb_gated_linear_bwd_workspace_size(n, d, f, X.dtype))
    tb.tb_gated_linear_bwd(dH, X, Wg, Wu, G, U, dX if dx else None, dWg if dw else None, dWu if dw else None, ws,
                           activation=act)
    return dX, dWg, dWu


def near(got, want, slack, what):
    """got is want's rounding to its type, give or take `slack` before the rounding."""
    half = torch.finfo(got.dtype).eps / 2
    tiny = torch.finfo(got.dtype).smallest_normal * half
    off = (got.double() - want).abs() - (half * (want.abs() + slack) + slack + tiny)
    worst = off.max().item()
    assert worst <= 0, f"{what}: {worst} over the bound, {(off > 0).sum().item()} of {off.numel()}"


def check_forward(X, Wg, Wu, act, H, G, U):
    d = X.shape[1]
    x, wg, wu = X.double(), Wg.double(), Wu.double()
    g, u = x @ wg.T, x @ wu.T
    sg, su = ((d / 16 + 16) * F32 * (x.abs() @ w.abs().T) for w in (wg, wu))
    if G is not None:
        near(G, g, sg, "G")
        near(U, u, su, "U")
    a = ACT[act](g)
    slack = SLOPE[act] * sg * u.abs() + a.abs() * su + sg * su * SLOPE[act] + 16 * F32 * (a * u).abs() \
        + 2.0 ** -120 * (1 + u.abs()) + 16 * F32 * g.abs() * u.abs() * 2.0 ** -4
    near(H, a * u, slack, "H")


def check_backward(dH, X, Wg, Wu, G, U, act, dX, dWg, dWu):
    n, d, f = *X.shape, Wg.shape[0]
    half = torch.finfo(X.dtype).eps / 2
    g, u = G.double().requires_grad_(), U.double().requires_grad_()
    dg, du = torch.autograd.grad(ACT[act](g) * u, (g, u), dH.double())
    x, wg, wu = X.double(), Wg.double(), Wu.double()
    # what dG and dU are off by: one rounding, and fp32's where the slope's terms cancel
    base = 16 * F32 * dH.double().abs()
    eg = half * dg.abs() + base * (u.abs() * (1 + g.abs())).detach() + 2.0 ** -120
    eu = half * du.abs() + base * g.abs().detach() + 2.0 ** -120
    if X.dtype == torch.float16:      # held times the power of two that brings the largest to 2^14 or more
        most = max(dg.abs().max().item(), du.abs().max().item())
        eg, eu = eg + most * 2.0 ** -14 * 2.0 ** -25, eu + most * 2.0 ** -14 * 2.0 ** -25
    if dX is not None:
        slack = (eg @ wg.abs() + eu @ wu.abs()) + (2 * f / 16 + 32) * F32 * (dg.abs() @ wg.abs() + du.abs() @ wu.abs())
        near(dX, dg @ wg + du @ wu, slack, "dX")
    if dWg is not None:
        for got, y, e, what in ((dWg, dg, eg, "dWg"), (dWu, du, eu, "dWu")):
            slack = e.T @ x.abs() + (n / 16 + 32) * F32 * (y.abs().T @ x.abs())
            near(got, y.T @ x, slack, what)


# one row; the pair's first CTA alone; a row more than it; two row tiles; widths that are no whole
# tile, no whole box, no whole stage; few tiles of long contractions (split); many tiles
SIZES = [(1, 64, 64), (1, 8, 8), (3, 4096, 256), (16, 1024, 2056), (127, 192, 328), (128, 72, 1000), (129, 520, 264),
         (257, 64, 512), (300, 1160, 40), (1000, 776, 2048), (2049, 256, 96), (16, 2048, 11008), (4, 8192, 72)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("n, d, f", SIZES)
def test_forward(tb, n, d, f, dtype):
    X, Wg, Wu, _ = inputs(n, d, f, dtype, seed=n + d + f)
    act = ["silu", "gelu", "gelu_tanh"][(n + d // 8 + f // 8) % 3]
    H, G, U = forward(tb, X, Wg, Wu, act)
    check_forward(X, Wg, Wu, act, H, G, U)
    again, _, _ = forward(tb, X, Wg, Wu, act, keep=False)
    assert torch.equal(again, H)
    assert tb.tb_device_error() == 0


def test_a_very_long_contraction(tb):
    """More elements than 64 accumulators take: as many parts as it needs."""
    n, d, f = 2, 65 * 65536, 8
    X, Wg, Wu, _ = inputs(n, d, f, torch.bfloat16, seed=3)
    H, G, U = forward(tb, X, Wg, Wu, "silu")
    check_forward(X, Wg, Wu, "silu", H, G, U)
    assert tb.tb_device_error() == 0


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("n, d, f", SIZES + [(5000, 64, 136), (40000, 16, 24)])
def test_backward(tb, n, d, f, dtype):
    X, Wg, Wu, dH = inputs(n, d, f, dtype, seed=n + d + f, grad=1e-4 if dtype == torch.bfloat16 else 1e-2)
    act = ["silu", "gelu", "gelu_tanh"][(n + d // 8 + f // 8) % 3]
    G, U = (X.float() @ Wg.float().T).to(dtype), (X.float() @ Wu.float().T).to(dtype)
    dX, dWg, dWu = backward(tb, dH, X, Wg, Wu, G, U, act)
    check_backward(dH, X, Wg, Wu, G, U, act, dX, dWg, dWu)
    assert torch.equal(backward(tb, dH, X, Wg, Wu, G, U, act, dw=False)[0], dX)
    _, again_g, again_u = backward(tb, dH, X, Wg, Wu, G, U, act, dx=False)
    assert torch.equal(again_g, dWg) and torch.equal(again_u, dWu)
    assert tb.tb_device_error() == 0
