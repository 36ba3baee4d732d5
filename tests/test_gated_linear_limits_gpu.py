"""The activations and their slopes at the ends of their types: where powers of G leave fp32, a slope is 0 or 1."""
import pytest
import torch

from test_gated_linear_gpu import ACT, backward, near

pytestmark = pytest.mark.gpu
BF, HALF = torch.bfloat16, torch.float16
LARGE = [8.0, 15.9, 16.1, 30.0, 100.0, 1e4, 6e4]
HUGE = [1e9, 1e12, 1e13, 2e13, 1e18, 1.8e19, 2e19, 1e25, 1e30, 1e37, 2.1e38, 3.3e38]


@pytest.fixture(scope="module")
def tb():
    import ln_backward_gb300
    return ln_backward_gb300


@pytest.mark.parametrize("act", list(ACT))
@pytest.mark.parametrize("dtype", [BF, HALF])
def test_slopes_of_large_values(tb, dtype, act):
    """One row of G by itself: dWg is dG times X's one, dWu the activation of each element (by a dH that keeps it in range)."""
    big = LARGE + (HUGE if dtype == BF else [])
    g = torch.tensor([s * x for x in big for s in (1, -1)], device="cuda")
    f = (g.numel() + 7) // 8 * 8
    G = torch.zeros(1, f, device="cuda")
    G[0, :g.numel()] = g
    G = G.to(dtype)
    X, W = torch.zeros(1, 8, dtype=dtype, device="cuda"), torch.zeros(f, 8, dtype=dtype, device="cuda")
    X[0, 0] = 1
    dH, U = torch.full_like(G, 0.5), torch.full_like(G, 2.0)
    dX, dWg, dWu = backward(tb, dH, X, W, W, G, U, act)
    g64 = G.double().requires_grad_()
    a = ACT[act](g64)
    slope, = torch.autograd.grad(a.sum(), g64)
    slope = slope.nan_to_num(0.0)                # (64 bits' own cube of 1e37 and more is not needed: both ends are flat)
    slope = torch.where(G.double().abs() > 100, (G > 0).double(), slope)
    # fp32's terms of the slope cancel where it is flat; fp16: held times a power of two by the largest of all
    slack = 32 * 2.0 ** -23 * torch.ones_like(slope) * (1 + (G.double().abs() < 100) * 16)
    most = max(1.0, (a.detach() * 0.5).abs().max().item())
    floor = most * 2.0 ** -39 if dtype == HALF else 0.0
    near(dWg[:, 0], slope[0], slack[0] + floor, "dWg")
    near(dWu[:, 0], (a.detach() * 0.5)[0], 64 * 2.0 ** -23 * (1 + a.detach()[0].abs()) + floor, "dWu")
    assert (dX == 0).all() and tb.tb_device_error() == 0
