"""The gated projections and their gradients where a pair of CTAs works on tile after tile: more tiles than two
accumulators hold, more row tiles than are walked together, tiles of fp32 sums before tiles of 16-bit results."""
import pytest
import torch

from test_gated_linear_gpu import backward, check_backward, check_forward, forward, inputs

pytestmark = pytest.mark.gpu
BF, HALF = torch.bfloat16, torch.float16


@pytest.fixture(scope="module")
def tb():
    import ln_backward_gb300
    return ln_backward_gb300


# few rows: dX's contraction is cut into sums, dW's, of one to four stages, is not: sums and results leave a pair in turn
@pytest.mark.parametrize("n, d, f", [(16, 2048, 4096), (64, 2048, 8192), (50, 720, 5376), (24, 216, 9328), (256, 1024, 4096),
                                     (58, 248, 10296), (33, 2696, 880), (200, 1656, 2152)])
@pytest.mark.parametrize("dtype", [BF, HALF])
def test_sums_of_one_product_beside_results_of_the_other(tb, n, d, f, dtype):
    X, Wg, Wu, dH = inputs(n, d, f, dtype, seed=n + d + f, grad=1e-4 if dtype == BF else 1e-2)
    G, U = (X.float() @ Wg.float().T).to(dtype), (X.float() @ Wu.float().T).to(dtype)
    first = backward(tb, dH, X, Wg, Wu, G, U, "silu")
    check_backward(dH, X, Wg, Wu, G, U, "silu", *first)
    for _ in range(20):
        assert all(torch.equal(x, y) for x, y in zip(backward(tb, dH, X, Wg, Wu, G, U, "silu"), first))
    assert tb.tb_device_error() == 0


# 20 row tiles, the last a row high, of five and more columns of tiles: three and more tiles a pair
@pytest.mark.parametrize("n, d, f, dtype, act", [(4865, 200, 1672, BF, "silu"), (4865, 64, 4096, HALF, "gelu"), (8192, 512, 1408, BF, "gelu_tanh")])
def test_many_tiles(tb, n, d, f, dtype, act):
    X, Wg, Wu, dH = inputs(n, d, f, dtype, seed=n, grad=1e-4 if dtype == BF else 1e-2)
    H, G, U = forward(tb, X, Wg, Wu, act)
    check_forward(X, Wg, Wu, act, H, G, U)
    check_backward(dH, X, Wg, Wu, G, U, act, *backward(tb, dH, X, Wg, Wu, G, U, act))
    assert tb.tb_device_error() == 0
