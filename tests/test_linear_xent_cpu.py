"""What the output layer's loss refuses, without a GPU: every check returns before any CUDA call
and no pointer is dereferenced."""
import ctypes

import pytest
import torch

OK, INVALID, DTYPE, MISALIGNED, ALIAS, WORKSPACE = 0, 1, 2, 3, 4, 5
F32, F16, BF16 = 0, 1, 2
N, D, V = 16, 64, 100


@pytest.fixture(scope="module")
def tb():
    import __graft_entry__
    __graft_entry__.build()
    import ln_backward_gb300
    return ln_backward_gb300


BASE = dict(H=0x1000000, W=0x2000000, t=0x3000000, loss=0x4000000, lse=0x5000000, dloss=0x6000000,
            dH=0x7000000, dW=0x8000000, n=N, d=D, v=V, dtype=BF16, ws=0x9000000, ws_bytes=0)


def fwd(tb, **how):
    a = {**BASE, **how}
    return tb._binding.lib.tb_linear_xent(a["H"], a["W"], a["t"], a["loss"], a["lse"], a["n"], a["d"], a["v"], -100,
                                          a["dtype"], a["ws"], a["ws_bytes"], None)


def bwd(tb, **how):
    a = {**BASE, **how}
    return tb._binding.lib.tb_linear_xent_bwd(a["dloss"], a["H"], a["W"], a["t"], a["lse"], a["dH"], a["dW"], a["n"],
                                              a["d"], a["v"], -100, a["dtype"], a["ws"], a["ws_bytes"], None)


SHARED = [
    (dict(n=-1), INVALID), (dict(d=0), INVALID), (dict(v=0), INVALID), (dict(d=-1), INVALID),
    (dict(n=2 ** 31), INVALID), (dict(v=2 ** 31), INVALID), (dict(d=2 ** 31), INVALID),
    (dict(n=2 ** 25, d=2 ** 16), INVALID), (dict(v=2 ** 25, d=2 ** 16), INVALID),
    (dict(dtype=F32), DTYPE), (dict(dtype=7), DTYPE), (dict(H=None), INVALID), (dict(W=None), INVALID),
    (dict(t=None), INVALID), (dict(lse=None), INVALID), (dict(H=0x1000008), MISALIGNED),
    (dict(W=0x2000002), MISALIGNED), (dict(t=0x3000004), MISALIGNED), (dict(lse=0x5000002), MISALIGNED)]


@pytest.mark.parametrize("how, want", SHARED + [
    (dict(loss=None), INVALID), (dict(loss=0x4000001), MISALIGNED), (dict(loss=0x5000000), ALIAS),
    (dict(lse=0x4000000 + 4 * N - 4), ALIAS), (dict(loss=0x1000000 + 2 * N * D - 4), ALIAS),
    (dict(lse=0x2000000), ALIAS), (dict(loss=0x3000000), ALIAS)])
def test_loss_refusals(tb, how, want):
    assert fwd(tb, **how) == want


@pytest.mark.parametrize("how, want", SHARED + [
    (dict(dloss=None), INVALID), (dict(dH=None, dW=None), INVALID), (dict(dloss=0x6000002), MISALIGNED),
    (dict(dH=0x7000001), MISALIGNED), (dict(dW=0x8000001), MISALIGNED), (dict(dH=0x1000000), ALIAS),
    (dict(dW=0x2000000 + 2 * V * D - 2), ALIAS), (dict(dH=0x8000000), ALIAS), (dict(dH=0x6000000), ALIAS),
    (dict(dW=0x5000000), ALIAS), (dict(dH=0x3000000), ALIAS)])
def test_gradient_refusals(tb, how, want):
    assert bwd(tb, **how) == want


def test_no_rows_needs_no_gpu(tb):
    assert fwd(tb, n=0) == OK
    assert bwd(tb, n=0, dW=None) == OK
    assert bwd(tb, n=0, dH=None, dW=0x8000001) == MISALIGNED


@pytest.mark.parametrize("name", ["tb_linear_xent_workspace_size", "tb_linear_xent_bwd_workspace_size"])
def test_workspace_queries(tb, name):
    f, n = getattr(tb._binding.lib, name), ctypes.c_size_t(5)
    assert f(N, D, V, BF16, None) == INVALID
    assert f(-1, D, V, BF16, ctypes.byref(n)) == INVALID
    assert f(N, 0, V, BF16, ctypes.byref(n)) == INVALID
    assert f(N, D, V, F32, ctypes.byref(n)) == DTYPE
    assert f(0, D, V, BF16, ctypes.byref(n)) == OK and n.value == 0


def test_binding_refusals(tb):
    H, W = torch.zeros(N, D, dtype=torch.bfloat16), torch.zeros(V, D, dtype=torch.bfloat16)
    t, f = torch.zeros(N, dtype=torch.int64), torch.zeros(N)
    with pytest.raises(ValueError, match="share D"):
        tb.tb_linear_xent(H, W[:, :32], t, f, f, None)
    with pytest.raises(ValueError, match="share D"):
        tb.tb_linear_xent(H, W.half(), t, f, f, None)
    with pytest.raises(ValueError, match="targets"):
        tb.tb_linear_xent(H, W, t.int(), f, f, None)
    with pytest.raises(ValueError, match="loss"):
        tb.tb_linear_xent(H, W, t, f[:-1], f, None)
    with pytest.raises(ValueError, match="lse"):
        tb.tb_linear_xent_bwd(f, H, W, t, f.double(), H, W, None)
    with pytest.raises(ValueError, match="dW"):
        tb.tb_linear_xent_bwd(f, H, W, t, f, None, W.float(), None)
    with pytest.raises(ValueError, match="CUDA"):
        tb.tb_linear_xent(H, W, t, f, f.clone(), None)


@pytest.mark.parametrize("how, refused", [(dict(H=0x1000002, d=63), False), (dict(W=0x2000006, d=65), False),
                                          (dict(H=0x1000001, d=63), True), (dict(W=0x2000003, d=63), True),
                                          (dict(H=0x1000002, d=72), True), (dict(W=0x2000008, d=8), True)])
def test_alignment_of_the_operands(tb, how, refused):
    """16 bytes where the matrices are read as they are, an element where a padded copy is."""
    for call in (fwd, bwd):
        assert (call(tb, **how) == MISALIGNED) == refused
