"""What the gated projections refuse, without a GPU: every check returns before any CUDA call and no
pointer is dereferenced; and what the binding refuses."""
import ctypes

import pytest
import torch

OK, INVALID, DTYPE, MISALIGNED, ALIAS, WORKSPACE = 0, 1, 2, 3, 4, 5
F32, F16, BF16 = 0, 1, 2
N, D, F = 16, 64, 96
BASE = dict(X=0x1000000, Wg=0x2000000, Wu=0x3000000, H=0x4000000, G=0x5000000, U=0x6000000, dH=0x7000000, dX=0x8000000, dWg=0x9000000,
            dWu=0xA000000, n=N, d=D, f=F, act=0, dtype=BF16, ws=0xB000000, ws_bytes=0)


@pytest.fixture(scope="module")
def tb():
    import __graft_entry__
    __graft_entry__.build()
    import ln_backward_gb300
    return ln_backward_gb300


def fwd(tb, **how):
    a = {**BASE, **how}
    return tb._binding.lib.tb_gated_linear(a["X"], a["Wg"], a["Wu"], a["H"], a["G"], a["U"], a["n"], a["d"], a["f"], a["act"],
                                           a["dtype"], a["ws"], ctypes.c_size_t(a["ws_bytes"]), None)


def bwd(tb, **how):
    a = {**BASE, **how}
    return tb._binding.lib.tb_gated_linear_bwd(a["dH"], a["X"], a["Wg"], a["Wu"], a["G"], a["U"], a["dX"], a["dWg"], a["dWu"], a["n"],
                                               a["d"], a["f"], a["act"], a["dtype"], a["ws"], ctypes.c_size_t(a["ws_bytes"]), None)


SHARED = [
    (dict(n=-1), INVALID), (dict(d=0), INVALID), (dict(f=0), INVALID), (dict(d=-8), INVALID), (dict(d=12), INVALID), (dict(f=4), INVALID),
    (dict(n=2 ** 25), INVALID), (dict(d=2 ** 25), INVALID), (dict(f=2 ** 25), INVALID), (dict(n=2 ** 24, d=2 ** 16), INVALID),
    (dict(n=2 ** 24, f=2 ** 16), INVALID), (dict(d=2 ** 20, f=2 ** 20), INVALID), (dict(dtype=F32), DTYPE), (dict(dtype=9), DTYPE),
    (dict(act=-1), INVALID), (dict(act=3), INVALID), (dict(X=None), INVALID), (dict(Wg=None), INVALID), (dict(Wu=None), INVALID),
    (dict(G=None), INVALID), (dict(U=None), INVALID), (dict(X=0x1000008), MISALIGNED), (dict(Wg=0x2000002), MISALIGNED),
    (dict(Wu=0x3000004), MISALIGNED), (dict(G=0x5000008), MISALIGNED), (dict(U=0x6000002), MISALIGNED)]


@pytest.mark.parametrize("how, want", SHARED + [
    (dict(H=None), INVALID), (dict(H=0x4000008), MISALIGNED), (dict(H=0x1000000), ALIAS), (dict(H=0x2000000 + 2 * F * D - 16), ALIAS),
    (dict(G=0x4000000), ALIAS), (dict(U=0x5000000 + 2 * N * F - 16), ALIAS), (dict(U=0x3000000), ALIAS)])
def test_forward_refusals(tb, how, want):
    assert fwd(tb, **how) == want


@pytest.mark.parametrize("how, want", SHARED + [
    (dict(dH=None), INVALID), (dict(dH=0x7000008), MISALIGNED), (dict(dWg=None), INVALID), (dict(dWu=None), INVALID),
    (dict(dX=None, dWg=None, dWu=None), INVALID), (dict(dX=0x8000008), MISALIGNED), (dict(dWg=0x9000002), MISALIGNED),
    (dict(dX=0x1000000), ALIAS), (dict(dWu=0x9000000), ALIAS), (dict(dWg=0x2000000), ALIAS), (dict(dX=0x7000000), ALIAS),
    (dict(dWu=0x6000000), ALIAS)])
def test_gradient_refusals(tb, how, want):
    assert bwd(tb, **how) == want


def test_no_rows_needs_no_gpu(tb):
    assert fwd(tb, n=0) == OK
    assert bwd(tb, n=0, dWg=None, dWu=None) == OK
    assert bwd(tb, n=0, dWg=0x9000008) == MISALIGNED


@pytest.mark.parametrize("name", ["tb_gated_linear_workspace_size", "tb_gated_linear_bwd_workspace_size"])
def test_workspace_queries(tb, name):
    call, size = getattr(tb._binding.lib, name), ctypes.c_size_t(7)
    assert call(0, D, F, BF16, ctypes.byref(size)) == OK and size.value == 0
    assert call(N, D, F, BF16, None) == INVALID
    assert call(N, D + 1, F, BF16, ctypes.byref(size)) == INVALID
    assert call(N, D, F, F32, ctypes.byref(size)) == DTYPE


def test_binding_refuses(tb):
    bf = torch.bfloat16
    X, W, H = torch.zeros(N, D, dtype=bf), torch.zeros(F, D, dtype=bf), torch.zeros(N, F, dtype=bf)
    with pytest.raises(ValueError, match="CUDA"):
        tb.tb_gated_linear(X, W, W.clone(), H)
    for bad, what in (((X, W, W[:8], H), "must be"), ((X, W[:, :8], W[:, :8], H), "must be"), ((X, W.half(), W, H), "dtype"),
                      ((X, W, W, H[:4]), "H must hold"), ((X, W, W, H, H[:4], H), "G must hold")):
        with pytest.raises(ValueError, match=what):
            tb.tb_gated_linear(*bad)
    with pytest.raises(ValueError, match="activation"):
        tb.tb_gated_linear(X, W, W, H, activation="tanh")
    with pytest.raises(ValueError, match="dX must hold"):
        tb.tb_gated_linear_bwd(H, X, W, W, H, H, X[:4], W, W, None)
