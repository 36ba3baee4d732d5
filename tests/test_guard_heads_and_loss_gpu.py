"""Guard regions around every output and every workspace of the rotary, query/key norm and
output-layer entry points (see test_guard_gpu.py), and what they refuse of a workspace.

The sizes take every way in which a call is cut up: several pieces of the vocabulary, dH split over it,
dW over the rows, padded copies, eight and sixteen epilogue warps, results that leave by TMA and
element by element."""
import ctypes

import pytest
import torch

from test_guard_gpu import Guarded
from test_linear_xent_gpu import problem

pytestmark = pytest.mark.gpu
BF, HF, FP = torch.bfloat16, torch.float16, torch.float32
OK, ALIAS, WORKSPACE, MISALIGNED = 0, 4, 5, 3


@pytest.fixture(scope="module")
def tb():
    import ln_backward_gb300
    return ln_backward_gb300


@pytest.mark.parametrize("dtype", [BF, HF, FP])
@pytest.mark.parametrize("shape, rot, shift", [((2, 7, 4, 2, 128), 128, 0), ((1, 131, 3, 1, 80), 32, 0), ((3, 5, 2, 1, 33), 18, 2),
                                               ((1, 9, 5, 2, 180), 60, 0), ((1, 601, 1, 1, 64), 64, 0), ((2, 3, 2, 1, 512), 256, 4)])
def test_heads_stay_in_bounds(tb, shape, rot, shift, dtype):
    b, s, hq, hk, d = shape
    g = torch.Generator(device="cuda").manual_seed(5)
    q, k, gq, gk = (torch.randn(b, s, h, d, generator=g, device="cuda").to(dtype) for h in (hq, hk, hq, hk))
    gam = [torch.ones(d, device="cuda") for _ in range(2)]
    freqs, _ = tb.tb_rope_freqs(rot)
    shift = shift // 2 * q.element_size()
    # [heads, dim] rows end the buffer where a view of another layout would go on
    out = [Guarded((b, s, h, d), dtype, shift) for h in (hq, hk, hq, hk)]
    inv = [Guarded((b, s, h), FP, 4) for h in (hq, hk)]
    dg = [Guarded((d,), FP, 4) for _ in range(2)]
    ws = Guarded((tb.tb_qk_norm_rope_bwd_workspace_size(*shape, dtype),), torch.uint8)
    for fn in (tb.tb_rope, tb.tb_rope_bwd):
        fn(q, k, out[0].t, out[1].t, freqs)
    tb.tb_qk_norm_rope(q, k, *gam, out[0].t, out[1].t, inv[0].t, inv[1].t, freqs=freqs, interleaved=True)
    tb.tb_qk_norm_rope_bwd(gq, gk, q, k, inv[0].t, inv[1].t, *gam, out[2].t, out[3].t, dg[0].t, dg[1].t, freqs=freqs,
                           interleaved=True, workspace=ws.t)
    for x in (*out, *inv, *dg, ws):
        assert x.margins_intact()


@pytest.mark.parametrize("dtype", [BF, HF, FP])
def test_heads_of_a_joint_buffer_stay_in_their_rows(tb, dtype):
    """Outputs that are slices: what lies between their rows is as it was."""
    b, s, hq, hk, d, rot = 2, 9, 3, 2, 80, 48
    buf = torch.full((b, s, hq + 2 * hk + 1, d + 16), 7.0, dtype=dtype, device="cuda")
    q, k = (torch.randn(b, s, h, d, device="cuda").to(dtype) for h in (hq, hk))
    yq, yk = buf[:, :, :hq, :d], buf[:, :, hq + hk:hq + 2 * hk, 16:]
    freqs, _ = tb.tb_rope_freqs(rot)
    tb.tb_qk_norm_rope(q, k, torch.ones(d, device="cuda"), torch.ones(d, device="cuda"), yq, yk, freqs=freqs)
    tb.tb_rope(q, k, yq, yk, freqs)
    yq.fill_(7.0)
    yk.fill_(7.0)
    assert (buf == 7.0).all()


LOSS = [(1, 8, 1, BF), (37, 72, 300, BF), (300, 200, 2049, HF), (130, 33, 515, BF), (257, 40, 1000, HF), (37, 768, 9001, BF),
        (20000, 32, 7000, BF), (20000, 33, 7000, HF), (5000, 40, 600, BF), (6000, 7, 3, HF), (1021, 768, 5003, HF),
        (16500, 64, 300, BF)]


@pytest.mark.parametrize("shift", [0, 2])
@pytest.mark.parametrize("n, d, v, dtype", LOSS)
def test_loss_stays_in_bounds(tb, n, d, v, dtype, shift):
    H, W, t, dloss = problem(n, d, v, dtype, 21)
    loss, lse = Guarded((n,), FP, 2 * shift), Guarded((n,), FP, 2 * shift)
    ws = Guarded((tb.tb_linear_xent_workspace_size(n, d, v, dtype),), torch.uint8)
    tb.tb_linear_xent(H, W, t, loss.t, lse.t, ws.t)
    for x in (loss, lse, ws):
        assert x.margins_intact()
    dH, dW = Guarded((n, d), dtype, shift), Guarded((v, d), dtype, shift)
    ws = Guarded((tb.tb_linear_xent_bwd_workspace_size(n, d, v, dtype),), torch.uint8)
    for want in ((dH.t, dW.t), (dH.t, None), (None, dW.t)):
        tb.tb_linear_xent_bwd(dloss, H, W, t, lse.t, *want, ws.t)
        for x in (dH, dW, ws):
            assert x.margins_intact()
    assert dH.t.isfinite().all() and dW.t.isfinite().all()


def code(call):
    """Status of a binding's call."""
    import ln_backward_gb300 as tb
    try:
        call()
    except tb.TbError as e:
        return e.code
    return OK


@pytest.mark.parametrize("d", [64, 33])
def test_workspaces_of_the_loss_that_are_refused(tb, d):
    n, v = 40, 300
    H, W, t, dloss = problem(n, d, v, BF, 22)
    loss, lse = torch.zeros(n, device="cuda"), torch.zeros(n, device="cuda")
    dH, dW = torch.zeros_like(H), torch.zeros_like(W)
    need = tb.tb_linear_xent_workspace_size(n, d, v, BF), tb.tb_linear_xent_bwd_workspace_size(n, d, v, BF)
    big = torch.zeros(max(need) + 64, dtype=torch.uint8, device="cuda")

    def fwd(ws):
        return code(lambda: tb.tb_linear_xent(H, W, t, loss, lse, ws))

    def bwd(ws):
        return code(lambda: tb.tb_linear_xent_bwd(dloss, H, W, t, lse, dH, dW, ws))

    for call, size in ((fwd, need[0]), (bwd, need[1])):
        assert call(None) == WORKSPACE and call(big[:size - 1]) == WORKSPACE
        assert call(big[8:8 + size]) == MISALIGNED
        assert call(big[16:16 + size]) == OK
        for x in (H, W, t, lse) + ((loss,) if call is fwd else (dloss, dH, dW)):
            # a workspace that ends in, begins in or holds the buffer
            lib, at, end = tb._binding.lib, x.data_ptr(), x.data_ptr() + x.numel() * x.element_size()
            for p in ((at + 16 - size) // 16 * 16, (end - 1) // 16 * 16, (at - size // 2) // 16 * 16):
                s = torch.cuda.current_stream().cuda_stream
                if call is fwd:
                    got = lib.tb_linear_xent(H.data_ptr(), W.data_ptr(), t.data_ptr(), loss.data_ptr(), lse.data_ptr(), n, d,
                                             v, -100, 2, p, ctypes.c_size_t(size), s)
                else:
                    got = lib.tb_linear_xent_bwd(dloss.data_ptr(), H.data_ptr(), W.data_ptr(), t.data_ptr(), lse.data_ptr(),
                                                 dH.data_ptr(), dW.data_ptr(), n, d, v, -100, 2, p, ctypes.c_size_t(size), s)
                if p < end and p + size > at:
                    assert got == ALIAS
    torch.cuda.synchronize()


def test_workspaces_of_the_norm_that_are_refused(tb):
    b, s, hq, hk, d = 2, 3, 4, 2, 64
    q, k, dq, dk = (torch.randn(b, s, h, d, device="cuda").to(BF) for h in (hq, hk, hq, hk))
    inv = [torch.ones(b, s, h, device="cuda") for h in (hq, hk)]
    gam = [torch.ones(d, device="cuda") for _ in range(4)]
    size = tb.tb_qk_norm_rope_bwd_workspace_size(b, s, hq, hk, d, BF)
    big = torch.zeros(size + 64, dtype=torch.uint8, device="cuda")

    def call(ws, dgq=gam[2], oq=dq):
        return code(lambda: tb.tb_qk_norm_rope_bwd(q, k, q, k, *inv, *gam[:2], oq, dk, dgq, gam[3], workspace=ws))

    assert call(None) == WORKSPACE and call(big[:size - 1]) == WORKSPACE and call(big[4:4 + size]) == MISALIGNED
    assert call(big[16:16 + size]) == OK
    inside = big[16:16 + 4 * d].view(FP)
    assert call(big[:size], dgq=inside) == ALIAS
    assert call(big[:size], oq=big[1024:1024 + 2 * q.numel()].view(BF).view(q.shape)) == ALIAS


def test_reads_and_writes_beyond_32_bits(tb):
    """An output layer of more than 2^31 weights: the rows at its end are read and written."""
    n, d, v = 9, 4096, 600_001
    g = torch.Generator(device="cuda").manual_seed(23)
    W = torch.zeros(v, d, dtype=BF, device="cuda")
    W[-5:] = torch.randn(5, d, generator=g, device="cuda").to(BF) * 0.05
    H = torch.randn(n, d, generator=g, device="cuda").to(BF)
    t = torch.tensor([0, 1, v - 1, v - 2, v - 5, v - 6, v // 2, -100, v - 1], device="cuda")
    loss, lse = torch.empty(n, device="cuda"), torch.empty(n, device="cuda")
    ws = torch.empty(max(tb.tb_linear_xent_workspace_size(n, d, v, BF), tb.tb_linear_xent_bwd_workspace_size(n, d, v, BF)),
                     dtype=torch.uint8, device="cuda")
    tb.tb_linear_xent(H, W, t, loss, lse, ws)
    l = H.double() @ W[-5:].double().T                    # all other logits are 0
    want = torch.log(l.exp().sum(-1) + (v - 5))
    keep = t >= 0
    logit = torch.where(t >= v - 5, l.gather(1, (t - (v - 5)).clamp(0, 4)[:, None])[:, 0], 0.0)
    room = 2.0 ** -23 * (d + 8) * (H.double().abs() @ W[-5:].double().abs().T).max() + 2.0 ** -24 * (v / 8 + 600)
    assert ((lse.double() - want).abs() <= room).all()
    assert ((loss.double() - (want - logit) * keep).abs() <= 2 * room).all()
    dloss, dH, dW = torch.full((n,), 1.0, device="cuda"), torch.empty_like(H), torch.full_like(W, 3.0)
    tb.tb_linear_xent_bwd(dloss, H, W, t, lse, dH, dW, ws)
    p = (l - lse.double()[:, None]).exp()
    p[torch.arange(n, device="cuda"), (t - (v - 5)).clamp(0, 4)] -= (t >= v - 5).double()
    p *= keep[:, None]
    half = torch.finfo(BF).eps / 2
    ref = p.T @ H.double()
    size = p.abs().T @ H.double().abs()
    assert ((dW[-5:].double() - ref).abs() <= size * (2 * half + 2.0 ** -12) + ref.abs() * half).all()
    ref, size = p @ W[-5:].double(), p.abs() @ W[-5:].double().abs()
    assert ((dH.double() - ref).abs() <= size * (half + 2.0 ** -12) + ref.abs() * half).all()
    rest = torch.exp(-lse.double())                       # p of every other column
    for row in (2, 1000, v // 2 + 1, v - 7):              # rows that are nobody's target
        ref = (rest * keep) @ H.double()
        assert ((dW[row].double() - ref).abs() <= (rest * keep) @ H.double().abs() * (2 * half + 2.0 ** -12) + ref.abs() * half).all()
