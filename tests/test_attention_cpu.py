"""What the attention calls refuse, without a GPU: every check returns before any CUDA call and no
pointer is dereferenced; and what the binding refuses."""
import ctypes

import pytest
import torch

OK, INVALID, DTYPE, MISALIGNED, ALIAS, WORKSPACE = 0, 1, 2, 3, 4, 5
F32, F16, BF16 = 0, 1, 2
B, S, HQ, HK, D = 2, 100, 4, 2, 64
NAMES = ("q", "k", "v", "out", "dout", "dq", "dk", "dv")


@pytest.fixture(scope="module")
def tb():
    import __graft_entry__
    __graft_entry__.build()
    import ln_backward_gb300
    return ln_backward_gb300


def heads(tb, at, n, **how):
    h = dict(data=at, stride_batch=S * n * D, stride_seq=n * D, stride_head=D, heads=n)
    h.update(how)
    return tb._binding.tb_heads(*(h[k] for k in ("data", "stride_batch", "stride_seq", "stride_head", "heads")))


def args(tb, how):
    a = dict(lse=0x90000000, batch=B, seq=S, dim=D, offsets=None, sequences=0, scale=0.125, dtype=BF16, ws=0xA0000000,
             ws_bytes=1 << 30)
    a.update({k: v for k, v in how.items() if k not in NAMES})
    for i, name in enumerate(NAMES):
        n = HK if name in ("k", "v", "dk", "dv") else HQ
        given = how.get(name, {})
        a[name] = None if given is None else ctypes.byref(heads(tb, 0x10000000 * (i + 1), n, **given))
    return a


def fwd(tb, **how):
    a = args(tb, how)
    return tb._binding.lib.tb_attention(a["q"], a["k"], a["v"], a["out"], a["lse"], a["batch"], a["seq"], a["dim"], a["offsets"],
                                        a["sequences"], a["scale"], a["dtype"], None)


def bwd(tb, **how):
    a = args(tb, how)
    return tb._binding.lib.tb_attention_bwd(a["dout"], a["q"], a["k"], a["v"], a["out"], a["lse"], a["dq"], a["dk"], a["dv"],
                                            a["batch"], a["seq"], a["dim"], a["offsets"], a["sequences"], a["scale"], a["dtype"],
                                            a["ws"], ctypes.c_size_t(a["ws_bytes"]), None)


Q = 0x10000000
SHARED = [
    (dict(batch=-1), INVALID), (dict(seq=-1), INVALID), (dict(seq=2 ** 25 + 1), INVALID), (dict(batch=2 ** 20 + 1), INVALID),
    (dict(dim=0), INVALID), (dict(dim=-8), INVALID), (dict(dim=12), INVALID), (dict(dim=136), INVALID), (dict(dim=256), INVALID),
    (dict(scale=0.0), INVALID), (dict(scale=-1.0), INVALID), (dict(scale=float("nan")), INVALID), (dict(scale=float("inf")), INVALID),
    (dict(dtype=F32), DTYPE), (dict(dtype=9), DTYPE),
    (dict(offsets=0xB0000000, sequences=3), INVALID),                    # offsets with a batch
    (dict(offsets=0xB0000000, sequences=-1, batch=1), INVALID), (dict(sequences=1), INVALID),
    (dict(offsets=0xB0000004, sequences=1, batch=1), MISALIGNED),
    (dict(q=None), INVALID), (dict(k=None), INVALID), (dict(v=None), INVALID), (dict(q=dict(data=None)), INVALID),
    (dict(q=dict(heads=-1)), INVALID), (dict(k=dict(heads=3), v=dict(heads=3)), INVALID),
    (dict(v=dict(heads=1)), INVALID), (dict(k=dict(stride_seq=0)), INVALID), (dict(q=dict(stride_batch=-8)), INVALID),
    (dict(v=dict(stride_head=0)), INVALID), (dict(k=dict(stride_batch=1 << 39)), INVALID),
    (dict(q=dict(data=Q + 8)), MISALIGNED), (dict(k=dict(data=2 * Q + 2)), MISALIGNED), (dict(q=dict(stride_seq=HQ * D + 4)), MISALIGNED),
    (dict(lse=0x90000002), MISALIGNED)]


@pytest.mark.parametrize("how, want", SHARED + [
    (dict(out=None), INVALID), (dict(out=dict(heads=2)), INVALID), (dict(out=dict(data=4 * Q + 8)), MISALIGNED),
    (dict(out=dict(data=Q)), ALIAS), (dict(out=dict(data=2 * Q)), ALIAS), (dict(out=dict(data=3 * Q + 16)), ALIAS),
    (dict(out=dict(stride_seq=D)), ALIAS),                               # rows of its own that meet
    (dict(lse=Q + 64), ALIAS), (dict(lse=4 * Q), ALIAS),
    (dict(offsets=4 * Q + 8, sequences=2, batch=1), ALIAS), (dict(offsets=0x90000008, sequences=2, batch=1), ALIAS)])
def test_forward_refusals(tb, how, want):
    assert fwd(tb, **how) == want


@pytest.mark.parametrize("how, want", SHARED + [
    (dict(lse=None), INVALID), (dict(dout=None), INVALID), (dict(dq=None), INVALID), (dict(dk=None), INVALID), (dict(dv=None), INVALID),
    (dict(dq=dict(heads=2)), INVALID), (dict(dk=dict(heads=1)), INVALID), (dict(dout=dict(heads=3)), INVALID),
    (dict(dq=dict(data=6 * Q + 8)), MISALIGNED), (dict(dk=dict(stride_head=D + 4)), MISALIGNED),
    (dict(dq=dict(data=Q)), ALIAS), (dict(dk=dict(data=2 * Q)), ALIAS), (dict(dv=dict(data=7 * Q)), ALIAS), (dict(dq=dict(data=5 * Q)), ALIAS),
    (dict(dv=dict(data=4 * Q)), ALIAS), (dict(lse=6 * Q), ALIAS),
    (dict(ws=None), WORKSPACE), (dict(ws_bytes=100), WORKSPACE), (dict(ws=0xA0000008), MISALIGNED), (dict(ws=Q), ALIAS),
    (dict(ws=8 * Q), ALIAS), (dict(ws=0x90000000 - 256), ALIAS)])
def test_gradient_refusals(tb, how, want):
    assert bwd(tb, **how) == want


def test_views_of_one_buffer_are_told_apart(tb):
    """dq, dk and dv as slices of a joint buffer pass every check but the workspace's."""
    n = HQ + 2 * HK
    strides = dict(stride_batch=S * n * D, stride_seq=n * D)
    joint = dict(dq=dict(data=6 * Q, **strides), dk=dict(data=6 * Q + 2 * HQ * D, **strides), dv=dict(data=6 * Q + 2 * (HQ + HK) * D, **strides))
    assert bwd(tb, ws=None, **joint) == WORKSPACE
    joint["dv"]["data"] -= 2 * D
    assert bwd(tb, ws=None, **joint) == ALIAS


def test_nothing_to_do_needs_no_gpu(tb):
    assert fwd(tb, batch=0) == OK and fwd(tb, seq=0) == OK
    assert bwd(tb, batch=0, ws=None) == OK and bwd(tb, seq=0, ws=None) == OK
    assert fwd(tb, offsets=0xB0000000, sequences=0, batch=1) == OK
    none = dict(heads=0)
    assert fwd(tb, q=none, out=none) == OK


def test_workspace_queries(tb):
    size = ctypes.c_size_t(7)
    call = tb._binding.lib.tb_attention_bwd_workspace_size
    assert call(B, S, HQ, HK, D, BF16, ctypes.byref(size)) == OK and size.value >= 8 * B * HQ * S
    assert call(0, S, HQ, HK, D, BF16, ctypes.byref(size)) == OK and size.value == 0
    assert call(B, S, HQ, HK, D, BF16, None) == INVALID
    assert call(B, S, HQ, 3, D, BF16, ctypes.byref(size)) == INVALID
    assert call(B, S, HQ, HK, 132, BF16, ctypes.byref(size)) == INVALID
    assert call(B, S, HQ, HK, D, F32, ctypes.byref(size)) == DTYPE


def test_binding_refuses(tb):
    q, k = torch.zeros(1, 8, 4, 64, dtype=torch.bfloat16), torch.zeros(1, 8, 2, 64, dtype=torch.bfloat16)
    o = torch.zeros_like(q)
    with pytest.raises(ValueError, match="CUDA"):
        tb.tb_attention(q, k, k.clone(), o)
    for bad, what in (((q[0], k, k, o), "q must be"), ((q, k[:, :4], k, o), "k must be"), ((q, k, k[:, :, :1], o), "heads"),
                      ((q, k, k, k), "heads"), ((q, k.half(), k, o), "must be torch.bfloat16"),
                      ((q.transpose(2, 3).contiguous().transpose(2, 3), k, k, o), "contiguous")):
        with pytest.raises(ValueError, match=what):
            tb.tb_attention(*bad)


def test_no_query_head_leaves_no_gradient_of_keys(tb):
    """dk and dv would be sums over nothing: heads of keys without one that asks them are refused, no head at all is not."""
    none = dict(heads=0)
    query = dict(q=none, dout=none, out=none, dq=none)
    assert bwd(tb, **query) == INVALID
    assert bwd(tb, **query, k=none, v=none, dk=none, dv=none, ws=None) == OK


def test_scale_that_leaves_the_range_in_powers_of_two(tb):
    assert fwd(tb, scale=3e38) == INVALID and bwd(tb, scale=3e38) == INVALID
    assert fwd(tb, scale=2.0 ** 127, batch=0) == OK


def test_workspace_of_a_call_beyond_every_grid(tb):
    size = ctypes.c_size_t(7)
    call = tb._binding.lib.tb_attention_bwd_workspace_size
    assert call(2 ** 20, 2 ** 25, 2 ** 20, 2 ** 20, 128, BF16, ctypes.byref(size)) == INVALID
    assert call(1, 2 ** 25, 64, 8, 128, BF16, ctypes.byref(size)) == OK and size.value >= 8 * 64 * 2 ** 25
