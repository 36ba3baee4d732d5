"""Attention of nothing: sizes of 0 that are answered, and those that are refused with the library's own error."""
import pytest
import torch

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.fixture(scope="module")
def tb():
    import ln_backward_gb300
    return ln_backward_gb300


def tensors(b, s, hq, hk, d):
    make = lambda h: torch.zeros(b, s, h, d, dtype=BF, device="cuda")
    return [make(h) for h in (hq, hk, hk, hq, hq)], torch.zeros(b, hq, s, device="cuda"), [make(h) for h in (hq, hk, hk)]


@pytest.mark.parametrize("sizes", [(0, 8, 4, 2, 64), (2, 0, 4, 2, 64), (2, 8, 0, 0, 64)])
def test_nothing_to_do(tb, sizes):
    (q, k, v, dout, out), lse, grads = tensors(*sizes)
    tb.tb_attention(q, k, v, out, lse)
    tb.tb_attention_bwd(dout, q, k, v, out, lse, *grads, None)
    assert tb.tb_device_error() == 0


def test_heads_of_no_element_are_refused(tb):
    (q, k, v, dout, out), lse, grads = tensors(2, 8, 4, 2, 0)
    for call in (lambda: tb.tb_attention(q, k, v, out, lse), lambda: tb.tb_attention_bwd(dout, q, k, v, out, lse, *grads, None)):
        with pytest.raises(tb.TbError) as e:
            call()
        assert e.value.code == 1
