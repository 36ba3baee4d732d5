"""Rotary positions and the norm of queries and keys on the head sizes that change how a head is
dealt to lanes: every number of lanes that is known when compiling, two units a lane, whole warps;
the general kernel's largest heads; views whose strides pass 32 bits; the serving form's bits.

The checks are those of test_rope_gpu.py."""
import pytest
import torch

import rope_reference as ref
import test_rope_gpu as base

pytestmark = pytest.mark.gpu
BF, HF, FP = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module")
def tb():
    import ln_backward_gb300
    return ln_backward_gb300


# 16-bit heads in 16-byte vectors: 5, 6, 4, 8, 12, 16, 24, 32 lanes, and 10 that are not compiled in;
# the same sizes in fp32: 10, 12, 8, 16, 24, 32 and more than a warp has
SIZES = [((2, 5, 7, 3, 80), 80), ((1, 9, 6, 1, 80), 32), ((2, 4, 6, 2, 96), 96), ((3, 3, 5, 5, 96), 32),
         ((2, 3, 4, 2, 64), 32), ((1, 7, 3, 2, 128), 64), ((2, 3, 5, 2, 192), 192), ((1, 5, 2, 1, 160), 160),
         ((1, 4, 3, 1, 256), 256), ((1, 5, 2, 1, 384), 128), ((1, 6, 3, 2, 512), 256), ((2, 3, 2, 1, 512), 512),
         # two units of two elements a lane, with units that no lane holds: 33, 45, 51 and 63 of them
         ((2, 3, 3, 1, 132), 132), ((1, 7, 3, 2, 180), 180), ((2, 5, 2, 1, 180), 60), ((1, 4, 2, 2, 204), 100),
         ((1, 3, 2, 1, 252), 4), ((1, 40, 1, 1, 180), 0),
         # aligned heads that are wider than a warp's vectors
         ((1, 3, 2, 1, 1024), 1024), ((1, 3, 2, 1, 264), 264)]


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype", [BF, HF, FP])
@pytest.mark.parametrize("shape, rot", [(s, r) for s, r in SIZES if r])
def test_rotation(tb, shape, rot, dtype, interleaved):
    base.test_rotation_and_its_gradient(tb, shape, rot, dtype, interleaved)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype", [BF, HF, FP])
@pytest.mark.parametrize("shape, rot", SIZES)
def test_norm(tb, shape, rot, dtype, interleaved):
    base.test_norm_and_rotation(tb, shape, rot, dtype, interleaved)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype", [BF, HF, FP])
@pytest.mark.parametrize("shape, rot", SIZES)
def test_norm_gradient(tb, shape, rot, dtype, interleaved):
    base.test_norm_gradient(tb, shape, rot, dtype, interleaved)


# gradients in which a warp takes several tokens, one after another
@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("shape, rot, interleaved", [((1, 6001, 3, 1, 180), 180, False), ((2, 3001, 5, 2, 96), 96, True),
                                                     ((1, 5003, 7, 1, 80), 80, False), ((1, 4001, 2, 1, 512), 256, True)])
def test_gradient_in_place_over_many_tokens(tb, shape, rot, interleaved, dtype):
    base.test_gradient_in_place_over_many_tokens(tb, shape, rot, interleaved, dtype)


@pytest.mark.parametrize("dtype", [BF, HF, FP])
@pytest.mark.parametrize("shape, rot", [((2, 7, 4, 2, 128), 128), ((2, 9, 3, 3, 80), 40), ((1, 5, 3, 1, 33), 32)])
def test_serving_form_gives_the_same_bits(tb, shape, rot, dtype):
    turns, freqs, pos, angle, gam = base._case(shape, rot, 41)
    xq, xk, _ = base.make(shape, dtype, "qkv", 42)
    saved = [torch.empty_like(x) for x in (xq, xk)]
    plain = [torch.empty_like(x) for x in (xq, xk)]
    inv = [torch.empty(x.shape[:3], device="cuda") for x in (xq, xk)]
    kw = dict(eps=1e-5, freqs=freqs, positions=pos)
    tb.tb_qk_norm_rope(xq, xk, *gam, *saved, *inv, **kw)
    tb.tb_qk_norm_rope(xq, xk, *gam, *plain, **kw)
    for a, b in zip(saved, plain):
        assert torch.equal(a, b)


@pytest.mark.parametrize("dim, rot", [(128, 128), (33, 18)])      # vectors, one element at a time
def test_strides_that_pass_32_bits(tb, dim, rot):
    """A cache's rows 2^31 elements and more apart, in every dimension."""
    far = (1 << 31) + 256
    buf = torch.empty(far + 4096, dtype=BF, device="cuda")
    turns, freqs = ref.frequencies(rot)
    for shape, strides in (((2, 3, 2, dim), (far, 2 * dim, dim)), ((3, 2, 2, dim), (2 * dim, far, dim)),
                           ((2, 3, 2, dim), (3 * dim, dim, far))):
        x = torch.as_strided(buf, shape, (*strides, 1))
        x.copy_(torch.randn(shape, device="cuda"))
        want = x.clone()
        pos = torch.randint(0, 1000, shape[:2], device="cuda")
        angle = ref.angles(pos, turns)
        y = torch.empty_like(want)
        tb.tb_rope(x, None, y, None, freqs, positions=pos)                  # from far rows
        ref.check(y, ref.rotate(want.double(), angle, rot, False), ref.pair_sums(want.double(), rot, False) * ref.SIN)
        tb.tb_rope(want, None, x, None, freqs, positions=pos)               # to far rows
        assert torch.equal(x, y)
        inv = torch.empty(shape[:3], device="cuda")
        g = torch.ones(dim, device="cuda")
        tb.tb_qk_norm_rope(x, None, g, None, x, None, inv, freqs=freqs, positions=pos)
        dx, dg = torch.empty_like(y), torch.empty(dim, device="cuda")
        ws = torch.empty(tb.tb_qk_norm_rope_bwd_workspace_size(*shape[:3], 0, dim, BF), dtype=torch.uint8, device="cuda")
        z = torch.empty_like(y)
        tb.tb_qk_norm_rope(y, None, g, None, z, None, freqs=freqs, positions=pos)
        assert torch.equal(x, z)
        tb.tb_qk_norm_rope_bwd(z, None, y, None, inv, None, g, None, dx, None, dg, None, freqs=freqs, positions=pos,
                               workspace=ws)
        tb.tb_qk_norm_rope_bwd(x, None, y, None, inv, None, g, None, x, None, dg, None, freqs=freqs, positions=pos,
                               workspace=ws)
        assert torch.equal(x, dx)
