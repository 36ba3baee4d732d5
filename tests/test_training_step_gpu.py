"""The operators of one decoder layer's training step together, as a training loop calls them:
queries and keys normed and rotated (tb_qk_norm_rope), causal attention, the output layer's loss
(tb_linear_xent), and back: tb_linear_xent_bwd, tb_softmax_bwd_causal, tb_qk_norm_rope_bwd, then
AdamW on the gradients. Products that the library leaves to others are torch's, in fp32."""
import pytest
import torch

import rope_reference as ref

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.fixture(scope="module")
def tb():
    import ln_backward_gb300
    return ln_backward_gb300


def attention_inputs(seed):
    """One layer's joint projection output, gammas, output weights and targets."""
    b, s, h, hk, d, v = 2, 64, 4, 2, 64, 1000
    g = torch.Generator(device="cuda").manual_seed(seed)
    qkv = torch.randn(b, s, h + 2 * hk, d, generator=g, device="cuda").to(BF)
    gq, gk = (1 + 0.1 * torch.randn(d, generator=g, device="cuda") for _ in range(2))
    W = (0.2 * torch.randn(v, h * d, generator=g, device="cuda")).to(BF)
    t = torch.randint(0, v, (b * s,), generator=g, device="cuda")
    t[torch.rand(b * s, generator=g, device="cuda") < 0.2] = -100
    return (b, s, h, hk, d, v), qkv, gq, gk, W, t


def forward64(dims, qkv, gq, gk, W, t, angle):
    """The mean loss in 64 bits, differentiable."""
    b, s, h, hk, d, v = dims
    q, _ = ref.normed(qkv[:, :, :h], gq, 1e-6)
    k, _ = ref.normed(qkv[:, :, h:h + hk], gk, 1e-6)
    q, k = (ref.rotate(x, angle, d, False) for x in (q, k))
    k, val = (x.repeat_interleave(h // hk, 2) for x in (k, qkv[:, :, h + hk:]))
    score = torch.einsum("bshd,bthd->bhst", q, k) * d ** -0.5
    score = score.masked_fill(torch.ones(s, s, dtype=torch.bool, device="cuda").triu(1), -torch.inf)
    out = torch.einsum("bhst,bthd->bshd", score.softmax(-1), val).reshape(b * s, h * d)
    logits = out @ W.T
    keep = t != -100
    loss = torch.logsumexp(logits, -1) - logits.gather(1, torch.where(keep, t, 0)[:, None])[:, 0]
    return (loss * keep).sum() / keep.sum()


def step(tb, dims, qkv, gq, gk, W, t, freqs, positions):
    """Loss and gradients with the library's operators."""
    b, s, h, hk, d, v = dims
    rep = h // hk
    q, k, val = qkv[:, :, :h], qkv[:, :, h:h + hk], qkv[:, :, h + hk:]
    yq, yk = torch.empty(b, h, s, d, device="cuda", dtype=BF), torch.empty(b, hk, s, d, device="cuda", dtype=BF)
    inv = [torch.empty(b, s, n, device="cuda") for n in (h, hk)]
    kw = dict(freqs=freqs, positions=positions)
    tb.tb_qk_norm_rope(q, k, gq, gk, yq.transpose(1, 2), yk.transpose(1, 2), *inv, eps=1e-6, **kw)
    kr, vr = yk.repeat_interleave(rep, 1).float(), val.transpose(1, 2).repeat_interleave(rep, 1).float()
    score = (yq.float() @ kr.transpose(-1, -2)) * d ** -0.5
    score.masked_fill_(torch.ones(s, s, dtype=torch.bool, device="cuda").triu(1), -torch.inf)
    P = score.softmax(-1)
    H = (P @ vr).transpose(1, 2).reshape(b * s, h * d).to(BF)

    n = (t != -100).sum()
    loss, lse = torch.empty(b * s, device="cuda"), torch.empty(b * s, device="cuda")
    ws = torch.empty(tb.tb_linear_xent_workspace_size(b * s, h * d, v, BF), dtype=torch.uint8, device="cuda")
    tb.tb_linear_xent(H, W, t, loss, lse, ws)
    dloss = torch.ones(b * s, device="cuda") / n
    dH, dW = torch.empty_like(H), torch.empty_like(W)
    ws = torch.empty(tb.tb_linear_xent_bwd_workspace_size(b * s, h * d, v, BF), dtype=torch.uint8, device="cuda")
    tb.tb_linear_xent_bwd(dloss, H, W, t, lse, dH, dW, ws)

    dO = dH.float().view(b, s, h, d).transpose(1, 2)
    dP = (dO @ vr.transpose(-1, -2)).reshape(b * h * s, s)
    dS = torch.empty_like(dP)
    tb.tb_softmax_bwd_causal(dP, P.reshape(b * h * s, s), dS, period=s)
    dS = dS.view(b, h, s, s) * d ** -0.5
    dq_out = (dS @ kr).to(BF)
    dk_out = (dS.transpose(-1, -2) @ yq.float()).view(b, hk, rep, s, d).sum(2).to(BF)
    dqkv = torch.empty_like(qkv)
    dqkv[:, :, h + hk:] = (P.transpose(-1, -2) @ dO).view(b, hk, rep, s, d).sum(2).transpose(1, 2)
    dg = [torch.empty(d, device="cuda") for _ in range(2)]
    ws = torch.empty(tb.tb_qk_norm_rope_bwd_workspace_size(b, s, h, hk, d, BF), dtype=torch.uint8, device="cuda")
    tb.tb_qk_norm_rope_bwd(dq_out.transpose(1, 2), dk_out.transpose(1, 2), q, k, *inv, gq, gk, dqkv[:, :, :h],
                           dqkv[:, :, h:h + hk], *dg, workspace=ws, **kw)
    return loss.sum() / n, {"qkv": dqkv, "gq": dg[0], "gk": dg[1], "W": dW}


def test_gradients_of_a_decoder_layer(tb):
    dims, qkv, gq, gk, W, t = attention_inputs(0)
    b, s, h, hk, d, v = dims
    turns, freqs = ref.frequencies(d)
    positions = torch.arange(s, device="cuda").expand(b, s).contiguous()
    loss, grads = step(tb, dims, qkv, gq, gk, W, t, freqs, positions)
    leaves = {"qkv": qkv, "gq": gq, "gk": gk, "W": W}
    x64 = {n: x.double().requires_grad_() for n, x in leaves.items()}
    want = forward64(dims, x64["qkv"], x64["gq"], x64["gk"], x64["W"], t, ref.angles(positions, turns))
    want.backward()
    # H's rounding to bf16 (half a step: 2^-9 of it at most) moves a logit by 2^-9 of its terms
    assert abs(loss.item() - want.item()) <= 2.0 ** -9 * abs(want.item())
    for n, g in grads.items():
        # q, k, H, G, dH, dq_out or dk_out, the result: at most seven roundings of 2^-9 on the way,
        # doubled once for the softmax's p (dp = p dl, with l's error twice that of q or k)
        off = (g.double() - x64[n].grad).norm() / x64[n].grad.norm()
        assert off <= 14 * 2.0 ** -9, f"{n}: {off:.4f}"


def test_the_optimizer_takes_the_gradients(tb):
    """AdamW over the output weights and the gammas, with the step's own gradient buffers."""
    dims, qkv, gq, gk, W, t = attention_inputs(1)
    b, s, h, hk, d, v = dims
    _, freqs = ref.frequencies(d)
    positions = torch.arange(s, device="cuda").expand(b, s).contiguous()
    master = W.float()
    m, mv = torch.zeros_like(master), torch.zeros_like(master)
    _, grads = step(tb, dims, qkv, gq, gk, W, t, freqs, positions)
    g64 = grads["W"].double()
    plan = tb.tb_adamw_plan_create([master], [m], [mv], [grads["W"]], [W])
    hp = dict(lr=1e-2, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.0)
    before = master.double()
    tb.tb_adamw_step(plan, 1, **hp, inv_loss_scale=1.0)
    # the first step: m_hat = g, v_hat = g^2, each formed with a few fp32 roundings
    want = before - 1e-2 * g64 / (g64.abs() + 1e-8)
    assert ((master.double() - want).abs() <= 2.0 ** -18 * 1e-2 + 2.0 ** -23 * before.abs()).all()
    assert not grads["W"].any() and torch.equal(W, master.to(BF))
    loss, grads = step(tb, dims, qkv, gq, gk, W, t, freqs, positions)      # and the next step runs
    assert torch.isfinite(loss) and grads["W"].isfinite().all()
