"""How attention and the gated projections are used: on other streams, in captured graphs, with workspaces of any
content and no byte more than asked for, beside memory that is not theirs, and together as a decoder layer's
training step."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.fixture(scope="module")
def tb():
    import ln_backward_gb300
    return ln_backward_gb300


class Attention:
    """One attention layer's forward and gradient over fixed buffers."""

    def __init__(self, tb, offsets=None, dtype=BF, d=64, tokens=700, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        make = lambda h: torch.randn(1, tokens, h, d, generator=g, device="cuda").to(dtype)
        self.tb, self.q, self.k, self.v, self.dout = tb, make(4), make(2), make(2), make(4)
        self.out, self.lse = torch.zeros_like(self.q), torch.zeros(1, 4, tokens, device="cuda")
        self.grads = [torch.zeros_like(x) for x in (self.q, self.k, self.v)]
        self.offsets = torch.tensor(offsets or [0, 333, 600], device="cuda")
        self.ws = torch.full((tb.tb_attention_bwd_workspace_size(1, tokens, 4, 2, d, dtype),), 0x55, dtype=torch.uint8, device="cuda")
        self.inputs, self.results = [self.q, self.k, self.v, self.dout], [self.out, self.lse, *self.grads]

    def __call__(self, stream=None):
        self.tb.tb_attention(self.q, self.k, self.v, self.out, self.lse, offsets=self.offsets, stream=stream)
        self.tb.tb_attention_bwd(self.dout, self.q, self.k, self.v, self.out, self.lse, *self.grads, self.ws, offsets=self.offsets,
                                 stream=stream)


class Gated:
    """The gated projections' forward and gradient over fixed buffers; few rows split the contraction."""

    def __init__(self, tb, dtype=BF, n=300, d=264, f=520, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        make = lambda *s: torch.randn(*s, generator=g, device="cuda").to(dtype)
        self.tb, self.X, self.Wg, self.Wu, self.dH = tb, make(n, d), make(f, d) / 16, make(f, d) / 16, make(n, f)
        self.H, self.G, self.U = (torch.zeros(n, f, dtype=dtype, device="cuda") for _ in range(3))
        self.grads = [torch.zeros_like(x) for x in (self.X, self.Wg, self.Wu)]
        size = max(tb.tb_gated_linear_workspace_size(n, d, f, dtype), tb.tb_gated_linear_bwd_workspace_size(n, d, f, dtype))
        self.ws = torch.full((size,), 0x55, dtype=torch.uint8, device="cuda")
        self.inputs, self.results = [self.X, self.Wg, self.Wu, self.dH], [self.H, self.G, self.U, *self.grads]

    def __call__(self, stream=None):
        self.tb.tb_gated_linear(self.X, self.Wg, self.Wu, self.H, self.G, self.U, self.ws, stream=stream)
        self.tb.tb_gated_linear_bwd(self.dH, self.X, self.Wg, self.Wu, self.G, self.U, *self.grads, self.ws, stream=stream)


BOTH = [Attention, Gated, lambda tb, seed=0: Attention(tb, dtype=torch.float16, d=128, seed=seed),
        lambda tb, seed=0: Gated(tb, dtype=torch.float16, n=33, d=2048, f=64, seed=seed)]


def outcome(call):
    call()
    torch.cuda.synchronize()
    return [x.clone() for x in call.results]


@pytest.mark.parametrize("make", BOTH)
def test_other_streams(tb, make):
    want = outcome(make(tb, seed=1))
    calls = [make(tb, seed=1) for _ in range(2)]
    streams = [torch.cuda.Stream() for _ in calls]
    torch.cuda.synchronize()
    with torch.cuda.stream(streams[0]):
        calls[0]()                              # torch's current stream
    for _ in range(3):
        calls[1](streams[1])                    # a stream that is given, the same call again behind itself
    torch.cuda.synchronize()
    for c in calls:
        assert all(torch.equal(a, b) for a, b in zip(c.results, want))
    assert tb.tb_device_error() == 0


@pytest.mark.parametrize("make", BOTH)
def test_captured_and_replayed_on_new_inputs(tb, make):
    call, other = make(tb, seed=1), make(tb, seed=2)
    want = outcome(other)
    call()
    torch.cuda.synchronize()
    graphs = []
    for c in (call, make(tb, seed=3)):          # two graphs, each with its buffers
        s = torch.cuda.Stream()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            c()
        graphs.append((g, c))
    for x, y in zip(call.inputs, other.inputs):
        x.copy_(y)
    for _ in range(2):
        for g, _ in graphs:
            g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(call.results, want))
    assert all(torch.equal(a, b) for a, b in zip(graphs[1][1].results, outcome(make(tb, seed=3))))


def test_offsets_read_when_the_graph_runs(tb):
    call, other = Attention(tb), Attention(tb, offsets=[0, 1, 700])
    want = outcome(other)
    call()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    call.offsets.copy_(other.offsets)
    g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(call.results, want))


@pytest.mark.parametrize("make", BOTH)
def test_memory_around_results_and_workspaces(tb, make):
    """Every result and the workspace between guards in one allocation, the workspace of two contents."""
    call = make(tb, seed=4)
    want = outcome(call)
    room = 4096
    for fill in (0x00, 0xFF):
        held = []
        for x in [*call.results, call.ws]:
            n = x.numel() * x.element_size()
            mem = torch.full((n + 2 * room,), 0xA5, dtype=torch.uint8, device="cuda")
            mem[room:room + n] = fill
            held.append((mem, n, mem[room:room + n].view(x.dtype).view(x.shape)))
        views = [h[2] for h in held]
        if isinstance(call, Attention):
            call.out, call.lse, call.grads, call.ws = views[0], views[1], views[2:5], views[5]
            for v in views[:1] + views[2:5]:
                v[:, 600:] = 0                  # tokens of no sequence stay as they are
            views[1][..., 600:] = 0
        else:
            call.H, call.G, call.U, call.grads, call.ws = *views[:3], views[3:6], views[6]
        call()
        torch.cuda.synchronize()
        for (mem, n, _), v, w in zip(held, views, want):
            assert torch.equal(v, w)
        for mem, n, _ in held:
            assert (mem[:room] == 0xA5).all() and (mem[room + n:] == 0xA5).all()
    assert tb.tb_device_error() == 0


def test_workspaces_that_are_refused(tb):
    a, g = Attention(tb), Gated(tb)
    for call, ws in ((a, a.ws[:-1]), (g, g.ws[:-1]), (a, None), (g, None)):
        call.ws = ws
        with pytest.raises(tb.TbError) as e:
            call()
        assert e.value.code == 5
    torch.cuda.synchronize()


def test_far_offsets(tb):
    """Elements of a tensor further than 2^31 from its start."""
    tokens, d = 400, 64
    step = 8 * 1024 * 1024                     # elements from one token to the next: 6.7 GB of one buffer
    buf = torch.empty(tokens * step, dtype=BF, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(5)
    near = [torch.randn(1, tokens, h, d, generator=g, device="cuda").to(BF) for h in (2, 1, 1)]
    far, at = [], 0
    for x in near:
        h = x.shape[2]
        far.append(buf[at:].as_strided((1, tokens, h, d), (tokens * step, step, d, 1)))
        far[-1].copy_(x)
        at += h * d
    out = buf[at:].as_strided((1, tokens, 2, d), (tokens * step, step, d, 1))
    want, lse = torch.empty_like(near[0]), torch.empty(1, 2, tokens, device="cuda")
    tb.tb_attention(*near, want, lse)
    tb.tb_attention(*far, out)
    assert torch.equal(out, want)
    dout = torch.randn(1, tokens, 2, d, generator=g, device="cuda").to(BF)
    ws = torch.empty(tb.tb_attention_bwd_workspace_size(1, tokens, 2, 1, d, BF), dtype=torch.uint8, device="cuda")
    grads = [torch.empty_like(x) for x in near]
    tb.tb_attention_bwd(dout, *near, want, lse, *grads, ws)
    at += 2 * d
    far_grads = []
    for x in near:
        far_grads.append(buf[at:].as_strided(x.shape, (tokens * step, step, d, 1)))
        at += x.shape[2] * d
    tb.tb_attention_bwd(dout, *far, out, lse, *far_grads, ws)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(far_grads, grads))


def test_a_decoder_layer_trains(tb):
    """Norm and rotation of queries and keys, attention over packed sequences, the gated block and the output layer's
    loss, forward and backward, against the same layer in 64 bits.  Every operator rounds its results to bf16, a dozen
    one after another on the way to the first weights: each at most 2^-8 of a value, 12 * 2^-8 / 2 on average over values
    whose roundings have either sign."""
    n, d, heads, kv, dim, f, vocab = 300, 256, 4, 2, 64, 512, 1000
    g = torch.Generator(device="cuda").manual_seed(7)
    make = lambda *s, std=1.0: (torch.randn(*s, generator=g, device="cuda") * std).to(BF)
    x, w_qkv, w_o = make(n, d), make((heads + 2 * kv) * dim, d, std=d ** -0.5), make(d, heads * dim, std=0.06)
    wg, wu, wd, w_out = make(f, d, std=d ** -0.5), make(f, d, std=d ** -0.5), make(d, f, std=0.04), make(vocab, d, std=0.06)
    target = torch.randint(0, vocab, (n,), generator=g, device="cuda")
    offsets = torch.tensor([0, 130, 131, n], device="cuda")
    pos = torch.cat([torch.arange(b - a) for a, b in ((0, 130), (130, 131), (131, n))]).cuda()[None]
    freqs, _ = tb.tb_rope_freqs(dim)
    gam = [1 + 0.1 * torch.randn(dim, generator=g, device="cuda") for _ in range(2)]
    split = lambda t: t.view(1, n, heads + 2 * kv, dim).split((heads, kv, kv), 2)
    scratch = lambda size: torch.empty(size, dtype=torch.uint8, device="cuda")

    # forward
    qkv = x @ w_qkv.T
    q, k, v = split(qkv)
    rot = torch.empty_like(qkv)
    rq, rk, _ = split(rot)
    inv = [torch.empty(1, n, h, device="cuda") for h in (heads, kv)]
    tb.tb_qk_norm_rope(q, k, *gam, rq, rk, *inv, freqs=freqs, positions=pos)
    att, lse = torch.empty(1, n, heads, dim, dtype=BF, device="cuda"), torch.empty(1, heads, n, device="cuda")
    tb.tb_attention(rq, rk, v, att, lse, offsets=offsets)
    h1 = x + att.view(n, -1) @ w_o.T
    H, G, U = (torch.empty(n, f, dtype=BF, device="cuda") for _ in range(3))
    tb.tb_gated_linear(h1, wg, wu, H, G, U, scratch(tb.tb_gated_linear_workspace_size(n, d, f, BF)))
    h2 = h1 + H @ wd.T
    loss, lse2 = torch.empty(n, device="cuda"), torch.empty(n, device="cuda")
    tb.tb_linear_xent(h2, w_out, target, loss, lse2, scratch(tb.tb_linear_xent_workspace_size(n, d, vocab, BF)))
    # backward
    dh2, dw_out = torch.empty_like(h2), torch.empty_like(w_out)
    tb.tb_linear_xent_bwd(torch.full((n,), 1.0 / n, device="cuda"), h2, w_out, target, lse2, dh2, dw_out,
                          scratch(tb.tb_linear_xent_bwd_workspace_size(n, d, vocab, BF)))
    dH, dwd = dh2 @ wd, dh2.T @ H
    dh1, dwg, dwu = torch.empty_like(h1), torch.empty_like(wg), torch.empty_like(wu)
    tb.tb_gated_linear_bwd(dH, h1, wg, wu, G, U, dh1, dwg, dwu, scratch(tb.tb_gated_linear_bwd_workspace_size(n, d, f, BF)))
    dh1 = dh1 + dh2
    datt, dw_o = (dh1 @ w_o).view(1, n, heads, dim), dh1.T @ att.view(n, -1)
    drot, dqkv, dgam = torch.empty_like(qkv), torch.empty_like(qkv), [torch.empty(dim, device="cuda") for _ in range(2)]
    drq, drk, _ = split(drot)
    dq, dk, dv = split(dqkv)
    tb.tb_attention_bwd(datt, rq, rk, v, att, lse, drq, drk, dv, scratch(tb.tb_attention_bwd_workspace_size(1, n, heads, kv, dim, BF)),
                        offsets=offsets)
    tb.tb_qk_norm_rope_bwd(drq, drk, q, k, *inv, *gam, dq, dk, *dgam, freqs=freqs, positions=pos,
                           workspace=scratch(tb.tb_qk_norm_rope_bwd_workspace_size(1, n, heads, kv, dim, BF)))
    dw_qkv, dx = dqkv.T @ x, dqkv @ w_qkv + dh1
    assert tb.tb_device_error() == 0

    # the same in 64 bits, by autograd
    leaves = [t.double().requires_grad_() for t in (x, w_qkv, w_o, wg, wu, wd, w_out, *gam)]
    X, Wqkv, Wo, Wg, Wu, Wd, Wout, gq, gk = leaves
    a, b, c = split(X @ Wqkv.T)
    w = 10000.0 ** (-2.0 * torch.arange(dim // 2, dtype=torch.float64, device="cuda") / dim)
    angle = pos.double()[0, :, None, None] * w

    def turned(t, gamma):
        t = t[0] * (t[0].square().mean(-1, keepdim=True) + 1e-6).rsqrt() * gamma
        lo, hi = t[..., :dim // 2], t[..., dim // 2:]
        return torch.cat((lo * angle.cos() - hi * angle.sin(), lo * angle.sin() + hi * angle.cos()), -1)

    a, b, c = turned(a, gq), turned(b, gk).repeat_interleave(heads // kv, 1), c[0].repeat_interleave(heads // kv, 1)
    of = torch.searchsorted(offsets, torch.arange(n, device="cuda"), right=True)
    seen = torch.ones(n, n, dtype=torch.bool, device="cuda").tril() & (of[:, None] == of[None])
    scores = torch.einsum("ihd,jhd->hij", a, b) * dim ** -0.5
    o = torch.einsum("hij,jhd->ihd", scores.masked_fill(~seen, -math.inf).softmax(-1), c)
    h = X + o.reshape(n, -1) @ Wo.T
    h = h + (torch.nn.functional.silu(h @ Wg.T) * (h @ Wu.T)) @ Wd.T
    want = torch.nn.functional.cross_entropy(h @ Wout.T, target)
    want.backward()
    assert abs(loss.mean().item() - want.item()) <= 2.0 ** -8 * want.item()
    for name, got, leaf in zip(("x", "w_qkv", "w_o", "wg", "wu", "wd", "w_out", "gamma_q", "gamma_k"),
                               (dx, dw_qkv, dw_o, dwg, dwu, dwd, dw_out, *dgam), leaves):
        off = (got.double() - leaf.grad).norm() / leaf.grad.norm()
        assert off <= 12 * 2.0 ** -9, f"{name}: {off.item()}"
