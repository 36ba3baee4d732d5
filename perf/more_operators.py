"""Cases, plain forms and framework calls of the two blocks of a decoder layer between its norms:
causal attention over whole prompts, with grouped heads and packed sequences, and the gated
feed-forward projections with their activation.  Each has its gradient.

A case is a dict of plain values; ``prepare`` makes its inputs on the GPU, ``run`` makes one
call of the operator (in elementary torch operations, or through ln_backward_gb300 where
``own`` is set), ``exact`` gives the outputs in 64 bits, and ``work`` the bytes and operations
one call cannot do without.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


# ----------------------------------------------------------------------------- cases
def _attention(op, dtype, lens, hq, hk, dim, layout, name=None):
    """lens: one sequence length for each batch entry ("4x4096"), or those of packed sequences ("97,1,300")."""
    c = dict(op=op, dtype=dtype, lens=lens, heads_q=hq, heads_k=hk, head_dim=dim, layout=layout)
    if name:
        c["name"] = name
    return c


def _gated(op, dtype, rows, hidden, inner, act, name=None):
    c = dict(op=op, dtype=dtype, rows=rows, hidden=hidden, inner=inner, act=act)
    if name:
        c["name"] = name
    return c


PACKED = "2047,1,513,1290,64,129,1733,300,7,1408,700"     # 8,192 tokens


def listed():
    return [
        # one short prompt, as it is answered: latency
        _attention("attn", "bf16", "97", 32, 8, 128, "qkv", "attn short prompt bf16"),
        # a training batch of a 7B decoder: 32 heads of 128, q, k, v views of one projection's output
        _attention("attn", "bf16", "4x4096", 32, 32, 128, "qkv", "attn train bf16"),
        # sequences of any length packed into one row of 8,192 tokens, grouped heads
        _attention("attn", "bf16", PACKED, 32, 8, 128, "qkv", "attn packed bf16"),
        # one long prompt, few heads of 64, heads before positions
        _attention("attn", "fp16", "1x16384", 8, 2, 64, "bhsd", "attn long fp16"),
        # the gradient of the training batch
        _attention("attn_bwd", "bf16", "4x4096", 32, 32, 128, "qkv", "attn bwd train bf16"),
        # the gradient of the packed row
        _attention("attn_bwd", "bf16", PACKED, 32, 8, 128, "qkv", "attn bwd packed bf16"),
        # GPT-2 small's heads at an odd length, fp16
        _attention("attn_bwd", "fp16", "5x777", 12, 12, 64, "bhsd", "attn bwd odd fp16"),
        # serving: one token for each of 16 requests, 7B decoder
        _gated("gated", "bf16", 16, 4096, 11008, "silu", "gated few rows bf16"),
        # training: what the gradient needs is kept
        _gated("gated_train", "bf16", 8192, 4096, 11008, "silu", "gated train bf16"),
        # a small model at a ragged number of rows
        _gated("gated_train", "fp16", 1021, 768, 2048, "gelu_tanh", "gated train ragged fp16"),
        # the gradients with respect to the inputs and both weights
        _gated("gated_bwd", "bf16", 8192, 4096, 11008, "silu", "gated bwd train bf16"),
        _gated("gated_bwd", "fp16", 1021, 768, 2048, "gelu_tanh", "gated bwd ragged fp16"),
    ]


def _spread(rng, lo, hi):
    """A whole number between lo and hi, spread over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["attn", "attn", "attn_bwd", "attn_bwd", "gated", "gated_train", "gated_bwd"])
    dtype = rng.choice(["bf16", "bf16", "fp16"])
    if op.startswith("gated"):
        hidden = 8 * _spread(rng, 8, 512)
        inner = 8 * _spread(rng, 8, 1376)
        rows = _spread(rng, 1, 256) if op == "gated" else _spread(rng, 17, 8192)
        return _gated(op, dtype, rows, hidden, inner, rng.choice(["silu", "silu", "gelu", "gelu_tanh"]))
    dim = rng.choice([64, 80, 96, 128, 128, 128, 8 * rng.randint(2, 16)])
    hk = rng.choice([1, 2, 4, 8])
    hq = min(32, hk * rng.choice([1, 2, 4, 8]))
    if rng.random() < 0.4:
        seq = _spread(rng, 1, 8192)
        batch = max(1, min(_spread(rng, 1, 16), 32 * 8192 * 8192 // (hq * seq * seq)))
        return _attention(op, dtype, "%dx%d" % (batch, seq), hq, hk, dim, rng.choice(["qkv", "bshd", "bhsd"]))
    lens, room = [], min(8192, int(8192 * math.sqrt(32 / hq)))
    for _ in range(_spread(rng, 1, 48)):
        n = _spread(rng, 1, 4096)
        if sum(lens) + n > room:
            break
        lens.append(n)
    return _attention(op, dtype, ",".join(map(str, lens)), hq, hk, dim, rng.choice(["qkv", "bshd"]))


def _lens(case):
    """(batch, seq, lengths of the sequences, whether they are packed into one row)."""
    if "x" in case["lens"]:
        b, s = map(int, case["lens"].split("x"))
        return b, s, [s] * b, False
    lens = [int(n) for n in case["lens"].split(",")]
    return 1, sum(lens), lens, True


# ----------------------------------------------------------------------------- inputs
def _views(case, make, kinds):
    """Queries, keys and values ("qkv") or one of them, [batch, seq, heads, head_dim] in the case's layout."""
    b, s, _, _ = _lens(case)
    hq, hk, d = case["heads_q"], case["heads_k"], case["head_dim"]
    if case["layout"] == "qkv" and kinds == "qkv":   # one projection's output
        buf = make((b, s, hq + 2 * hk, d))
        return buf[:, :, :hq], buf[:, :, hq:hq + hk], buf[:, :, hq + hk:]
    heads = [hq if kind == "q" else hk for kind in kinds]
    if case["layout"] == "bhsd":
        return tuple(make((b, h, s, d)).transpose(1, 2) for h in heads)
    return tuple(make((b, s, h, d)) for h in heads)


def prepare(case, seed):
    dt = DTYPES[case["dtype"]]
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) * 7919 + 29)

    def normal(shape, std=1.0):
        return torch.empty(shape, dtype=torch.float32, device="cuda").normal_(0.0, std, generator=g).to(dt)

    def empty(shape, dtype=dt):
        return torch.empty(shape, dtype=dtype, device="cuda")

    # fp16 trains with a loss scale
    small = 0.25 if dt == torch.float16 else 1e-3
    st = dict(case)
    if case["op"].startswith("gated"):
        n, d, f = case["rows"], case["hidden"], case["inner"]
        st["X"] = normal((n, d))
        st["Wg"], st["Wu"] = normal((f, d), 1.0 / math.sqrt(d)), normal((f, d), 1.0 / math.sqrt(d))
        if case["op"] == "gated_bwd":
            X = st["X"].float()
            st["G"], st["U"] = ((X @ st[w].float().t()).to(dt) for w in ("Wg", "Wu"))
            st["dH"] = normal((n, f), small)
            st["dX"], st["dWg"], st["dWu"] = empty((n, d)), empty((f, d)), empty((f, d))
        else:
            st["H"] = empty((n, f))
            if case["op"] == "gated_train":
                st["G"], st["U"] = empty((n, f)), empty((n, f))
        return st

    b, s, lens, packed = _lens(case)
    st["q"], st["k"], st["v"] = _views(case, normal, "qkv")
    st["scale"] = 1.5 / math.sqrt(case["head_dim"])
    st["offsets"] = torch.tensor([0] + lens).cumsum(0).to("cuda") if packed else None
    st["out"], = _views(case, empty, "q")
    st["lse"] = empty((b, case["heads_q"], s), torch.float32)
    if case["op"] == "attn_bwd":
        # what the forward left
        saved = _plain_attention(st)
        st["out"].copy_(saved["out"])
        st["lse"].copy_(saved["lse"])
        del saved
        st["dout"], = _views(case, lambda shape: normal(shape, small), "q")
        st["dq"], st["dk"], st["dv"] = _views(case, empty, "qkv")
    return st


# ----------------------------------------------------------------------------- plain forms
def _act(x, act):
    """The activation and its slope."""
    if act == "silu":
        s = 1.0 / (1.0 + (-x).exp())
        return x * s, s * (1.0 + x * (1.0 - s))
    if act == "gelu":
        c = 0.5 * (1.0 + torch.erf(x * math.sqrt(0.5)))
        return x * c, c + x * (-0.5 * x * x).exp() / math.sqrt(2 * math.pi)
    r = math.sqrt(2 / math.pi)
    t = (r * (x + 0.044715 * x * x * x)).tanh()
    return 0.5 * x * (1.0 + t), 0.5 * (1.0 + t) + 0.5 * x * (1.0 - t * t) * r * (1.0 + 3 * 0.044715 * x * x)


def _plain_gated(st):
    dt = st["X"].dtype
    X, Wg, Wu = st["X"].float(), st["Wg"].float(), st["Wu"].float()
    if st["op"] != "gated_bwd":
        G, U = X @ Wg.t(), X @ Wu.t()
        H = (_act(G, st["act"])[0] * U).to(dt)
        return {"H": H} if st["op"] == "gated" else {"H": H, "G": G.to(dt), "U": U.to(dt)}
    dH, U = st["dH"].float(), st["U"].float()
    a, slope = _act(st["G"].float(), st["act"])
    dG, dU = dH * U * slope, dH * a
    return {"dX": (dG @ Wg + dU @ Wu).to(dt), "dWg": (dG.t() @ X).to(dt), "dWu": (dU.t() @ X).to(dt)}


def _plain_open(st, s):
    """[seq, seq]: whether query i reads key j."""
    at = torch.arange(s, device="cuda")
    seen = at[None, :] <= at[:, None]
    if st["offsets"] is not None:
        of = torch.searchsorted(st["offsets"], at, right=True)
        seen &= of[None, :] == of[:, None]
    return seen


def _plain_heads(st, x):
    """[batch, heads_q, seq, head_dim] in 32 bits, key heads repeated for their queries."""
    x = x.float().transpose(1, 2)
    return x.repeat_interleave(st["heads_q"] // x.shape[1], 1)


def _plain_attention(st):
    q, k, v = (_plain_heads(st, st[n]) for n in "qkv")
    scores = (q @ k.transpose(2, 3)).mul_(st["scale"])
    scores.masked_fill_(~_plain_open(st, q.shape[2]), -math.inf)
    top = scores.max(-1, keepdim=True).values
    p = scores.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    out = (p @ v) / total
    return {"out": out.transpose(1, 2).to(st["q"].dtype), "lse": (top + total.log())[..., 0]}


def _plain_attention_bwd(st):
    dt, group = st["q"].dtype, st["heads_q"] // st["heads_k"]
    q, k, v, dout, out = (_plain_heads(st, st[n]) for n in ("q", "k", "v", "dout", "out"))
    p = (q @ k.transpose(2, 3)).mul_(st["scale"]).sub_(st["lse"][..., None]).exp_()
    p.masked_fill_(~_plain_open(st, q.shape[2]), 0.0)
    dv = p.transpose(2, 3) @ dout
    ds = (dout @ v.transpose(2, 3)).sub_((dout * out).sum(-1, keepdim=True)).mul_(p).mul_(st["scale"])
    dq, dk = ds @ k, ds.transpose(2, 3) @ q
    dk, dv = (x.unflatten(1, (-1, group)).sum(2) for x in (dk, dv))
    return {n: x.transpose(1, 2).to(dt) for n, x in (("dq", dq), ("dk", dk), ("dv", dv))}


# ----------------------------------------------------------------------------- the framework's calls
def _scratch(st, nbytes):
    """A workspace that the caller keeps from one call to the next."""
    ws = st.get("ws")
    if ws is None:
        ws = st["ws"] = torch.empty(nbytes(), dtype=torch.uint8, device="cuda")
    return ws


def _own_run(st):
    import ln_backward_gb300 as tb
    op = st["op"]
    if op == "attn":
        tb.tb_attention(st["q"], st["k"], st["v"], st["out"], st["lse"], scale=st["scale"], offsets=st["offsets"])
        return {"out": st["out"], "lse": st["lse"]}
    if op == "attn_bwd":
        q, k = st["q"], st["k"]
        ws = _scratch(st, lambda: tb.tb_attention_bwd_workspace_size(
            q.shape[0], q.shape[1], q.shape[2], k.shape[2], q.shape[3], q.dtype))
        tb.tb_attention_bwd(st["dout"], q, k, st["v"], st["out"], st["lse"], st["dq"], st["dk"], st["dv"], ws,
                            scale=st["scale"], offsets=st["offsets"])
        return {"dq": st["dq"], "dk": st["dk"], "dv": st["dv"]}
    X, Wg, Wu = st["X"], st["Wg"], st["Wu"]
    sizes = (*X.shape, Wg.shape[0], X.dtype)
    if op == "gated_bwd":
        ws = _scratch(st, lambda: tb.tb_gated_linear_bwd_workspace_size(*sizes))
        tb.tb_gated_linear_bwd(st["dH"], X, Wg, Wu, st["G"], st["U"], st["dX"], st["dWg"], st["dWu"], ws,
                               activation=st["act"])
        return {"dX": st["dX"], "dWg": st["dWg"], "dWu": st["dWu"]}
    ws = _scratch(st, lambda: tb.tb_gated_linear_workspace_size(*sizes))
    if op == "gated":
        tb.tb_gated_linear(X, Wg, Wu, st["H"], workspace=ws, activation=st["act"])
        return {"H": st["H"]}
    tb.tb_gated_linear(X, Wg, Wu, st["H"], st["G"], st["U"], workspace=ws, activation=st["act"])
    return {"H": st["H"], "G": st["G"], "U": st["U"]}


def run(state):
    if own:
        return _own_run(state)
    if state["op"].startswith("gated"):
        return _plain_gated(state)
    return _plain_attention(state) if state["op"] == "attn" else _plain_attention_bwd(state)


# ----------------------------------------------------------------------------- what a call cannot do without
def work(case):
    if case["op"].startswith("gated"):
        n, d, f = case["rows"], case["hidden"], case["inner"]
        if case["op"] == "gated_bwd":
            # one product for each of the three results; dX has two halves of the contraction
            return {"bytes": 2 * (3 * n * f + 2 * n * d + 4 * f * d), "flops": 8 * n * d * f}
        kept = 2 * n * f if case["op"] == "gated_train" else 0
        return {"bytes": 2 * (n * d + 2 * f * d + n * f + kept), "flops": 4 * n * d * f}
    b, s, lens, _ = _lens(case)
    hq, hk, d = case["heads_q"], case["heads_k"], case["head_dim"]
    pairs = hq * sum(n * (n + 1) // 2 for n in lens)
    qs, ks = 2 * b * s * hq * d, 2 * b * s * hk * d
    if case["op"] == "attn":
        return {"bytes": 2 * qs + 2 * ks + 4 * b * s * hq, "flops": 4 * pairs * d}
    # scores and dP again (they are not kept), dV, dK, dQ
    return {"bytes": 4 * qs + 4 * ks + 4 * b * s * hq, "flops": 10 * pairs * d}


# ----------------------------------------------------------------------------- 64 bits
def _exact_gated(case, st):
    if work(case)["flops"] > 8e12:   # about 10 seconds of 64-bit products
        return None
    X, Wg, Wu = (st[n].double() for n in ("X", "Wg", "Wu"))
    kind = {"silu": torch.nn.functional.silu, "gelu": torch.nn.functional.gelu,
            "gelu_tanh": lambda x: torch.nn.functional.gelu(x, approximate="tanh")}[case["act"]]
    if case["op"] != "gated_bwd":
        G, U = torch.einsum("nd,fd->nf", X, Wg), torch.einsum("nd,fd->nf", X, Wu)
        H = kind(G) * U
        return {"H": H} if case["op"] == "gated" else {"H": H, "G": G, "U": U}
    # the gradient of the product by autograd, the projections' transposes behind it
    G, U = (st[n].double().requires_grad_() for n in "GU")
    dG, dU = torch.autograd.grad(kind(G) * U, (G, U), st["dH"].double())
    return {"dX": torch.einsum("nf,fd->nd", dG, Wg) + torch.einsum("nf,fd->nd", dU, Wu),
            "dWg": torch.einsum("nf,nd->fd", dG, X), "dWu": torch.einsum("nf,nd->fd", dU, X)}


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"].startswith("gated"):
        return _exact_gated(case, st)
    if work(case)["flops"] > 8e12:
        return None
    b, s, lens, packed = _lens(case)
    group, scale = case["heads_q"] // case["heads_k"], st["scale"]
    res = {n: torch.zeros(st[n].shape, dtype=torch.float64, device="cuda")
           for n in (("out", "lse") if case["op"] == "attn" else ("dq", "dk", "dv"))}
    start = 0
    for i, n in enumerate(lens):
        row, span = (0, slice(start, start + n)) if packed else (i, slice(0, n))
        start += n
        hidden = torch.ones(n, n, dtype=torch.bool, device="cuda").triu(1)
        for h in range(case["heads_k"]):
            mine = slice(h * group, (h + 1) * group)
            q, k, v = st["q"][row, span, mine].double(), st["k"][row, span, h].double(), st["v"][row, span, h].double()
            logits = torch.einsum("ihd,jd->hij", q, k) * scale
            logits[:, hidden] = -math.inf
            if case["op"] == "attn":
                res["out"][row, span, mine] = torch.einsum("hij,jd->ihd", torch.softmax(logits, -1), v)
                res["lse"][row, mine, span] = torch.logsumexp(logits, -1)
                continue
            up, o = st["dout"][row, span, mine].double(), st["out"][row, span, mine].double()
            p = torch.exp(logits - st["lse"][row, mine, span, None].double())
            res["dv"][row, span, h] = torch.einsum("hij,ihd->jd", p, up)
            p *= torch.einsum("ihd,jd->hij", up, v) - torch.einsum("ihd,ihd->hi", up, o)[..., None]
            res["dq"][row, span, mine] = torch.einsum("hij,jd->ihd", p, k) * scale
            res["dk"][row, span, h] = torch.einsum("hij,ihd->jd", p, q) * scale
    return res
