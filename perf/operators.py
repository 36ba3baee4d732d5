"""Cases, plain forms and framework calls of the operators around attention's queries and keys
and of the loss at a decoder's output: rotary positions, the per-head RMS norm of queries and
keys with the rotation in the same pass, and the softmax cross entropy of a linear output layer
over a large vocabulary.  Each has its gradient.

A case is a dict of plain values; ``prepare`` makes its inputs on the GPU, ``run`` makes one
call of the operator (in elementary torch operations, or through ln_backward_gb300 where
``own`` is set), ``exact`` gives the outputs in 64 bits, and ``work`` the bytes and operations
one call cannot do without.
"""
import math

import torch

own = False

DTYPES = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}
TURN = 2 * math.pi
IGNORE = -100


# ----------------------------------------------------------------------------- cases
def _heads(op, dtype, batch, seq, hq, hk, dim, rot, interleaved, layout, far, stretch, name=None):
    c = dict(op=op, dtype=dtype, batch=batch, seq=seq, heads_q=hq, heads_k=hk, head_dim=dim,
             rotary_dim=rot, interleaved=interleaved, layout=layout, far=far, stretch=stretch)
    if name:
        c["name"] = name
    return c


def _loss(op, dtype, rows, vocab, hidden, name=None):
    c = dict(op=op, dtype=dtype, rows=rows, vocab=vocab, hidden=hidden)
    if name:
        c["name"] = name
    return c


def listed():
    return [
        # one new token for each of 32 requests, whose contexts have any length up to 131,072;
        # q and k are views of the fused projection's output
        _heads("rope", "bf16", 32, 1, 32, 8, 128, 128, False, "qkv", 131072, 1.0, "rope decode bf16"),
        # a training batch of a 7B decoder: 32 heads of 128
        _heads("rope", "bf16", 4, 4096, 32, 32, 128, 128, False, "qkv", 0, 1.0, "rope train bf16"),
        # gradient with adjacent pairs, part of an unusual head, heads before positions, fp32
        _heads("rope_bwd", "fp32", 3, 1023, 16, 4, 80, 32, True, "bhsd", 0, 4.0, "rope bwd partial fp32"),
        # serving: one token for each of 64 requests, positions far into a stretched context
        _heads("qk_norm", "bf16", 64, 1, 32, 8, 128, 128, False, "qkv", 131072, 8.0, "qk norm decode bf16"),
        # long-context training, grouped heads
        _heads("qk_norm_train", "bf16", 2, 8192, 32, 8, 128, 128, False, "qkv", 0, 1.0, "qk norm fwd bf16"),
        # its gradient, an ordinary batch
        _heads("qk_norm_bwd", "bf16", 4, 4096, 32, 8, 128, 128, False, "qkv", 0, 1.0, "qk norm bwd bf16"),
        # small heads, adjacent pairs on half of each, odd lengths
        _heads("qk_norm_bwd", "fp16", 5, 777, 12, 12, 64, 32, True, "bhsd", 0, 1.0, "qk norm bwd odd fp16"),
        # wide heads rotated in their first quarter, one long sequence, fp32
        _heads("qk_norm_bwd", "fp32", 1, 32768, 16, 2, 256, 64, False, "bshd", 0, 1.0, "qk norm bwd wide fp32"),
        # scoring a short text: few rows against the whole GPT-2 small vocabulary
        _loss("xent", "bf16", 37, 50257, 768, "loss few rows bf16"),
        # the loss of one training micro-batch, 7B decoder
        _loss("xent", "bf16", 8192, 32000, 4096, "loss fwd bf16"),
        # its gradient with respect to the hidden states and the output weights
        _loss("xent_bwd", "bf16", 8192, 32000, 4096, "loss bwd bf16"),
        # the GPT-2 small output layer in fp16, a ragged number of rows
        _loss("xent_bwd", "fp16", 1021, 50257, 768, "loss bwd ragged fp16"),
    ]


def _spread(rng, lo, hi):
    """A whole number between lo and hi, spread over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rope", "rope_bwd", "qk_norm", "qk_norm_train", "qk_norm_bwd", "xent", "xent_bwd"])
    if op.startswith("xent"):
        hidden = rng.choice([8 * _spread(rng, 8, 512), 64 * _spread(rng, 1, 64), _spread(rng, 33, 2049)])
        vocab = _spread(rng, 1000, 131072)
        rows = _spread(rng, 1, 8192)
        rows = max(1, min(rows, 8192 * 32000 * 4096 // (vocab * hidden), (1 << 30) // vocab))
        return _loss(op, rng.choice(["bf16", "bf16", "fp16"]), rows, vocab, hidden)
    dtype = rng.choice(["bf16", "bf16", "fp16", "fp32"])
    dim = rng.choice([64, 80, 96, 128, 128, 192, 256, 2 * rng.randint(17, 128)])
    rot = rng.choice([dim, dim, dim // 4 * 2, dim // 8 * 2])
    hk = rng.choice([1, 2, 4, 8, 12, 16, 32])
    hq = hk * rng.choice([1, 1, 2, 4, 8]) if hk <= 8 else hk
    if op == "qk_norm" or rng.random() < 0.25:
        batch, seq, far = _spread(rng, 1, 256), 1, 131072
    else:
        batch, seq, far = _spread(rng, 1, 16), _spread(rng, 2, 32768), rng.choice([0, 0, 65536])
    most = 4 * 4096 * 64 * 128 * 2 // (4 if dtype == "fp32" else 2)
    if batch * seq * (hq + hk) * dim > most // (2 if op.endswith("bwd") else 1):
        seq = max(1, most // (2 if op.endswith("bwd") else 1) // (batch * (hq + hk) * dim))
    return _heads(op, dtype, batch, seq, hq, hk, dim, rot, rng.random() < 0.4,
                  rng.choice(["qkv", "qkv", "bshd", "bhsd"]), far, rng.choice([1.0, 1.0, 4.0, 32.0]))


# ----------------------------------------------------------------------------- inputs
def _views(case, make):
    """Queries, keys of [batch, seq, heads, head_dim] in the case's layout, over buffers of make(shape)."""
    b, s, hq, hk, d = (case[k] for k in ("batch", "seq", "heads_q", "heads_k", "head_dim"))
    if case["layout"] == "qkv":   # one projection's output, the values behind the keys
        buf = make((b, s, hq + 2 * hk, d))
        return buf[:, :, :hq], buf[:, :, hq:hq + hk]
    if case["layout"] == "bhsd":
        return make((b, hq, s, d)).transpose(1, 2), make((b, hk, s, d)).transpose(1, 2)
    return make((b, s, hq, d)), make((b, s, hk, d))


def _inv_freq(rot, stretch):
    """Radians a position for each rotated pair, in double; positions divided by `stretch`."""
    return [10000.0 ** (-2.0 * i / rot) / stretch for i in range(rot // 2)]


def prepare(case, seed):
    dt = DTYPES[case["dtype"]]
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) * 7919 + 17)

    def normal(shape, std=1.0, mean=0.0, dtype=dt):
        return torch.empty(shape, dtype=torch.float32, device="cuda").normal_(mean, std, generator=g).to(dtype)

    st = dict(case)
    if case["op"].startswith("xent"):
        n, v, d = case["rows"], case["vocab"], case["hidden"]
        st["W"] = normal((v, d), 0.02)
        target = torch.randint(0, v, (n,), generator=g, device="cuda")
        # trained rows lean towards their target, some strongly: its logit is raised by 0..8
        lean = torch.rand((n, 1), generator=g, device="cuda") * (8.0 / (d * 0.02 ** 2))
        st["H"] = (normal((n, d), 1.0, 0.0, torch.float32) + lean * st["W"][target].float()).to(dt)
        # padding and prompt tokens take no part: about one row in eight, never the first
        skip = torch.rand((n,), generator=g, device="cuda") < 0.125
        skip[0] = False
        st["target"] = torch.where(skip, torch.full_like(target, IGNORE), target)
        if case["op"] == "xent":
            st["loss"] = torch.empty(n, dtype=torch.float32, device="cuda")
            st["lse"] = torch.empty(n, dtype=torch.float32, device="cuda")
        else:
            # the gradient of a mean over the rows that count (fp16 trains with a loss scale),
            # and the forward's saved sums
            st["dloss"] = (~skip).float() * ((1024.0 if dt == torch.float16 else 1.0) / (~skip).sum().float())
            st["lse"] = _log_sum_exp(st["H"].float() @ st["W"].float().t())
            st["dH"] = torch.empty_like(st["H"])
            st["dW"] = torch.empty_like(st["W"])
        return st

    b, s, hq, hk, d, rot = (case[k] for k in ("batch", "seq", "heads_q", "heads_k", "head_dim", "rotary_dim"))
    inv = _inv_freq(rot, case["stretch"])
    st["inv_freq"] = torch.tensor(inv, dtype=torch.float64, device="cuda")
    # the same as whole 2^-64 parts of a turn, as the framework keeps them
    turns = [int(round(f / TURN * 2.0 ** 64)) for f in inv]
    st["freqs"] = torch.tensor([t - (1 << 64) if t >= 1 << 63 else t for t in turns], dtype=torch.int64, device="cuda")
    start = torch.randint(0, case["far"] + 1, (b, 1), generator=g, device="cuda") if case["far"] else 0
    st["positions"] = (torch.arange(s, device="cuda")[None] + start).expand(b, s).contiguous()
    st["x"] = _views(case, normal)
    st["y"] = _views(case, lambda shape: torch.empty(shape, dtype=dt, device="cuda"))
    if case["op"].startswith("qk_norm"):
        st["gamma"] = tuple(normal((d,), 0.1, 1.0, torch.float32) for _ in range(2))
        st["eps"] = 1e-6
        if case["op"] == "qk_norm_train":
            st["inv_rms"] = tuple(torch.empty((b, s, h), dtype=torch.float32, device="cuda") for h in (hq, hk))
        if case["op"] == "qk_norm_bwd":
            st["inv_rms"] = tuple((x.double().square().mean(-1) + st["eps"]).rsqrt().float() for x in st["x"])
            st["dgamma"] = tuple(torch.empty(d, dtype=torch.float32, device="cuda") for _ in range(2))
            st["dy"] = _views(case, normal)
    elif case["op"] == "rope_bwd":
        st["dy"] = st["x"]
    return st


# ----------------------------------------------------------------------------- plain forms
def _log_sum_exp(logits):
    m = logits.max(-1, keepdim=True).values
    return ((logits - m).exp().sum(-1).log() + m[:, 0])


def _cos_sin(st):
    angle = st["positions"].double()[..., None] * st["inv_freq"]
    return angle.cos().float()[:, :, None], angle.sin().float()[:, :, None]


def _rotate(x, cos, sin, rot, interleaved):
    """Pairs (a, b) to (a cos - b sin, a sin + b cos); x in 32 bits, [batch, seq, heads, head_dim]."""
    r, rest = x[..., :rot], x[..., rot:]
    if interleaved:
        a, b = r[..., 0::2], r[..., 1::2]
        r = torch.stack((a * cos - b * sin, a * sin + b * cos), -1).flatten(-2)
    else:
        a, b = r[..., :rot // 2], r[..., rot // 2:]
        r = torch.cat((a * cos - b * sin, a * sin + b * cos), -1)
    return torch.cat((r, rest), -1)


def _plain_heads(st):
    cos, sin = _cos_sin(st)
    rot, inter, dt, op = st["rotary_dim"], st["interleaved"], DTYPES[st["dtype"]], st["op"]
    if op == "rope":
        q, k = (_rotate(x.float(), cos, sin, rot, inter).to(dt) for x in st["x"])
        return {"q": q, "k": k}
    if op == "rope_bwd":
        q, k = (_rotate(x.float(), cos, -sin, rot, inter).to(dt) for x in st["dy"])
        return {"dq": q, "dk": k}
    if op in ("qk_norm", "qk_norm_train"):
        (q, rq), (k, rk) = (_plain_norm(x, w, st["eps"], cos, sin, rot, inter) for x, w in zip(st["x"], st["gamma"]))
        out = {"q": q.to(dt), "k": k.to(dt)}
        return {**out, "inv_rms_q": rq, "inv_rms_k": rk} if op == "qk_norm_train" else out
    (dq, gq), (dk, gk) = (_plain_norm_bwd(*a, cos, sin, rot, inter)
                          for a in zip(st["dy"], st["x"], st["inv_rms"], st["gamma"]))
    return {"dq": dq.to(dt), "dk": dk.to(dt), "dgamma_q": gq, "dgamma_k": gk}


def _plain_norm(x, gamma, eps, cos, sin, rot, inter):
    x = x.float()
    inv = 1.0 / ((x * x).mean(-1) + eps).sqrt()
    return _rotate(x * inv[..., None] * gamma, cos, sin, rot, inter), inv


def _plain_norm_bwd(dy, x, inv, gamma, cos, sin, rot, inter):
    dn = _rotate(dy.float(), cos, -sin, rot, inter)
    xhat = x.float() * inv[..., None]
    # the sum over every token and head is long: 64 bits
    dgamma = (dn * xhat).sum((0, 1, 2), dtype=torch.float64).float()
    dxhat = dn * gamma
    return inv[..., None] * (dxhat - xhat * (dxhat * xhat).mean(-1, keepdim=True)), dgamma


def _plain_loss(st):
    H, W, t = st["H"].float(), st["W"].float(), st["target"]
    logits = H @ W.t()
    keep = t != IGNORE
    col = torch.where(keep, t, 0)[:, None]
    if st["op"] == "xent":
        lse = _log_sum_exp(logits)
        return {"loss": torch.where(keep, lse - logits.gather(1, col)[:, 0], 0.0), "lse": lse}
    p = (logits - st["lse"][:, None]).exp()
    p.scatter_add_(1, col, torch.full_like(col, -1, dtype=torch.float32))
    p = p * torch.where(keep, st["dloss"], 0.0)[:, None]
    return {"dH": (p @ W).to(st["H"].dtype), "dW": (p.t() @ H).to(st["W"].dtype)}


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
    if op == "xent":
        H, W = st["H"], st["W"]
        ws = _scratch(st, lambda: tb.tb_linear_xent_workspace_size(*H.shape, W.shape[0], H.dtype))
        tb.tb_linear_xent(H, W, st["target"], st["loss"], st["lse"], ws, ignore_index=IGNORE)
        return {"loss": st["loss"], "lse": st["lse"]}
    if op == "xent_bwd":
        H, W = st["H"], st["W"]
        ws = _scratch(st, lambda: tb.tb_linear_xent_bwd_workspace_size(*H.shape, W.shape[0], H.dtype))
        tb.tb_linear_xent_bwd(st["dloss"], H, W, st["target"], st["lse"], st["dH"], st["dW"], ws, ignore_index=IGNORE)
        return {"dH": st["dH"], "dW": st["dW"]}
    kw = dict(freqs=st["freqs"], positions=st["positions"], interleaved=st["interleaved"])
    (q, k), (yq, yk) = st["x"], st["y"]
    if op == "rope":
        tb.tb_rope(q, k, yq, yk, **kw)
        return {"q": yq, "k": yk}
    if op == "rope_bwd":
        tb.tb_rope_bwd(*st["dy"], yq, yk, **kw)
        return {"dq": yq, "dk": yk}
    if op == "qk_norm":
        tb.tb_qk_norm_rope(q, k, *st["gamma"], yq, yk, eps=st["eps"], **kw)
        return {"q": yq, "k": yk}
    if op == "qk_norm_train":
        tb.tb_qk_norm_rope(q, k, *st["gamma"], yq, yk, *st["inv_rms"], eps=st["eps"], **kw)
        return {"q": yq, "k": yk, "inv_rms_q": st["inv_rms"][0], "inv_rms_k": st["inv_rms"][1]}
    ws = _scratch(st, lambda: tb.tb_qk_norm_rope_bwd_workspace_size(
        q.shape[0], q.shape[1], q.shape[2], k.shape[2], q.shape[3], q.dtype))
    tb.tb_qk_norm_rope_bwd(*st["dy"], q, k, *st["inv_rms"], *st["gamma"], yq, yk, *st["dgamma"], workspace=ws, **kw)
    return {"dq": yq, "dk": yk, "dgamma_q": st["dgamma"][0], "dgamma_k": st["dgamma"][1]}


def run(state):
    if own:
        return _own_run(state)
    return _plain_loss(state) if state["op"].startswith("xent") else _plain_heads(state)


# ----------------------------------------------------------------------------- what a call cannot do without
def work(case):
    es = 4 if case["dtype"] == "fp32" else 2
    if case["op"].startswith("xent"):
        n, v, d = case["rows"], case["vocab"], case["hidden"]
        inputs = (n * d + v * d) * es + n * 8
        if case["op"] == "xent":
            return {"bytes": inputs + n * 8, "flops": 2 * n * v * d}
        # the logits again (they are not kept), and one product for each of the two gradients
        return {"bytes": 2 * (n * d + v * d) * es + n * 16, "flops": 6 * n * v * d}
    tokens = case["batch"] * case["seq"]
    heads, d, rot = case["heads_q"] + case["heads_k"], case["head_dim"], case["rotary_dim"]
    n = tokens * heads * d
    small = tokens * 8 + rot * 4
    turn = 3 * tokens * heads * rot
    if case["op"] in ("rope", "rope_bwd"):
        return {"bytes": 2 * n * es + small, "flops": turn}
    if case["op"] in ("qk_norm", "qk_norm_train"):
        saved = tokens * heads * 4 if case["op"] == "qk_norm_train" else 0
        return {"bytes": 2 * n * es + small + saved + 8 * d, "flops": turn + 4 * n}
    return {"bytes": 3 * n * es + small + tokens * heads * 4 + 16 * d, "flops": turn + 9 * n}


# ----------------------------------------------------------------------------- 64 bits
def _turned(x, st, sign):
    """x in 64 bits with its pairs, as complex numbers, multiplied by exp(i sign angle)."""
    rot = st["rotary_dim"]
    angle = sign * st["positions"].double()[:, :, None, None] * st["inv_freq"]
    x = x.clone()
    pair = x[..., :rot].unflatten(-1, (rot // 2, 2) if st["interleaved"] else (2, rot // 2))
    if not st["interleaved"]:
        pair = pair.transpose(-1, -2)
    z = torch.view_as_complex(pair.contiguous()) * torch.polar(torch.ones_like(angle), angle)
    back = torch.view_as_real(z)
    x[..., :rot] = (back if st["interleaved"] else back.transpose(-1, -2)).flatten(-2)
    return x


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "rope":
        return {"q": _turned(st["x"][0].double(), st, 1), "k": _turned(st["x"][1].double(), st, 1)}
    if op == "rope_bwd":
        return {"dq": _turned(st["dy"][0].double(), st, -1), "dk": _turned(st["dy"][1].double(), st, -1)}
    if op.startswith("qk_norm"):
        out = {}
        for i, name in enumerate("qk"):
            x, w = st["x"][i].double(), st["gamma"][i].double()
            if op != "qk_norm_bwd":
                inv = torch.rsqrt(torch.linalg.vector_norm(x, dim=-1).square() / case["head_dim"] + st["eps"])
                out[name] = _turned(w * x * inv[..., None], st, 1)
                if op == "qk_norm_train":
                    out["inv_rms_" + name] = inv
                continue
            inv = st["inv_rms"][i].double()[..., None]
            up = _turned(st["dy"][i].double(), st, -1)
            out["dgamma_" + name] = torch.einsum("bshd,bshd->d", up, x * inv)
            up = up * w
            out["d" + name] = inv * up - inv ** 3 * x * (torch.einsum("bshd,bshd->bsh", up, x)[..., None] / case["head_dim"])
        return out
    if 6 * case["rows"] * case["vocab"] * case["hidden"] > 8e12:   # about 10 seconds of 64-bit products
        return None
    n, v = case["rows"], case["vocab"]
    W, step = st["W"].double(), max(1, (1 << 28) // v)
    loss, lses, dH, dW = [], [], [], None if op == "xent" else torch.zeros_like(W)
    for lo in range(0, n, step):
        H, t = st["H"][lo:lo + step].double(), st["target"][lo:lo + step]
        logits = H @ W.T
        rows, keep = torch.arange(len(t), device="cuda"), t != IGNORE
        at = torch.where(keep, t, torch.zeros_like(t))
        if op == "xent":
            lses.append(torch.logsumexp(logits, -1))
            loss.append((lses[-1] - logits[rows, at]) * keep)
            continue
        grad = torch.exp(logits - st["lse"][lo:lo + step, None].double())
        grad[rows, at] -= 1.0
        grad *= (st["dloss"][lo:lo + step].double() * keep)[:, None]
        dH.append(grad @ W)
        dW += grad.T @ H
    return {"loss": torch.cat(loss), "lse": torch.cat(lses)} if op == "xent" else {"dH": torch.cat(dH), "dW": dW}
