"""The operators of a prompt encoder's layer, as cases that can be measured.

One layer of the encoder that produces a denoiser's text features is made of
attention over packed prompts (causal, grouped heads), Linears with bias,
activation and residual, and a gated feed-forward block.  This file holds
their cases, inputs, plain forms (elementary torch operations in fp32), values
in 64 bits and the bytes and operations each case cannot do without.
"""
import math

import torch

own = False

D = 128                     # head dimension of the framework's attention
SCALE = D ** -0.5


# ------------------------------------------------------------------ cases

def _lens(values):
    return ",".join(str(int(v)) for v in values)


def listed():
    return [
        # one new token against a long cache: the latency of token-by-token use
        dict(name="attn_token", op="attn", heads=32, kv_heads=8, q="1", k="8192"),
        # one new token for each of many sequences of different lengths
        dict(name="attn_tokens_ragged", op="attn", heads=32, kv_heads=8, q=_lens([1] * 48),
             k=_lens(100 + (i * 977) % 4000 for i in range(48))),
        # a batch of prompts from a few words to long ones (prompts and negative prompts)
        dict(name="attn_prompts_ragged", op="attn", heads=32, kv_heads=8,
             q=_lens(5 + (i * i * 37) % 700 for i in range(24)),
             k=_lens(5 + (i * i * 37) % 700 for i in range(24))),
        # one very long prompt
        dict(name="attn_prompt_long", op="attn", heads=32, kv_heads=8, q="16384", k="16384"),
        # output projection of one token: bias and residual
        dict(name="linear_token", op="linear", m=1, k=4096, n=4096, act="none", residual=True),
        # fused q | k | v projection of a prompt and its negative prompt
        dict(name="linear_prompt", op="linear", m=768, k=4096, n=6144, act="none", residual=False),
        # MLP up projection of a 1024 x 1024 pixel joint sequence
        dict(name="linear_long", op="linear", m=4608, k=4096, n=16384, act="gelu_tanh", residual=False),
        # feed-forward block of one token, of a prompt pair and of a long sequence
        dict(name="ffn_token", op="ffn", m=1, hidden=4096, mlp=11008, act="silu", train=False),
        dict(name="ffn_prompt", op="ffn", m=768, hidden=4096, mlp=11008, act="silu", train=False),
        dict(name="ffn_long", op="ffn", m=4608, hidden=4096, mlp=16384, act="gelu_tanh", train=False),
        # forward and backward of the block: a small model's odd batch, a full width one
        dict(name="ffn_train_small", op="ffn", m=333, hidden=1024, mlp=2816, act="silu", train=True),
        dict(name="ffn_train", op="ffn", m=4096, hidden=4096, mlp=11008, act="silu", train=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attn", "attn", "linear", "ffn"])
    if op == "attn":
        heads, kv_heads = rng.choice([(32, 8), (32, 32), (16, 2), (28, 4), (8, 8), (20, 4), (32, 1)])
        kind = rng.choice(["tokens", "prompts", "cached"])
        if kind == "tokens":
            n = _log(rng, 1, 96)
            q = [1] * n
            k = [_log(rng, 1, 6000) for _ in range(n)]
        else:
            n = _log(rng, 1, 32)
            q = [_log(rng, 1, 6000 / n ** 0.5) for _ in range(n)]
            k = [x + (_log(rng, 1, 2000) if kind == "cached" else 0) for x in q]
        return dict(op=op, heads=heads, kv_heads=kv_heads, q=_lens(q), k=_lens(k))
    m = _log(rng, 1, 4096)
    act = rng.choice(["silu", "gelu_tanh"])
    if op == "linear":
        return dict(op=op, m=m, k=8 * _log(rng, 16, 1024), n=_log(rng, 40, 12000),
                    act=rng.choice(["none", act]), residual=rng.random() < 0.5)
    train = rng.random() < 0.5
    return dict(op=op, m=m, hidden=8 * _log(rng, 32, 512), mlp=8 * _log(rng, 64, 1376), act=act, train=train)


# ------------------------------------------------------------------ inputs

def _ints(text):
    return [int(v) for v in text.split(",")]


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape, scale=1.0):
        return (torch.randn(shape, generator=g, device="cuda") * scale).to(torch.bfloat16)

    s = dict(case)
    if case["op"] == "attn":
        ql, kl = _ints(case["q"]), _ints(case["k"])
        # [n, 4]: first query row, queries, first key row, keys (a host table, as the call takes it)
        spans, q0, k0 = [], 0, 0
        for a, b in zip(ql, kl):
            spans.append((q0, a, k0, b))
            q0, k0 = q0 + a, k0 + b
        s["spans"] = torch.tensor(spans, dtype=torch.int32)
        s["q"] = normal(q0, case["heads"] * D)
        s["k"] = normal(k0, case["kv_heads"] * D)
        s["v"] = normal(k0, case["kv_heads"] * D)
        # the same table per row, for the plain form: sequence of a row and its place in it
        n = torch.arange(len(ql), device="cuda")
        tq, tk = torch.tensor(ql, device="cuda"), torch.tensor(kl, device="cuda")
        s["q_seq"], s["k_seq"] = n.repeat_interleave(tq), n.repeat_interleave(tk)
        qpos = torch.arange(q0, device="cuda") - (tq.cumsum(0) - tq)[s["q_seq"]]
        s["q_last"] = qpos + (tk - tq)[s["q_seq"]]                       # last key a query sees
        s["k_pos"] = torch.arange(k0, device="cuda") - (tk.cumsum(0) - tk)[s["k_seq"]]
    elif case["op"] == "linear":
        m, k, n = case["m"], case["k"], case["n"]
        s["a"], s["w"], s["bias"] = normal(m, k), normal(n, k, scale=0.02), normal(n, scale=0.02)
        s["res"] = normal(m, n) if case["residual"] else None
    else:
        m, h, f = case["m"], case["hidden"], case["mlp"]
        s["x"] = normal(m, h)
        s["wg"], s["wu"] = normal(f, h, scale=0.02), normal(f, h, scale=0.02)
        s["wd"] = normal(h, f, scale=0.02)
        s["dy" if case["train"] else "res"] = normal(m, h)
    return s


# ------------------------------------------------------------------ plain forms (fp32)

def _act(x, kind):
    if kind == "silu":
        return x / (1 + torch.exp(-x))
    if kind == "gelu_tanh":
        return 0.5 * x * (1 + torch.tanh(0.7978845608028654 * (x + 0.044715 * x * x * x)))
    return x


def _act_grad(x, kind):
    if kind == "silu":
        s = 1 / (1 + torch.exp(-x))
        return s * (1 + x * (1 - s))
    t = torch.tanh(0.7978845608028654 * (x + 0.044715 * x * x * x))
    return 0.5 * (1 + t) + 0.5 * x * (1 - t * t) * 0.7978845608028654 * (1 + 3 * 0.044715 * x * x)


def _attn_plain(s):
    heads, kvh = s["heads"], s["kv_heads"]
    grp = heads // kvh
    q = s["q"].float().view(-1, kvh, grp, D).permute(1, 2, 0, 3)         # [kvh, grp, Tq, D]
    k = s["k"].float().view(-1, kvh, D).permute(1, 2, 0)                 # [kvh, D, Tk]
    v = s["v"].float().view(-1, kvh, D).permute(1, 0, 2)                 # [kvh, Tk, D]
    tq = q.shape[2]
    p = torch.matmul(q.reshape(kvh, grp * tq, D) * SCALE, k)
    hidden = (s["q_seq"][:, None] != s["k_seq"][None, :]) | (s["k_pos"][None, :] > s["q_last"][:, None])
    p.view(kvh, grp, tq, -1).masked_fill_(hidden, -math.inf)
    top = p.amax(-1, keepdim=True)
    p.sub_(torch.where(top == -math.inf, torch.zeros_like(top), top)).exp_()
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p, v) / torch.where(total == 0, torch.ones_like(total), total)
    return o.view(kvh, grp, tq, D).permute(2, 0, 1, 3).reshape(tq, heads * D).to(torch.bfloat16)


def _linear_plain(s):
    y = _act(s["a"].float() @ s["w"].float().t() + s["bias"].float(), s["act"])
    if s["res"] is not None:
        y = y + s["res"].float()
    return y.to(torch.bfloat16)


def _ffn_plain(s):
    x, wg, wu, wd = (s[n].float() for n in ("x", "wg", "wu", "wd"))
    g, u = x @ wg.t(), x @ wu.t()
    a = _act(g, s["act"])
    h = a * u
    y = h @ wd.t()
    if not s["train"]:
        return (y + s["res"].float()).to(torch.bfloat16)
    dy = s["dy"].float()
    dh = dy @ wd
    dg, du = dh * u * _act_grad(g, s["act"]), dh * a
    out = dict(y=y, dx=dg @ wg + du @ wu, dgate=dg.t() @ x, dup=du.t() @ x, ddown=dy.t() @ h)
    return {n: t.to(torch.bfloat16) for n, t in out.items()}


# ------------------------------------------------------------------ the framework's calls

_ctx = []


def _own(s):
    from diffusion_transformer_text_dit_b200 import qi
    if not _ctx:
        _ctx.append(qi.Context())     # one context per process, as a program holds it
    ctx = _ctx[0]
    if s["op"] == "attn":
        return qi.qi_attn_causal_packed(ctx, s["q"], s["k"], s["v"], s["spans"], s["heads"], s["kv_heads"])
    act = {"none": qi.QI_ACT_NONE, "silu": qi.QI_ACT_SILU, "gelu_tanh": qi.QI_ACT_GELU_TANH}[s["act"]]
    if s["op"] == "linear":
        if "layer" not in s:          # the weight handle that a model keeps
            s["layer"] = qi.bf16_struct(s["w"], s["bias"])
        return qi.qi_linear_act(ctx, s["a"], s["layer"], act, residual=s["res"])
    if "layer" not in s:
        s["layer"] = qi.gated_ffn_struct(s["wg"], s["wu"], s["wd"], act)
    if not s["train"]:
        return qi.qi_gated_ffn_forward(ctx, s["layer"], s["x"], residual=s["res"])
    y, saved = qi.qi_gated_ffn_forward(ctx, s["layer"], s["x"], save=True)
    dx, dgate, dup, ddown = qi.qi_gated_ffn_backward(ctx, s["layer"], s["x"], s["dy"], saved)
    return dict(y=y, dx=dx, dgate=dgate, dup=dup, ddown=ddown)


def run(state):
    if own:
        return _own(state)
    return {"attn": _attn_plain, "linear": _linear_plain, "ffn": _ffn_plain}[state["op"]](state)


# ------------------------------------------------------------------ what a case cannot do without

def work(case):
    if case["op"] == "attn":
        ql, kl = _ints(case["q"]), _ints(case["k"])
        pairs, keys = 0, 0
        for a, b in zip(ql, kl):
            first = b - a + 1                       # keys the first query sees
            keys += b
            pairs += sum(max(0, first + i) for i in range(a))
        return dict(bytes=2 * D * (2 * case["heads"] * sum(ql) + 2 * case["kv_heads"] * keys),
                    flops=4 * D * case["heads"] * pairs)
    m = case["m"]
    if case["op"] == "linear":
        k, n = case["k"], case["n"]
        return dict(bytes=2 * (m * k + n * k + n + m * n * (2 if case["residual"] else 1)),
                    flops=2 * m * n * k)
    h, f = case["hidden"], case["mlp"]
    if case["train"]:                               # x, dy, weights in; y, dx, weight gradients out
        return dict(bytes=2 * (4 * m * h + 6 * h * f), flops=18 * m * h * f)
    return dict(bytes=2 * (3 * m * h + 3 * h * f), flops=6 * m * h * f)


# ------------------------------------------------------------------ values in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "attn":
        q, k, v = s["q"].double(), s["k"].double(), s["v"].double()
        per = case["heads"] // case["kv_heads"]
        out = torch.zeros_like(q)
        for q0, ql, k0, kl in s["spans"].tolist():
            at = torch.arange(ql, device="cuda")[:, None] + (kl - ql)
            see = torch.arange(kl, device="cuda")[None, :] <= at
            for head in range(case["heads"]):
                c, e = slice(head * D, head * D + D), slice(head // per * D, head // per * D + D)
                score = torch.einsum("id,jd->ij", q[q0:q0 + ql, c], k[k0:k0 + kl, e]) / math.sqrt(D)
                w = torch.softmax(torch.where(see, score, torch.full_like(score, -math.inf)), -1)
                out[q0:q0 + ql, c] = torch.nan_to_num(w) @ v[k0:k0 + kl, e]
        return out
    if case["op"] == "linear":
        z = torch.einsum("mk,nk->mn", s["a"].double(), s["w"].double()) + s["bias"].double()
        z = {"none": lambda t: t, "silu": lambda t: t * torch.sigmoid(t),
             "gelu_tanh": lambda t: torch.nn.functional.gelu(t, approximate="tanh")}[case["act"]](z)
        return z + s["res"].double() if case["residual"] else z
    x, wg, wu, wd = (s[n].double() for n in ("x", "wg", "wu", "wd"))
    gate, up = torch.einsum("mh,fh->mf", x, wg), torch.einsum("mh,fh->mf", x, wu)
    if case["act"] == "silu":
        sig = torch.sigmoid(gate)
        a, da = gate * sig, sig + gate * sig * (1 - sig)
    else:
        c = math.sqrt(2 / math.pi)
        t = torch.tanh(c * (gate + 0.044715 * gate ** 3))
        a = 0.5 * gate * (1 + t)
        da = 0.5 * (1 + t) + 0.5 * gate * (1 - t ** 2) * c * (1 + 0.134145 * gate ** 2)
    y = torch.einsum("mf,hf->mh", a * up, wd)
    if not case["train"]:
        return y + s["res"].double()
    dy = s["dy"].double()
    dh = torch.einsum("mh,hf->mf", dy, wd)
    dgate, dup = dh * up * da, dh * a
    return dict(y=y, dx=torch.einsum("mf,fh->mh", dgate, wg) + torch.einsum("mf,fh->mh", dup, wu),
                dgate=torch.einsum("mf,mh->fh", dgate, x), dup=torch.einsum("mf,mh->fh", dup, x),
                ddown=torch.einsum("mh,mf->hf", dy, a * up))
