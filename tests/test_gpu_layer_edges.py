"""Calls of the prompt-encoder layer operators at their edges, against 64-bit
formulas.  Tolerances count roundings with u = 2^-8, half a bf16 step relative
to the value, as in the tests of the shapes."""
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

from diffusion_transformer_text_dit_b200 import qi

pytestmark = pytest.mark.gpu
U = 2.0 ** -8
BF = torch.bfloat16


def rand(*shape, seed=0, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed * 7919 + sum(shape))
    return (torch.randn(shape, generator=g, device="cuda") * scale).to(BF)


def same_bits(a, b):
    """Equal bit patterns (NaN equal to itself, unlike torch.equal)."""
    assert a.dtype == b.dtype
    return torch.equal(a.contiguous().view(torch.int16), b.contiguous().view(torch.int16))


def acc_tol(a, b):
    """fp32 sum of a @ b^T (64-bit inputs): the tensor core adds 16 products at a
    time, k / 16 + 2 sums rounded by 2^-23 of the absolute values at most; times
    1.13, the largest slope of the activations."""
    return 1.13 * (a.shape[1] / 16 + 2) * 2.0 ** -23 * (a.abs() @ b.abs().T)


@pytest.mark.parametrize("M", [1025, 1100, 1152, 1153, 1280])
@pytest.mark.parametrize("n", [2304, 12000])
def test_products_that_follow_each_other_closely(ctx, M, n):
    """Products of one and of several tiles per pair of CTAs, whose last 128 rows
    exist or not, each started while the one before it ends: every one gives the
    bits it gives alone."""
    k = 1032
    ops = [(rand(M, k, seed=i), qi.bf16_struct(rand(n, k, seed=10 + i, scale=0.05), rand(n, seed=20 + i)))
           for i in range(3)]
    alone = []
    for a, w in ops:
        alone.append(qi.qi_linear_act(ctx, a, w, qi.QI_ACT_SILU))
        torch.cuda.synchronize()
    a, w = ops[0][0].double(), ops[0][1]._keep[0].double()
    ref = a @ w.T + ops[0][1]._keep[1].double()
    ref = ref * torch.sigmoid(ref)
    # (2^-16: the activation's own evaluation in fp32)
    assert ((alone[0].double() - ref).abs() <= acc_tol(a, w) + (U + 2.0 ** -16) * ref.abs()).all()
    outs = [[qi.qi_linear_act(ctx, x, y, qi.QI_ACT_SILU) for x, y in ops] for _ in range(8)]
    ctx.check()
    for got in outs:
        assert all(same_bits(x, y) for x, y in zip(got, alone))


def act64(x, act):
    if act == qi.QI_ACT_SILU:
        return x * torch.sigmoid(x)
    # 0.5 (1 + tanh z) = logistic(2 z), without the cancellation of 1 + tanh z at z << 0
    return x * torch.sigmoid(2 * (2 / np.pi) ** 0.5 * (x + 0.044715 * x ** 3))


@pytest.mark.parametrize("act", [qi.QI_ACT_SILU, qi.QI_ACT_GELU_TANH])
@pytest.mark.parametrize("M", [1, 40, 1300])
def test_gated_ffn_gradients_at_the_ends(ctx, M, act):
    """Gate values of both signs up to the largest: the activation's derivative goes to
    1 and 0, not to NaN.  Row 0 of dy and x and the weights pick act(g) and act'(g)
    out of the sums: one term each, the rest 0.  One rounding to bf16 (the output
    repeats it exactly) and 2^-15 for the evaluation in fp32 (two terms)."""
    ends = [0.0, 1e-3, 8.0, 40.0, 100.0, 3e4, 1.8e19, 2e19, 1e30, 3e38]
    g = torch.tensor([s * v for v in ends for s in (1.0, -1.0)] + [0.5, -0.5, 3.0, -3.0], device="cuda")
    F = H = len(g)
    up = torch.zeros(F, H, dtype=BF, device="cuda")
    gate = torch.eye(F, dtype=BF, device="cuda")
    down = torch.zeros(H, F, dtype=BF, device="cuda")
    down[0] = 1
    x, dy = (torch.zeros(M, H, dtype=BF, device="cuda") for _ in range(2))
    x[0, 0] = dy[0, 0] = 1
    gate_up = torch.cat([g, torch.ones_like(g)]).repeat(M, 1)
    dx, dgate, dup, ddown = qi.qi_gated_ffn_backward(ctx, qi.gated_ffn_struct(gate, up, down, act), x, dy, gate_up)
    ctx.check()
    at = g.double().requires_grad_(True)
    value = act64(at, act)
    slope = torch.autograd.grad(value.sum(), at)[0]
    for got, ref in ((dx[0], slope), (dgate[:, 0], slope), (dup[:, 0], value), (ddown[0], value)):
        ref = ref.detach()
        assert torch.isfinite(got).all()
        assert ((got.double() - ref).abs() <= (U + 2.0 ** -15) * ref.abs() + 1e-30).all()


FIRST_CALLS = """
import threading
import torch
from diffusion_transformer_text_dit_b200 import qi

torch.manual_seed(1)
n = 6
a, w = (torch.randn(300, 520, device="cuda").bfloat16() for _ in range(2))
q, k, v = (torch.randn(200, 256, device="cuda").bfloat16() for _ in range(3))
spans = torch.tensor([[0, 200, 0, 200]], dtype=torch.int32)
work = [(qi.Context(), torch.cuda.Stream(), torch.empty_like(q), torch.empty(300, 300, device="cuda").bfloat16())
        for _ in range(n)]
torch.cuda.synchronize()
ready, failed = threading.Barrier(n), []

def call(i):
    c, st, o, y = work[i]
    ready.wait()
    try:
        if i % 2:
            qi.qi_attn_causal_packed(c, q, k, v, spans, 2, 2, o=o, stream=st)
        qi.qi_linear_act(c, a, qi.bf16_struct(w), y=y, stream=st)
        if not i % 2:
            qi.qi_attn_causal_packed(c, q, k, v, spans, 2, 2, o=o, stream=st)
        c.check(st)
    except Exception as e:
        failed.append(e)

threads = [threading.Thread(target=call, args=(i,)) for i in range(n)]
[t.start() for t in threads]
[t.join() for t in threads]
assert not failed, failed
bits = lambda t: t.view(torch.int16)
assert all(torch.equal(bits(x[2]), bits(work[0][2])) and torch.equal(bits(x[3]), bits(work[0][3])) for x in work)
print("same")
"""


def test_first_calls_from_several_threads(ctx):
    """The first calls of a process, made at the same time by host threads with a
    context and a stream each (what the library looks up on first use, it looks up
    once for all or again with the same answer)."""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", FIRST_CALLS], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip() == "same", r.stderr


@pytest.mark.parametrize("T", [1, 70, 700])
def test_outputs_between_the_columns_of_their_inputs(ctx, T):
    """q | k | v | o, x | y | residual and x | dx | dy as column ranges of one block
    of rows: the bits of separate buffers, and the other columns as they were."""
    heads, kvh, H, F = 8, 2, 256, 520
    W, KW = heads * 128, kvh * 128
    block = rand(T, 2 * W + 2 * KW + 64, seed=3)
    before = block.clone()
    q, k, v, o = (block[:, a:b] for a, b in ((0, W), (W, W + KW), (W + KW, W + 2 * KW), (W + 2 * KW, 2 * W + 2 * KW)))
    spans = torch.tensor([[0, T, 0, T]], dtype=torch.int32)
    want = qi.qi_attn_causal_packed(ctx, *(t.contiguous() for t in (q, k, v)), spans, heads, kvh)
    qi.qi_attn_causal_packed(ctx, q, k, v, spans, heads, kvh, o=o)
    ctx.check()
    assert same_bits(o, want)
    o.copy_(before[:, W + 2 * KW:2 * W + 2 * KW])
    assert same_bits(block, before)

    for n, at in ((136, 2 * H), (131, 2 * H - 1)):     # rows that are 16-byte aligned, and not
        block = rand(T, 3 * H, seed=4)
        before = block.clone()
        a, y, res = block[:, :H], block[:, H:H + n], block[:, at:at + n]
        w = qi.bf16_struct(rand(n, H, seed=5, scale=0.05), rand(n, seed=6))
        want = qi.qi_linear_act(ctx, a.contiguous(), w, qi.QI_ACT_SILU, residual=res.contiguous())
        qi.qi_linear_act(ctx, a, w, qi.QI_ACT_SILU, residual=res, y=y)
        ctx.check()
        # (other rows may take another kernel, and another order of the sums: two roundings of sums that
        # differ by 2 (k / 16 + 2) 2^-23 sum |a w| < 2^-14 at most)
        assert ((y.double() - want.double()).abs() <= 2 * U * want.double().abs() + 2.0 ** -14).all()
        y.copy_(before[:, H:H + n])
        assert same_bits(block, before)

    ffn = qi.gated_ffn_struct(rand(F, H, seed=7, scale=H ** -0.5), rand(F, H, seed=8, scale=H ** -0.5),
                              rand(H, F, seed=9, scale=F ** -0.5))
    block = rand(T, 3 * H, seed=10)
    before = block.clone()
    x, dx, dy = block[:, :H], block[:, H:2 * H], block[:, 2 * H:]
    want, saved = qi.qi_gated_ffn_forward(ctx, ffn, x, save=True)
    full = qi.qi_gated_ffn_backward(ctx, ffn, x.contiguous(), dy.contiguous(), saved)
    got = qi.qi_gated_ffn_backward(ctx, ffn, x, dy, saved, dx=dx)
    ctx.check()
    assert all(same_bits(s, t) for s, t in zip(got, full))
    dx.copy_(before[:, H:2 * H])
    assert same_bits(block, before)
    qi.qi_gated_ffn_forward(ctx, ffn, x, residual=dy, y=dx)
    plain = qi.qi_gated_ffn_forward(ctx, ffn, x.contiguous(), residual=dy.contiguous())
    ctx.check()
    assert same_bits(dx, plain) and same_bits(dy, before[:, 2 * H:]) and same_bits(x, before[:, :H])


# ------------------------------------------------------------------ every key of a split range

def peaked(k, kvh, j, r, a=60.0):
    """Queries [n, heads * 128] that put about half of their weight each on the keys
    j[i, h] and r[i, h] of their key/value head: q scale = a (k_j / |k_j|^2 + k_r / |k_r|^2),
    so both score about a and the rest at most half of it (128 columns: |k_i k_j| is
    a tenth of |k|^2, five times that at most)."""
    n, heads = j.shape
    K = k.double().view(-1, kvh, 128)
    head = (torch.arange(heads, device="cuda") // (heads // kvh)).expand(n, heads)
    q = sum(K[x, head] / K[x, head].pow(2).sum(-1, keepdim=True) for x in (j, r))
    return (q * a * 128 ** 0.5).reshape(n, heads * 128).to(BF)


def check_peaked(q, k, v, spans, kvh, got, causal=True):
    """Against the formula in 64 bits; a key lost or counted twice would move the
    output by a third of a value at least, of which the tolerance (the weights' and
    the output's rounding to bf16, 2^-12 for the rest) is a hundredth."""
    heads = q.shape[1] // 128
    for q0, ql, k0, kl in spans:
        see = torch.arange(kl, device="cuda")[None] <= kl - ql + torch.arange(ql, device="cuda")[:, None]
        for h in range(heads):
            c, e = slice(h * 128, h * 128 + 128), h // (heads // kvh)
            kv = slice(e * 128, e * 128 + 128)
            s = q[q0:q0 + ql, c].double() @ k[k0:k0 + kl, kv].double().T * 128 ** -0.5
            if causal:
                s = s.masked_fill(~see, -np.inf)
            p, V = torch.softmax(s, -1), v[k0:k0 + kl, kv].double()
            o, mag = p @ V, p @ V.abs()
            assert ((got[q0:q0 + ql, c].double() - o).abs() <= U * o.abs() + (U * (1 + U) + 2.0 ** -12) * mag).all()


def test_token_every_key_of_a_split_range(ctx):
    """One token on 8191 keys, split over ranges: every key in turn carries half of
    the weight of one head, so one that is left out or taken twice shows."""
    heads, kvh, n = 8, 2, 8191
    k, v = rand(n, kvh * 128, seed=1), rand(n, kvh * 128, seed=2)
    calls = -(-n // 4)                         # 4 heads on each key/value head
    j = (torch.arange(calls * 4, device="cuda").view(calls, 1, 4) % n).expand(calls, 2, 4).reshape(calls, heads)
    r = (j + 3001 + 7 * torch.arange(calls, device="cuda")[:, None]) % n
    q = peaked(k, kvh, j, r)
    one = torch.tensor([[0, 1, 0, n]], dtype=torch.int32)
    assert qi.qi_attn_causal_packed_workspace_bytes(ctx, one, heads, kvh) > 0
    o = torch.empty_like(q)
    for i in range(calls):
        qi.qi_attn_causal_packed(ctx, q[i:i + 1], k, v, one, heads, kvh, o=o[i:i + 1])
    ctx.check()
    check_peaked(q, k, v, [(0, calls, 0, n)], kvh, o, causal=False)   # (a call each: all see all the keys)


def test_tokens_every_key_of_longer_ranges(ctx):
    """256 tokens that share 8191 keys (their ranges are longer than a single token's)."""
    heads, kvh, n, T = 8, 2, 8191, qi.QI_MAX_SEQS
    k, v = rand(n, kvh * 128, seed=1), rand(n, kvh * 128, seed=2)
    spans = [(i, 1, 0, n) for i in range(T)]
    for first in range(0, n, T * 4):
        j = ((first + torch.arange(T * 4, device="cuda")) % n).view(T, 1, 4).expand(T, 2, 4).reshape(T, heads)
        r = (j + 2999 + 13 * torch.arange(T, device="cuda")[:, None]) % n
        q = peaked(k, kvh, j, r)
        got = qi.qi_attn_causal_packed(ctx, q, k, v, torch.tensor(spans, dtype=torch.int32), heads, kvh)
        ctx.check()
        check_peaked(q, k, v, spans, kvh, got)


@pytest.mark.parametrize("ql,kl", [(300, 5000), (40, 3000), (2, 6001)])
def test_prompt_every_key_of_a_split_range(ctx, ql, kl):
    """Queries behind cached keys on tiles (and two rows of tokens) whose keys are
    split: every key carries weight somewhere, and at the diagonal the last key
    that a query sees and the first it does not."""
    heads, kvh = 8, 2
    k, v = rand(kl, kvh * 128, seed=1), rand(kl, kvh * 128, seed=2)
    table = torch.tensor([[0, ql, 0, kl]], dtype=torch.int32)
    assert qi.qi_attn_causal_packed_workspace_bytes(ctx, table, heads, kvh) > 0
    i = torch.arange(ql, device="cuda")
    last = (kl - ql + i)[:, None, None]                    # the last key that query i sees
    step = torch.arange(ql * 4, device="cuda").view(ql, 1, 4)
    picks = [(first + step) % (kl - ql + 1) for first in range(0, kl - ql + 1, ql * 4)]   # seen by every query
    picks += [(last - torch.arange(4, device="cuda") - 4 * a).clamp(min=0) for a in range(2)]
    picks.append((last + 1 + torch.arange(4, device="cuda")).clamp(max=kl - 1))            # past the diagonal
    for n, j in enumerate(picks):
        j = j.expand(ql, 2, 4).reshape(ql, heads)
        r = (j + 1009 + 17 * n) % (kl - ql + 1)
        q = peaked(k, kvh, j, r)
        got = qi.qi_attn_causal_packed(ctx, q, k, v, table, heads, kvh)
        ctx.check()
        check_peaked(q, k, v, [(0, ql, 0, kl)], kvh, got)


# ------------------------------------------------------------------ buffers of more than 2^31 values

@pytest.mark.parametrize("n,shift", [(40, 0), (41, 1)])
def test_linear_rows_past_2_to_31_values(ctx, n, shift):
    """Inputs, residual and outputs whose offsets pass 2^31 values and 2^32 bytes:
    aligned rows (TMA) and rows at odd addresses (single values)."""
    M, ld, k = 530000, 4096, 64
    block = torch.zeros(M, ld, dtype=BF, device="cuda")
    a, y, res = block[:, :k], block[:, 128 + shift:128 + shift + n], block[:, 256 + shift:256 + shift + n]
    a.copy_(rand(M, k, seed=1))
    res.copy_(rand(M, n, seed=2))
    w, b = rand(n, k, seed=3, scale=0.1), rand(n, seed=4)
    qi.qi_linear_act(ctx, a, qi.bf16_struct(w, b), qi.QI_ACT_SILU, residual=res, y=y)
    ctx.check()
    at = torch.cat([torch.arange(0, M, 997), torch.arange(2 ** 31 // ld - 300, 2 ** 31 // ld + 300),
                    torch.arange(2 ** 30 // ld - 300, 2 ** 30 // ld + 300), torch.arange(M - 300, M)]).cuda()
    A = a[at].double()
    ref = A @ w.double().T + b.double()
    ref = ref * torch.sigmoid(ref)
    tol = acc_tol(A, w.double()) + 2.0 ** -16 * ref.abs()
    ref = ref + res[at].double()
    assert ((y[at].double() - ref).abs() <= tol + U * ref.abs()).all()
    assert not block[:, 128 + shift + n:256].any() and not block[:, 64:128 + shift].any()


def test_gated_ffn_buffers_past_2_to_31_values(ctx):
    """Hidden values, saved gate | up and the backward scratch past 2^31 values: rows on
    both sides of the border, and gradients of the weights that come from them alone."""
    M, H, F = 140000, 64, 16384
    border = 2 ** 31 // F                      # row of h that begins at value 2^31
    x = rand(M, H, seed=1)
    wg, wu, wd = rand(F, H, seed=2, scale=H ** -0.5), rand(F, H, seed=3, scale=H ** -0.5), rand(H, F, seed=4,
                                                                                           scale=F ** -0.5)
    ffn = qi.gated_ffn_struct(wg, wu, wd)
    y, saved = qi.qi_gated_ffn_forward(ctx, ffn, x, save=True)
    at = torch.cat([torch.arange(0, 300), torch.arange(border // 2 - 150, border // 2 + 150),
                    torch.arange(border - 150, border + 150), torch.arange(M - 300, M)]).cuda()
    dy = torch.zeros(M, H, dtype=BF, device="cuda")
    dy[at] = rand(len(at), H, seed=5)
    got = qi.qi_gated_ffn_backward(ctx, ffn, x, dy, saved)
    ctx.check()
    X, Y, G, W, D = x[at].double(), dy[at].double(), wg.double(), wu.double(), wd.double()
    g, u = X @ G.T, X @ W.T
    tg, tu = acc_tol(X, G), acc_tol(X, W)
    assert ((saved[at, :F].double() - g).abs() <= tg).all() and ((saved[at, F:].double() - u).abs() <= tu).all()
    g, u = saved[at, :F].double(), saved[at, F:].double()
    s = torch.sigmoid(g)
    act, slope = g * s, s * (1 + g * (1 - s))
    h, th = act * u, (U + 2.0 ** -16) * (act * u).abs()
    ref = h @ D.T
    tol = th @ D.abs().T + acc_tol(h, D) * (1 + U)
    assert ((y[at].double() - ref).abs() <= tol + U * (ref.abs() + tol)).all()
    # one rounding of dg, du and h to bf16, 2^-16 for the activations (the slope: 2^-17 of its terms, below
    # 1.2 (1 + |g|)), the fp32 sums, one rounding of each gradient
    eps = U * (1 + U) + 2.0 ** -16
    dh, tdh = Y @ D, acc_tol(Y, D.T)
    dg, tdg = dh * u * slope, (eps * slope.abs() + 2.0 ** -17 * 1.2 * (1 + g.abs())) * (dh * u).abs() + tdh * (u * slope).abs()
    du, tdu = dh * act, eps * (dh * act).abs() + tdh * act.abs()
    h, th = act * u, eps * (act * u).abs()
    rows = 2.0 ** -23 * (M / 16 + 2) * 1.13    # sums over all M rows, of which the others are 0
    refs = [(dg @ G + du @ W, tdg @ G.abs() + tdu @ W.abs() + acc_tol(dg, G.T) + acc_tol(du, W.T)),
            (dg.T @ X, tdg.T @ X.abs() + rows * (dg.abs().T @ X.abs())),
            (du.T @ X, tdu.T @ X.abs() + rows * (du.abs().T @ X.abs())),
            (Y.T @ h, Y.abs().T @ th + rows * (Y.abs().T @ h.abs()))]
    for i, (t, (ref, tol)) in enumerate(zip(got, refs)):
        t = (t[at] if i == 0 else t).double()
        assert ((t - ref).abs() <= 1.01 * tol + U * (ref.abs() + tol) + 1e-30).all()
    assert not got[0][300:border // 2 - 150].any()      # dx of rows without a gradient


@pytest.mark.parametrize("M", [1, 12, 60, 300, 700, 1300])
@pytest.mark.parametrize("n", [1, 3, 131, 2301])
def test_linear_odd_outputs_in_aligned_rows(ctx, M, n):
    """An odd number of columns in rows that are 16-byte aligned (y and residual parts
    of padded buffers): nothing behind the last column is written."""
    k, pad = 136, -(-n // 8) * 8 + 8
    a, w, b = rand(M, k), rand(n, k, seed=1, scale=0.1), rand(n, seed=2)
    res, out = rand(M, pad, seed=3), rand(M + 1, pad, seed=4)
    before = out.clone()
    qi.qi_linear_act(ctx, a, qi.bf16_struct(w, b), qi.QI_ACT_SILU, residual=res[:, :n], y=out[:M, :n])
    ctx.check()
    ref = a.double() @ w.double().T + b.double()
    ref = ref * torch.sigmoid(ref)
    tol = acc_tol(a.double(), w.double()) + 2.0 ** -16 * ref.abs()
    ref = ref + res[:, :n].double()
    assert ((out[:M, :n].double() - ref).abs() <= tol + U * ref.abs()).all()
    assert same_bits(out[:M, n:], before[:M, n:]) and same_bits(out[M:], before[M:])
