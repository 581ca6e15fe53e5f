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
