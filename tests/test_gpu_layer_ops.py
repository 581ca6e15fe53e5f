"""The prompt-encoder layer operators against their formulas in 64 bits.

Tolerances are sums of the roundings that an output passes through, with
u = 2^-8, half a bf16 step relative to the value:
  Linear      u |y| + (fp32 sum)  with fp32 sum <= k/16 2^-23 sum |a w| (the
              tensor core adds 16 products at a time), times 1.13, the largest
              slope of the activations
  attention   u |o| for the output and u sum_j p_j |v_j| for the weights, which
              enter P V as bf16; scores and sums in fp32: 2^-12 of the same sum
  activations 2^-16 of the value: the exponent's argument is at most 128 before
              the result vanishes, its rounding 2^-24 of that
  feed-forward  u per rounded operand (h, dg, du), weighted by the absolute
              values of what it is multiplied with, and u of the output
"""
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


def within(got, ref, tol, what=""):
    got = got.double()
    assert torch.isfinite(got).all(), what
    over = ((got - ref).abs() - tol).max().item()
    assert over <= 0, f"{what}: off by {over:.3e} more than {tol.max().item():.3e}"


def same_bits(a, b):
    """Equal bit patterns (NaN equal to itself, unlike torch.equal)."""
    assert a.dtype == b.dtype
    return torch.equal(a.contiguous().view(torch.int16), b.contiguous().view(torch.int16))


# ------------------------------------------------------------------ attention

def table(rows):
    return torch.tensor(rows, dtype=torch.int32).reshape(-1, 4)


def packed(ql, kl):
    rows, a, b = [], 0, 0
    for x, y in zip(ql, kl):
        rows.append((a, x, b, y))
        a, b = a + x, b + y
    return table(rows), a, b


def attn_ref(q, k, v, spans, heads, kvh, scale=128 ** -0.5):
    """(o, sum_j p_j |v_j|) in 64 bits; rows outside every sequence are NaN."""
    G = heads // kvh
    o = torch.full((q.shape[0], heads * 128), float("nan"), dtype=torch.float64, device="cuda")
    mag = torch.zeros_like(o)
    for q0, ql, k0, kl in spans.tolist():
        i = torch.arange(ql, device="cuda")[:, None]
        j = torch.arange(kl, device="cuda")[None, :]
        see = j <= kl - ql + i
        for h in range(heads):
            Q = q[q0:q0 + ql, h * 128:h * 128 + 128].double()
            K = k[k0:k0 + kl, h // G * 128:h // G * 128 + 128].double()
            V = v[k0:k0 + kl, h // G * 128:h // G * 128 + 128].double()
            s = (Q @ K.T * scale).masked_fill(~see, -float("inf"))
            p = torch.softmax(s, -1).nan_to_num(0.0) if kl else s   # a row that sees nothing: 0
            c = slice(h * 128, h * 128 + 128)
            o[q0:q0 + ql, c] = p @ V
            mag[q0:q0 + ql, c] = p @ V.abs()
    return o, mag


def attn_tol(o, mag):
    return U * o.abs() + (U * (1 + U) + 2.0 ** -12) * mag + 1e-30


def check_attn(ctx, q, k, v, spans, heads, kvh, **kw):
    got = qi.qi_attn_causal_packed(ctx, q, k, v, spans, heads, kvh, **kw)
    ctx.check()
    o, mag = attn_ref(q, k, v, spans, heads, kvh, kw.get("sm_scale") or 128 ** -0.5)
    mine = ~o.isnan().any(1)
    within(got[mine], o[mine], attn_tol(o[mine], mag[mine]), "attention")
    return got


HEADS = [(4, 4), (8, 2), (7, 1), (6, 2), (16, 1), (5, 1), (128, 1)]


@pytest.mark.parametrize("heads,kvh", HEADS)
def test_attention_ragged_prompts(ctx, heads, kvh):
    """Whole prompts around tile edges, empty ones among them."""
    ql = [1, 0, 17, 31, 32, 33, 64, 65, 127, 128, 129, 200, 3]
    spans, nq, nk = packed(ql, ql)
    check_attn(ctx, rand(nq, heads * 128), rand(nk, kvh * 128, seed=1), rand(nk, kvh * 128, seed=2),
               spans, heads, kvh)


@pytest.mark.parametrize("heads,kvh", [(8, 2), (7, 1), (4, 4)])
def test_attention_behind_cached_keys(ctx, heads, kvh):
    """Prompts and single tokens behind cached keys; more queries than keys (the
    first ones see nothing: zeros); no keys at all."""
    ql = [1, 5, 40, 1, 130, 9, 70, 4, 1]
    kl = [1, 260, 140, 515, 131, 4, 1, 0, 0]
    spans, nq, nk = packed(ql, kl)
    got = check_attn(ctx, rand(nq, heads * 128), rand(nk, kvh * 128, seed=1),
                     rand(nk, kvh * 128, seed=2), spans, heads, kvh)
    for q0, a, _, b in spans.tolist():
        if a > b:
            assert (got[q0:q0 + a - b] == 0).all()
    none = table([(0, 3, 0, 0)])
    empty = torch.empty(0, kvh * 128, dtype=BF, device="cuda")
    got = qi.qi_attn_causal_packed(ctx, rand(3, heads * 128), empty, empty, none, heads, kvh)
    ctx.check()
    assert (got == 0).all()


@pytest.mark.parametrize("ql,kl", [([1], [4096]), ([1], [8191]), ([1, 1, 1], [9000, 3, 2500]),
                                   ([2, 40], [6001, 3000]), ([300], [5000])])
@pytest.mark.parametrize("heads,kvh", [(8, 2), (3, 1)])
def test_attention_split_over_keys(ctx, ql, kl, heads, kvh):
    """Few queries, many keys: the key range is split over CTAs and joined; the
    result has the same bits every time and does not depend on what the
    workspace held."""
    spans, nq, nk = packed(ql, kl)
    n = qi.qi_attn_causal_packed_workspace_bytes(ctx, spans, heads, kvh)
    assert n > 0
    q, k, v = rand(nq, heads * 128), rand(nk, kvh * 128, seed=1), rand(nk, kvh * 128, seed=2)
    got = check_attn(ctx, q, k, v, spans, heads, kvh)
    ws = torch.full((n,), 255, dtype=torch.uint8, device="cuda")   # NaN patterns
    again = qi.qi_attn_causal_packed(ctx, q, k, v, spans, heads, kvh, workspace=ws)
    ctx.check()
    assert same_bits(got, again)


def test_attention_many_sequences_share_keys(ctx):
    """The largest table, out of order, all tokens reading one shared prefix."""
    heads, kvh, n = 8, 2, qi.QI_MAX_SEQS
    g = torch.Generator().manual_seed(5)
    ql = torch.randint(0, 4, (n,), generator=g).tolist()
    start = np.concatenate([[0], np.cumsum(ql)])[:-1]
    rows = [(int(start[i]), ql[i], int(i % 7), 40 + (i * 13) % 300) for i in range(n)]
    rows = [rows[i] for i in torch.randperm(n, generator=g)]
    check_attn(ctx, rand(sum(ql), heads * 128), rand(400, kvh * 128, seed=1),
               rand(400, kvh * 128, seed=2), table(rows), heads, kvh)


@pytest.mark.parametrize("heads,kvh", [(8, 2), (3, 1), (32, 1), (40, 1), (96, 1)])
def test_attention_short_sequences_beside_long_ones(ctx, heads, kvh):
    """Single tokens, some behind a few keys and some behind thousands, in one table
    with prompts: more units of work than an ordered list holds, and fewer."""
    for tokens in (6, qi.QI_MAX_SEQS - 4):
        ql = [1] * tokens + [700, 128, 33, 0]
        kl = [1 + (i * 97) % 400 for i in range(tokens - 3)] + [2048, 2049, 5000, 700, 900, 33, 0]
        spans, nq, nk = packed(ql, kl)
        got = check_attn(ctx, rand(nq, heads * 128), rand(nk, kvh * 128, seed=1), rand(nk, kvh * 128, seed=2),
                         spans, heads, kvh)
        assert got.shape == (nq, heads * 128)


def test_attention_fused_rows_and_strides(ctx):
    """q, k, v as column ranges of one fused block, o into a wider padded buffer:
    the columns and rows around the result stay as they were."""
    heads, kvh = 8, 2
    ql, kl = [50, 1, 190], [50, 70, 190]
    spans = table([(3, 50, 0, 50), (60, 1, 100, 70), (70, 190, 200, 190)])
    block = rand(400, (heads + 2 * kvh) * 128 + 8, seed=3)
    q = block[:, :heads * 128]
    k = block[:, heads * 128:(heads + kvh) * 128]
    v = block[:, (heads + kvh) * 128:(heads + 2 * kvh) * 128]
    wide = torch.full((400, heads * 128 + 64), 7.0, dtype=BF, device="cuda")
    o = wide[:, 32:32 + heads * 128]
    check_attn(ctx, q, k, v, spans, heads, kvh, o=o)
    mine = torch.zeros(400, dtype=torch.bool)
    for q0, a, _, _ in spans.tolist():
        mine[q0:q0 + a] = True
    assert (wide[~mine.cuda()] == 7).all()
    assert (wide[:, :32] == 7).all() and (wide[:, 32 + heads * 128:] == 7).all()


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_attention_rows_outside_a_sequence_do_not_matter(ctx, bad):
    """Key rows before, between and behind the sequences (unwritten cache rows, a
    neighbour's) may hold anything, inside tiles that the sequences use too."""
    heads, kvh = 8, 2
    spans = table([(0, 30, 5, 30), (30, 1, 64, 77), (31, 140, 200, 333), (171, 2, 600, 3), (173, 1, 700, 4099)])
    q = rand(174, heads * 128)
    k, v = rand(5000, kvh * 128, seed=1), rand(5000, kvh * 128, seed=2)
    mine = torch.zeros(5000, dtype=torch.bool, device="cuda")
    for _, _, k0, n in spans.tolist():
        mine[k0:k0 + n] = True
    clean = check_attn(ctx, q, k, v, spans, heads, kvh)
    k[~mine] = bad
    v[~mine] = bad
    got = qi.qi_attn_causal_packed(ctx, q, k, v, spans, heads, kvh)
    ctx.check()
    assert same_bits(got, clean)


def test_attention_bad_queries_stay_in_their_row(ctx):
    """A query row that is not finite makes its own row not finite and no other."""
    heads, kvh, n = 8, 2, 70
    spans = table([(0, n, 0, n)])
    q, k, v = rand(n, heads * 128), rand(n, kvh * 128, seed=1), rand(n, kvh * 128, seed=2)
    clean = check_attn(ctx, q, k, v, spans, heads, kvh)
    q[33] = float("nan")
    got = qi.qi_attn_causal_packed(ctx, q, k, v, spans, heads, kvh)
    ctx.check()
    assert got[33].isnan().all()
    rest = [i for i in range(n) if i != 33]
    assert same_bits(got[rest], clean[rest])


def test_attention_large_scores(ctx):
    """Scores that grow along the keys by far more than the range of exp: the
    reference maximum moves many times."""
    heads, kvh, n = 4, 1, 700
    spans = table([(0, n, 0, n), (n, 1, 0, n)])
    q, k = rand(n + 1, heads * 128, scale=4.0), rand(n, kvh * 128, seed=1, scale=4.0)
    k *= torch.linspace(0.01, 3, n, device="cuda").to(BF)[:, None]
    check_attn(ctx, q, k, rand(n, kvh * 128, seed=2), spans, heads, kvh)
    check_attn(ctx, q, k, rand(n, kvh * 128, seed=2), spans, heads, kvh, sm_scale=1e-4)


def test_attention_long_prompt(ctx):
    """A prompt of many tiles, every row against the formula."""
    heads, kvh, n = 8, 2, 5003
    spans = table([(0, n, 0, n)])
    q, k, v = rand(n, heads * 128), rand(n, kvh * 128, seed=1), rand(n, kvh * 128, seed=2)
    check_attn(ctx, q, k, v, spans, heads, kvh)


def test_attention_offsets_past_32_bits(ctx):
    """Key rows whose offset in the buffer passes 2^31 values and 2^32 bytes."""
    heads, kvh, ld, rows = 2, 1, 4096, 530000
    cache = torch.empty(rows, ld, dtype=BF, device="cuda")
    k, v = cache[:, :128], cache[:, 128:256]
    k[rows - 900:], v[rows - 900:] = rand(900, 128, seed=1), rand(900, 128, seed=2)
    spans = table([(0, 200, rows - 300, 300), (200, 1, rows - 900, 900)])
    q = rand(201, heads * 128)
    got = qi.qi_attn_causal_packed(ctx, q, k, v, spans, heads, kvh)
    near = table([(0, 200, 600, 300), (200, 1, 0, 900)])
    want = qi.qi_attn_causal_packed(ctx, q, rand(900, 128, seed=1), rand(900, 128, seed=2), near, heads, kvh)
    ctx.check()
    assert same_bits(got, want)


def test_attention_captured_and_replayed(ctx):
    """A captured call (split and unsplit sequences) replays on new contents of the
    same buffers; two graphs may share one workspace."""
    heads, kvh = 8, 2
    spans, nq, nk = packed([1, 90, 1], [5000, 90, 33])
    n = qi.qi_attn_causal_packed_workspace_bytes(ctx, spans, heads, kvh)
    ws = torch.empty(max(n, 16), dtype=torch.uint8, device="cuda")
    bufs, graphs = [], []
    for i in range(2):
        q, k, v = rand(nq, heads * 128), rand(nk, kvh * 128, seed=1), rand(nk, kvh * 128, seed=2)
        o = torch.zeros(nq, heads * 128, dtype=BF, device="cuda")
        qi.qi_attn_causal_packed(ctx, q, k, v, spans, heads, kvh, o=o, workspace=ws)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            qi.qi_attn_causal_packed(ctx, q, k, v, spans, heads, kvh, o=o, workspace=ws)
        bufs.append((q, k, v, o))
        graphs.append(g)
    for rnd in range(2):
        for i, (q, k, v, o) in enumerate(bufs):
            q.copy_(rand(nq, heads * 128, seed=20 + i + rnd))
            v.copy_(rand(nk, kvh * 128, seed=30 + i + rnd))
            o.zero_()
        graphs[0].replay()
        graphs[1].replay()
        torch.cuda.synchronize()
        ctx.check()
        for q, k, v, o in bufs:
            want = qi.qi_attn_causal_packed(ctx, q, k, v, spans, heads, kvh)
            torch.cuda.synchronize()
            assert same_bits(o, want)


def test_attention_two_streams(ctx):
    """Two calls at once on two streams, each with its own workspace."""
    heads, kvh = 8, 2
    spans, nq, nk = packed([1, 200], [7000, 300])
    other = qi.Context()
    work = []
    for i, c in enumerate((ctx, other)):
        q, k, v = (rand(nq, heads * 128, seed=i), rand(nk, kvh * 128, seed=5 + i), rand(nk, kvh * 128, seed=9 + i))
        want = check_attn(c, q, k, v, spans, heads, kvh)
        work.append((c, q, k, v, want, torch.cuda.Stream()))
    torch.cuda.synchronize()
    outs = [[] for _ in work]
    for _ in range(5):
        for i, (c, q, k, v, want, st) in enumerate(work):
            outs[i].append(qi.qi_attn_causal_packed(c, q, k, v, spans, heads, kvh, stream=st))
    torch.cuda.synchronize()
    for got, (c, _, _, _, want, st) in zip(outs, work):
        c.check(st)
        assert all(same_bits(g, want) for g in got)
    other.close()


# ------------------------------------------------------------------ Linear

def act64(x, act):
    if act == qi.QI_ACT_SILU:
        return x * torch.sigmoid(x)
    if act == qi.QI_ACT_GELU_TANH:
        # 0.5 (1 + tanh z) = logistic(2 z), without the cancellation of 1 + tanh z at z << 0
        return x * torch.sigmoid(2 * (2 / np.pi) ** 0.5 * (x + 0.044715 * x ** 3))
    return x


def act64_grad(x, act):
    x = x.detach().requires_grad_(True)
    with torch.enable_grad():
        return torch.autograd.grad(act64(x, act).sum(), x)[0]


def acc_tol(a, b):
    """fp32 sum of a @ b^T (64-bit inputs): see the module's first lines."""
    k = a.shape[1]
    return 1.13 * (k / 16 + 2) * 2.0 ** -23 * (a.abs() @ b.abs().T)


def check_linear(ctx, a, w, bias, act, res=None, **kw):
    y = qi.qi_linear_act(ctx, a, qi.bf16_struct(w, bias), act, residual=res, **kw)
    ctx.check()
    ref = act64(a.double() @ w.double().T + (bias.double() if bias is not None else 0), act)
    tol = acc_tol(a.double(), w.double()) + 2.0 ** -16 * ref.abs()
    if res is not None:
        ref = ref + res.double()
    within(y, ref, tol + U * ref.abs() + 1e-30, "linear")
    return y


@pytest.mark.parametrize("M", [1, 2, 8, 9, 16, 17, 64, 127, 128, 129, 300, 768])
@pytest.mark.parametrize("n,k", [(256, 64), (40, 200), (1000, 1032), (1536, 512)])
def test_linear_shapes(ctx, M, n, k):
    a, w, b = rand(M, k), rand(n, k, seed=1, scale=0.05), rand(n, seed=2)
    check_linear(ctx, a, w, b, qi.QI_ACT_NONE)
    check_linear(ctx, a, w, None, qi.QI_ACT_SILU, rand(M, n, seed=3))
    check_linear(ctx, a, w, b, qi.QI_ACT_GELU_TANH, rand(M, n, seed=4))


@pytest.mark.parametrize("M", [7, 16, 20, 24, 25, 31, 32, 33, 95, 250, 257, 400])
@pytest.mark.parametrize("n,k", [(8, 8), (24, 72), (200, 128), (256, 192), (520, 4096), (2000, 520), (6000, 264)])
def test_linear_few_rows(ctx, M, n, k):
    """Around the last row counts that stream the weights, and sizes whose K is shared
    by several CTAs: fewer pieces of K than CTAs, unequal shares, two tiles of rows."""
    a, w, b = rand(M, k), rand(n, k, seed=1, scale=0.05), rand(n, seed=2)
    check_linear(ctx, a, w, b, qi.QI_ACT_SILU, rand(M, n, seed=3))
    check_linear(ctx, a, w, None, qi.QI_ACT_NONE)


@pytest.mark.parametrize("M", [1, 5, 40, 260, 777])
@pytest.mark.parametrize("n", [1, 3, 33, 255, 257, 1001])
def test_linear_odd_outputs(ctx, M, n):
    """Any n and any row distance of y and residual: odd ones have unaligned rows."""
    k = 136
    a, w, b = rand(M, k), rand(n, k, seed=1, scale=0.1), rand(n, seed=2)
    check_linear(ctx, a, w, b, qi.QI_ACT_SILU, rand(M, n, seed=3))
    wide = torch.full((M, n + 5), 3.0, dtype=BF, device="cuda")
    res = rand(M, n + 2, seed=5)[:, 1:1 + n]
    check_linear(ctx, a, w, b, qi.QI_ACT_NONE, res, y=wide[:, 2:2 + n])
    assert (wide[:, :2] == 3).all() and (wide[:, 2 + n:] == 3).all()


@pytest.mark.parametrize("M,n,k", [(1, 4096, 4096), (3, 4096, 16384), (768, 6144, 4096),
                                   (200, 2048, 8192), (4608, 4096, 1024), (50, 12001, 1024)])
def test_linear_full_width(ctx, M, n, k):
    check_linear(ctx, rand(M, k), rand(n, k, seed=1, scale=0.02), rand(n, seed=2, scale=0.02),
                 qi.QI_ACT_GELU_TANH, rand(M, n, seed=3))


@pytest.mark.parametrize("M,n", [(600, 1100), (1300, 1100), (1000, 2300), (520, 4000), (1100, 130)])
def test_linear_tile_widths(ctx, M, n):
    """Sizes whose tiles are 256, 192 or 128 columns wide, with cut last tiles."""
    a, w, b = rand(M, 520), rand(n, 520, seed=1, scale=0.05), rand(n, seed=2)
    check_linear(ctx, a, w, b, qi.QI_ACT_SILU, rand(M, n, seed=3))


@pytest.mark.parametrize("M", [1, 12, 70, 513])
def test_linear_in_place_strided_and_zero_rows(ctx, M):
    """residual == y, strided rows of a, rows behind the last one untouched."""
    n, k = 384, 320
    block = rand(M + 3, 2 * k, seed=7)
    a = block[:M, k:]
    w, b = rand(n, k, seed=1, scale=0.05), rand(n, seed=2)
    y = rand(M + 2, n, seed=9)
    before = y.clone()
    want = check_linear(ctx, a, w, b, qi.QI_ACT_NONE, before[:M].clone())
    qi.qi_linear_act(ctx, a, qi.bf16_struct(w, b), qi.QI_ACT_NONE, residual=y[:M], y=y[:M])
    qi.qi_linear_act(ctx, a[:0], qi.bf16_struct(w, b), qi.QI_ACT_NONE, residual=y[:0], y=y[:0])
    ctx.check()
    assert same_bits(y[:M], want) and same_bits(y[M:], before[M:])


def test_linear_bits_do_not_depend_on_earlier_calls(ctx):
    """The choice of kernel goes by the sizes alone: a product gives the same bits
    before and after others of its kind."""
    sizes = [(64, 4096, 4096), (40, 520, 4096), (200, 2048, 2048), (300, 1024, 2816), (600, 1500, 1024)]
    ops = [(rand(M, k), qi.bf16_struct(rand(n, k, seed=1, scale=0.02))) for M, n, k in sizes]
    first = [qi.qi_linear_act(ctx, a, w) for a, w in ops]
    again = [qi.qi_linear_act(ctx, a, w) for a, w in reversed(ops)][::-1]
    ctx.check()
    assert all(same_bits(x, y) for x, y in zip(first, again))


def test_linear_activations_at_the_ends(ctx):
    """Large values of both signs: the activations reach x and 0, not NaN."""
    x = torch.tensor([0.0, -0.0, 1e-3, 8.0, -8.0, 40.0, -40.0, 100.0, -100.0, 3e4, -3e4, 1e30, -1e30, 3e38, -3e38],
                     device="cuda").to(BF)
    for M in (1, 40):
        a = torch.zeros(M, 16, dtype=BF, device="cuda")
        a[:, 0] = 1
        w = torch.zeros(len(x), 16, dtype=BF, device="cuda")
        w[:, 0] = x
        for act in (qi.QI_ACT_SILU, qi.QI_ACT_GELU_TANH):
            y = qi.qi_linear_act(ctx, a, qi.bf16_struct(w), act)
            ctx.check()
            ref = act64(x.double(), act).nan_to_num(0.0)
            within(y, ref.expand(M, -1), (U + 2.0 ** -18) * ref.abs().expand(M, -1) + 1e-30, "ends")


# ------------------------------------------------------------------ gated feed-forward block

def ffn_case(M, H, F, seed=0):
    # weights N(0, 1/fan in): pre-activations of size 1
    return (rand(M, H, seed=seed), rand(F, H, seed=seed + 1, scale=H ** -0.5),
            rand(F, H, seed=seed + 2, scale=H ** -0.5), rand(H, F, seed=seed + 3, scale=F ** -0.5))


def check_forward(ctx, x, wg, wu, wd, act, res=None, **kw):
    w = qi.gated_ffn_struct(wg, wu, wd, act)
    y, gu = qi.qi_gated_ffn_forward(ctx, w, x, residual=res, save=True, **kw)
    ctx.check()
    F = wg.shape[0]
    X, G, Uw, D = x.double(), wg.double(), wu.double(), wd.double()
    g, u = X @ G.T, X @ Uw.T
    tg, tu = acc_tol(X, G), acc_tol(X, Uw)
    assert gu.dtype == torch.float32
    within(gu[:, :F], g, tg + 1e-30, "gate")     # kept in fp32: no rounding but the sum's
    within(gu[:, F:], u, tu + 1e-30, "up")
    a = act64(g, act)
    h = a * u
    th = U * h.abs() + 2.0 ** -16 * h.abs() + tg * u.abs() + tu * a.abs() + tg * tu
    ref = h @ D.T
    tol = th @ D.abs().T + acc_tol(h, D) * (1 + U)
    if res is not None:
        ref = ref + res.double()
    within(y, ref, tol + U * (ref.abs() + tol) + 1e-30, "ffn")
    only = qi.qi_gated_ffn_forward(ctx, w, x, residual=res)
    ctx.check()
    assert same_bits(only, y)      # saving for the backward pass changes nothing
    return w, y, gu


def check_backward(ctx, w, x, wg, wu, wd, act, gu, dy):
    F = wg.shape[0]
    got = qi.qi_gated_ffn_backward(ctx, w, x, dy, gu)
    ctx.check()
    X, G, Uw, D, Y = x.double(), wg.double(), wu.double(), wd.double(), dy.double()
    g, u = gu[:, :F].double(), gu[:, F:].double()
    a, da = act64(g, act), act64_grad(g, act)
    dh, th = Y @ D, acc_tol(Y, D.T)
    eps = U * (1 + U) + 2.0 ** -16     # one rounding to bf16; the activations' fp32 evaluation
    # act' near its zero is a difference: its error is 2^-17 of the terms, which are below 1.2 (1 + |g|)
    dg, tdg = dh * u * da, (eps * da.abs() + 2.0 ** -17 * 1.2 * (1 + g.abs())) * (dh * u).abs() + th * (u * da).abs()
    du, tdu = dh * a, eps * (dh * a).abs() + th * a.abs()
    h, thh = a * u, eps * (a * u).abs()
    refs = dict(dx=(dg @ G + du @ Uw, tdg @ G.abs() + tdu @ Uw.abs() + acc_tol(dg, G.T) + acc_tol(du, Uw.T)),
                dgate=(dg.T @ X, tdg.T @ X.abs() + acc_tol(dg.T, X.T)),
                dup=(du.T @ X, tdu.T @ X.abs() + acc_tol(du.T, X.T)),
                ddown=(Y.T @ h, Y.abs().T @ thh + acc_tol(Y.T, h.T)))
    for t, (name, (ref, tol)) in zip(got, refs.items()):
        within(t, ref, 1.01 * tol + U * (ref.abs() + tol) + 1e-30, name)
    return dict(zip(refs, got))


SHAPES = [(1, 64, 128), (16, 200, 72), (25, 136, 328), (32, 520, 200), (33, 64, 4096), (40, 4096, 64), (9, 64, 8192), (17, 256, 520), (100, 512, 1384), (333, 1024, 2816), (129, 8, 8),
          (700, 1032, 264), (780, 264, 2000)]


@pytest.mark.parametrize("act", [qi.QI_ACT_SILU, qi.QI_ACT_GELU_TANH])
@pytest.mark.parametrize("M,H,F", SHAPES)
def test_gated_ffn_forward_and_backward(ctx, M, H, F, act):
    x, wg, wu, wd = ffn_case(M, H, F)
    w, y, gu = check_forward(ctx, x, wg, wu, wd, act, rand(M, H, seed=8))
    check_backward(ctx, w, x, wg, wu, wd, act, gu, rand(M, H, seed=9))


@pytest.mark.parametrize("M,H,F", [(1, 4096, 11008), (12, 4096, 11008), (768, 4096, 11008), (1500, 2048, 5504)])
def test_gated_ffn_full_width(ctx, M, H, F):
    x, wg, wu, wd = ffn_case(M, H, F)
    w, y, gu = check_forward(ctx, x, wg, wu, wd, qi.QI_ACT_SILU, rand(M, H, seed=8))
    if M > 16:
        check_backward(ctx, w, x, wg, wu, wd, qi.QI_ACT_SILU, gu, rand(M, H, seed=9))


@pytest.mark.parametrize("act", [qi.QI_ACT_SILU, qi.QI_ACT_GELU_TANH])
def test_gated_ffn_gradients_against_differences(ctx, act):
    """sum(dy y) along a direction of x and of each weight, by central differences of
    the 64-bit forward, against the gradients.  Step e = 1e-4: the difference is off
    by e^2 (1e-8) relative; the gradients by their roundings, which add up in the
    inner product with a random direction like their absolute values at most."""
    M, H, F = 60, 128, 264
    x, wg, wu, wd = ffn_case(M, H, F)
    w = qi.gated_ffn_struct(wg, wu, wd, act)
    dy = rand(M, H, seed=9)
    _, gu = qi.qi_gated_ffn_forward(ctx, w, x, save=True)
    got = qi.qi_gated_ffn_backward(ctx, w, x, dy, gu)
    ctx.check()
    at = [t.double() for t in (x, wg, wu, wd)]

    def loss(p):
        X, G, Uw, D = p
        return ((act64(X @ G.T, act) * (X @ Uw.T)) @ D.T * dy.double()).sum().item()

    for i, grad in enumerate(got):
        d = rand(*at[i].shape, seed=40 + i).double()
        e = 1e-4
        hi, lo = list(at), list(at)
        hi[i], lo[i] = at[i] + e * d, at[i] - e * d
        diff = (loss(hi) - loss(lo)) / (2 * e)
        # roundings: gate_up, dg / du / h and the gradient itself, 4 u each at most relative
        # to products of absolute values, which exceed |gradient| by the cancellation in its
        # sum: sqrt(rows summed) for random signs
        n = max(H, F, M)
        tol = 4 * U * n ** 0.5 * (grad.double() * d).norm().item()
        assert abs(diff - (grad.double() * d).sum().item()) <= tol + 1e-6 * abs(diff)


@pytest.mark.parametrize("M,H,F", [(300, 256, 520), (1100, 512, 1384)])
def test_gated_ffn_gradients_keep_their_precision(ctx, M, H, F):
    """Relative error (2-norm) of every gradient against 64 bits.  What rounds: the
    gradient itself, and dg, du or h as an operand; g and u do not.  A rounding to
    bf16 is off by 2^-8 times a uniform number in (-1, 1) relative to the power of
    two below the value: 2^-8 / sqrt(3) at 1, half that at 2, and with the values
    spread over that octave sqrt(1 / ln 16) = 0.60 of it in the mean square,
    1.36e-3 of the value; at most 2^-8 / sqrt(3) = 2.26e-3 whatever the spread.
    Two of them in quadrature: 3.19e-3 at most.  g and u rounded too would add
    two or three more."""
    x, wg, wu, wd = ffn_case(M, H, F)
    w = qi.gated_ffn_struct(wg, wu, wd)
    dy = rand(M, H, seed=9)
    _, gu = qi.qi_gated_ffn_forward(ctx, w, x, save=True)
    got = qi.qi_gated_ffn_backward(ctx, w, x, dy, gu)
    ctx.check()
    X, G, Uw, D, Y = x.double(), wg.double(), wu.double(), wd.double(), dy.double()
    g, u = X @ G.T, X @ Uw.T
    dh = Y @ D
    dg, du = dh * u * act64_grad(g, qi.QI_ACT_SILU), dh * act64(g, qi.QI_ACT_SILU)
    refs = (dg @ G + du @ Uw, dg.T @ X, du.T @ X, Y.T @ (act64(g, qi.QI_ACT_SILU) * u))
    for t, ref in zip(got, refs):
        assert ((t.double() - ref).norm() / ref.norm()).item() <= 3.19e-3


def test_gated_ffn_wanted_gradients_strides_and_zero_rows(ctx):
    M, H, F, act = 90, 256, 512, qi.QI_ACT_SILU
    x, wg, wu, wd = ffn_case(M, H, F)
    w = qi.gated_ffn_struct(wg, wu, wd, act)
    dy = rand(M, H, seed=9)
    y, gu = qi.qi_gated_ffn_forward(ctx, w, x, save=True)
    full = dict(zip(("dx", "dgate", "dup", "ddown"), qi.qi_gated_ffn_backward(ctx, w, x, dy, gu)))
    ctx.check()
    for want in (("dx",), ("dgate",), ("dup", "ddown"), ("ddown",), ("dx", "dup")):
        part = dict(zip(full, qi.qi_gated_ffn_backward(ctx, w, x, dy, gu, want=want)))
        ctx.check()
        for name, t in part.items():
            assert (t is None) == (name not in want)
            assert t is None or same_bits(t, full[name])
    # strided rows in and out
    xs = torch.full((M, H + 64), float("nan"), dtype=BF, device="cuda")
    ds, ys, os = xs.clone(), xs.clone(), xs.clone()
    xs[:, :H], ds[:, 8:8 + H] = x, dy
    y2, gu2 = qi.qi_gated_ffn_forward(ctx, w, xs[:, :H], y=ys[:, 16:16 + H], save=True)
    got = qi.qi_gated_ffn_backward(ctx, w, xs[:, :H], ds[:, 8:8 + H], gu2, dx=os[:, :H])
    ctx.check()
    assert same_bits(ys[:, 16:16 + H], y) and same_bits(gu2, gu)
    assert ys[:, :16].isnan().all() and ys[:, 16 + H:].isnan().all() and os[:, H:].isnan().all()
    for a, b in zip(got, full.values()):
        assert same_bits(a, b)
    # no rows: weight gradients are sums over nothing
    dx, dg, du, dd = qi.qi_gated_ffn_backward(ctx, w, x[:0], dy[:0], gu[:0])
    assert dx.shape == (0, H) and not dg.any() and not du.any() and not dd.any()
    assert qi.qi_gated_ffn_forward(ctx, w, x[:0]).shape == (0, H)
    # in place: y = x + block(x)
    z = x.clone()
    qi.qi_gated_ffn_forward(ctx, w, z, residual=z, y=z)
    want = qi.qi_gated_ffn_forward(ctx, w, x, residual=x)
    ctx.check()
    assert same_bits(z, want)


def test_gated_ffn_rows_do_not_mix(ctx):
    """A row that is not finite stays in its row of the forward pass and of dx."""
    M, H, F = 40, 128, 256
    x, wg, wu, wd = ffn_case(M, H, F)
    w = qi.gated_ffn_struct(wg, wu, wd)
    clean = qi.qi_gated_ffn_forward(ctx, w, x)
    x[7] = float("nan")
    y, gu = qi.qi_gated_ffn_forward(ctx, w, x, save=True)
    dx = qi.qi_gated_ffn_backward(ctx, w, x, rand(M, H, seed=9), gu, want=("dx",))[0]
    ctx.check()
    rest = [i for i in range(M) if i != 7]
    assert y[7].isnan().all() and same_bits(y[rest], clean[rest])
    assert dx[7].isnan().all() and torch.isfinite(dx[rest]).all()


def test_gated_ffn_captured_backward(ctx):
    """Forward and backward captured into one graph and replayed on new inputs."""
    M, H, F = 80, 256, 384
    x, wg, wu, wd = ffn_case(M, H, F)
    w = qi.gated_ffn_struct(wg, wu, wd)
    dy = rand(M, H, seed=9)

    def step():
        y, gu = qi.qi_gated_ffn_forward(ctx, w, x, save=True)
        return (y, *qi.qi_gated_ffn_backward(ctx, w, x, dy, gu))

    step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = step()
    for seed in (50, 51):
        x.copy_(rand(M, H, seed=seed))
        g.replay()
        torch.cuda.synchronize()
        ctx.check()
        for a, b in zip(out, step()):
            assert same_bits(a, b)


# ------------------------------------------------------------------ together

def rms64(x):
    return x * torch.rsqrt(x.pow(2).mean(-1, keepdim=True) + 1e-6)


def test_encoder_layer_of_packed_prompts(ctx):
    """One layer of a prompt encoder over a packed batch (a prompt, its negative
    prompt, an empty one), then one more token of each against the cached keys:
    the token's rows equal, within rounding, what the longer prompts give."""
    H, heads, kvh, F = 1024, 8, 2, 2816
    W, KW = heads * 128, kvh * 128
    lens = [150, 37, 0, 1]
    T = sum(lens)
    w = dict(qkv=rand(W + 2 * KW, H, seed=1, scale=H ** -0.5), b=rand(W + 2 * KW, seed=2, scale=0.1),
             out=rand(H, W, seed=3, scale=W ** -0.5))
    _, wg, wu, wd = ffn_case(1, H, F, seed=4)
    ffn = qi.gated_ffn_struct(wg, wu, wd)
    qkv_l, out_l = qi.bf16_struct(w["qkv"], w["b"]), qi.bf16_struct(w["out"])

    def layer(x, spans, cache=None):
        qkv = qi.qi_linear_act(ctx, rms64(x.double()).to(BF), qkv_l)
        q, k, v = qkv[:, :W], qkv[:, W:W + KW], qkv[:, W + KW:]
        if cache is not None:
            kc, vc, rows = cache
            kc[rows], vc[rows] = k, v
            k, v = kc, vc
        o = qi.qi_attn_causal_packed(ctx, q, k, v, spans, heads, kvh)
        x = qi.qi_linear_act(ctx, o, out_l, residual=x)
        return qi.qi_gated_ffn_forward(ctx, ffn, rms64(x.double()).to(BF), residual=x), (k, v)

    def layer64(x, spans):
        qkv = rms64(x).to(BF).double() @ w["qkv"].double().T + w["b"].double()
        q, k, v = qkv[:, :W], qkv[:, W:W + KW], qkv[:, W + KW:]
        x = x + attn_ref(q, k, v, spans, heads, kvh)[0] @ w["out"].double().T
        n = rms64(x)
        return x + (act64(n @ wg.double().T, qi.QI_ACT_SILU) * (n @ wu.double().T)) @ wd.double().T

    x = rand(T, H, seed=6)
    spans, _, _ = packed(lens, lens)
    y, _ = layer(x, spans)
    ctx.check()
    ref = layer64(x.double(), spans)
    # about eight roundings of relative size u/sqrt(3) each in quadrature on a residual stream
    # whose branches are of its own size
    assert ((y.double() - ref).norm() / ref.norm()).item() < 8 ** 0.5 * U
    # the last token of each prompt on its own, behind the cached keys of the others
    live = [n for n in lens if n]
    starts = np.concatenate([[0], np.cumsum(live)])[:-1]
    last = torch.tensor(starts + np.array(live) - 1, device="cuda")
    kc = torch.full((T + 50, KW), float("nan"), dtype=BF, device="cuda")
    vc = kc.clone()
    qkv = qi.qi_linear_act(ctx, rms64(x.double()).to(BF), qkv_l)
    kc[:T], vc[:T] = qkv[:, W:W + KW], qkv[:, W + KW:]
    kc[last], vc[last] = float("nan"), float("nan")
    one = table([(i, 1, int(starts[i]), live[i]) for i in range(len(live))])
    z, _ = layer(x[last].contiguous(), one, (kc, vc, last))
    ctx.check()
    assert ((z.double() - ref[last]).norm() / ref[last].norm()).item() < 8 ** 0.5 * U
