"""Further refusals of the prompt-encoder layer calls, on the host and before
anything is launched.  Run without a GPU: the calls get a zeroed stand-in for a
context (of which a check reads the SM count only) and pointers that nothing
may follow."""
import ctypes as C

import numpy as np
import pytest
import torch

from diffusion_transformer_text_dit_b200 import build_lib, qi

P = 1 << 20            # a 16-byte aligned address for pointers that must not be read
INV, SHAPE, ALIGN, WS = (qi.QI_ERR_INVALID_ARG, qi.QI_ERR_UNSUPPORTED_SHAPE, qi.QI_ERR_ALIGNMENT,
                         qi.QI_ERR_WORKSPACE)


@pytest.fixture(scope="module")
def L():
    build_lib.build()
    return qi.lib()


@pytest.fixture(scope="module")
def dummy():
    """Zeroed memory in the place of a context: device 0, 148 SMs."""
    buf = (C.c_int32 * 4096)()
    buf[1] = 148
    return buf


def attn(L, ctx, spans, **kw):
    t = np.asarray(spans, np.int32).reshape(-1, 4)
    a = dict(q=16 * P, ldq=512, q_rows=16, k=32 * P, ldk=256, v=48 * P, ldv=256, k_rows=8192, heads=4,
             kv_heads=2, scale=0.1, o=64 * P, ldo=512, ws=None, ws_bytes=0)
    a.update(kw)
    return L.qi_attn_causal_packed(C.addressof(ctx), a["q"], a["ldq"], a["q_rows"], a["k"], a["ldk"], a["v"],
                                   a["ldv"], a["k_rows"], a["heads"], a["kv_heads"], 128, t.ctypes.data, len(t),
                                   a["scale"], a["o"], a["ldo"], a["ws"], a["ws_bytes"], None)


def linear(L, ctx, **kw):
    a = dict(a=P, M=4, lda=64, w=2 * P, bias=None, n=40, k=64, act=0, res=None, ldr=0, y=3 * P, ldy=40)
    a.update(kw)
    w = qi.qi_linear_bf16()
    w.w, w.bias, w.n, w.k = a["w"], a["bias"], a["n"], a["k"]
    return L.qi_linear_act(C.addressof(ctx), a["a"], a["M"], a["lda"], C.byref(w), a["act"], a["res"], a["ldr"],
                           a["y"], a["ldy"], None)


def refused(got, code, text):
    """The code, and that the check in question gave it."""
    return got == code and text in qi.last_error()


@pytest.mark.parametrize("at", ["q", "k", "v", "o"])
@pytest.mark.parametrize("end", [False, True])
def test_attention_workspace_over_a_buffer(L, dummy, at, end):
    """Partial results over q, k, v or o: refused whether the workspace begins in the
    buffer or the buffer in the last bytes of the workspace."""
    t = np.array([[0, 1, 0, 8192]], np.int32)
    n = C.c_size_t()
    assert L.qi_attn_causal_packed_workspace_bytes(C.addressof(dummy), t.ctypes.data, 1, 4, 2, C.byref(n)) == qi.QI_OK
    base = dict(q=16 * P, k=32 * P, v=48 * P, o=64 * P)[at]
    ws = base - n.value + 16 if end else base + 128
    assert refused(attn(L, dummy, t, ws=ws, ws_bytes=n.value), INV, "workspace overlaps")


def test_linear_output_over_the_bias(L, dummy):
    for bias in (3 * P, 3 * P + 304, 3 * P - 64):
        assert refused(linear(L, dummy, bias=bias), INV, "y overlaps")


def test_linear_rows_at_odd_addresses(L, dummy):
    """Any row distance is taken, but a bf16 value lies at an even address."""
    assert refused(linear(L, dummy, y=3 * P + 1), ALIGN, "2-byte")
    assert refused(linear(L, dummy, res=4 * P + 1, ldr=40), ALIGN, "2-byte")
    assert refused(linear(L, dummy, y=3 * P + 1, res=3 * P + 1, ldr=40), ALIGN, "2-byte")


@pytest.mark.parametrize("span,heads,kvh", [((0, 2 ** 31 - 1, 0, 4), 1, 1), ((0, 2 ** 30 + 1, 0, 4), 1, 1),
                                            ((0, 1, 0, 2 ** 31 - 1), 1, 1), ((0, 1, 0, 2 ** 30), 4096, 4096)])
def test_attention_sizes_past_the_index_range(L, dummy, span, heads, kvh):
    """Lengths whose tiles or key ranges would not be counted in 32 bits."""
    t = np.array([span], np.int32)
    n = C.c_size_t()
    c = C.addressof(dummy)
    assert refused(L.qi_attn_causal_packed_workspace_bytes(c, t.ctypes.data, 1, heads, kvh, C.byref(n)), SHAPE, "2^")
    rows = 2 ** 31 - 1
    got = attn(L, dummy, t, heads=heads, kv_heads=kvh, q_rows=rows, k_rows=rows, ldq=heads * 128, ldo=heads * 128,
               ldk=kvh * 128, ldv=kvh * 128)
    assert refused(got, SHAPE, "2^")


def test_attention_plans_within_the_index_range(L, dummy):
    """A million keys behind each of many tokens that share them, and the longest prompt."""
    n = C.c_size_t()
    for spans, heads, kvh in (([(i, 1, 0, 1 << 20) for i in range(qi.QI_MAX_SEQS)], 64, 8),
                              ([(0, 1 << 20, 0, 1 << 20)], 32, 8)):
        t = np.array(spans, np.int32)
        assert L.qi_attn_causal_packed_workspace_bytes(C.addressof(dummy), t.ctypes.data, len(t), heads, kvh,
                                                       C.byref(n)) == qi.QI_OK
        # token ranges of 256 to 512 keys, each a partial result of G rows of 130 fp32 values
        if len(t) > 1:
            per_key = qi.QI_MAX_SEQS * heads * 130 * 4
            assert (1 << 20) // 512 * per_key <= n.value <= (1 << 20) // 256 * per_key
        else:
            assert n.value == 0


def test_product_sizes_past_the_index_range(L, dummy):
    big = 2 ** 30 + 8
    for kw in (dict(M=2 ** 31 - 1), dict(M=big), dict(n=2 ** 31 - 1, ldy=2 ** 31 - 1), dict(n=big, ldy=big),
               dict(k=big, lda=big)):
        assert refused(linear(L, dummy, **kw), SHAPE, "2^30")
    n = C.c_size_t()
    for hidden, mlp, M in ((big, 16, 4), (64, big // 2 + 4, 4), (64, 128, 2 ** 31 - 1)):
        w = qi.qi_gated_ffn()
        w.gate, w.up, w.down, w.hidden, w.mlp, w.act = P, 2 * P, 3 * P, hidden, mlp, qi.QI_ACT_SILU
        args = [C.addressof(dummy), C.byref(w), 4 * P, M, hidden]
        assert refused(L.qi_gated_ffn_workspace_bytes(C.byref(w), M, 0, C.byref(n)), SHAPE, "2^")
        assert refused(L.qi_gated_ffn_forward(*args, None, 0, 5 * P, hidden, None, 6 * P, 1 << 20, None), SHAPE, "2^")
        assert refused(L.qi_gated_ffn_backward(*args, 5 * P, hidden, 7 * P, None, 0, None, None, None, 6 * P, 1 << 20,
                                               None), SHAPE, "2^")


def test_columns_of_one_block_are_no_overlap(L, dummy):
    """Columns of one block of rows share no byte although their address ranges
    interleave: the calls get past the check (to the next one, of the workspace)."""
    ld = 512 + 256 + 256 + 512
    kw = dict(q=16 * P, k=16 * P + 1024, v=16 * P + 1536, q_rows=8192, k_rows=8192, ldq=ld, ldk=ld, ldv=ld, ldo=ld)
    t = [(0, 1, 0, 8192)]
    assert refused(attn(L, dummy, t, o=16 * P + 2048, **kw), WS, "workspace")
    # one row of queries, whose own distance says nothing
    assert refused(attn(L, dummy, t, o=16 * P + 2048, **dict(kw, q_rows=1, ldq=512, ldo=512)), WS, "workspace")
    w = qi.qi_gated_ffn()
    w.gate, w.up, w.down, w.hidden, w.mlp, w.act = P, 2 * P, 3 * P, 64, 128, qi.QI_ACT_SILU
    got = L.qi_gated_ffn_backward(C.addressof(dummy), C.byref(w), 4 * P, 4, 192, 4 * P + 256, 192, 7 * P, 4 * P + 128,
                                  192, None, None, None, None, 0, None)
    assert refused(got, WS, "workspace")


def test_columns_that_share_bytes_are_refused(L, dummy):
    """One column too many, behind the block's end and around it, and another row distance."""
    t = [(0, 4, 0, 4)]
    ld = 512 + 256 + 256 + 512
    kw = dict(q=16 * P, k=16 * P + 1024, v=16 * P + 1536, k_rows=16, ldq=ld, ldk=ld, ldv=ld, ldo=ld)
    for off in (2032, 2064, 2048 + 2 * ld + 16, 2048 - 16 - 2 * ld):
        assert refused(attn(L, dummy, t, o=16 * P + off, **kw), INV, "o overlaps")
    assert refused(attn(L, dummy, t, o=16 * P + 2048, **dict(kw, ldo=ld + 8)), INV, "o overlaps")
    w = qi.qi_gated_ffn()
    w.gate, w.up, w.down, w.hidden, w.mlp, w.act = P, 2 * P, 3 * P, 64, 128, qi.QI_ACT_SILU
    for off in (112, 144, 256):
        got = L.qi_gated_ffn_backward(C.addressof(dummy), C.byref(w), 4 * P, 4, 192, 4 * P + 256, 192, 7 * P,
                                      4 * P + off, 192, None, None, None, None, 0, None)
        assert refused(got, INV, "overlaps an input")
    for kw in (dict(lda=104, y=P + 126, ldy=104), dict(lda=104, y=P + 130, ldy=104), dict(lda=104, y=P + 128, ldy=105),
               dict(lda=152, y=P + 128, ldy=152, res=P + 206, ldr=152)):
        assert refused(linear(L, dummy, a=P, **kw), INV, "y overlaps")


# ------------------------------------------------------------------ binding

def zeros(*shape, dtype=torch.bfloat16, device="cpu"):
    return torch.zeros(*shape, dtype=dtype, device=device)


@pytest.mark.parametrize("w,bias,text", [
    (zeros(4, 8, dtype=torch.float16), None, "weight"), (zeros(4, 8, dtype=torch.float32), None, "weight"),
    (zeros(4), None, "weight"), (zeros(4, 8), zeros(3), "bias"), (zeros(4, 8), zeros(8), "bias"),
    (zeros(4, 8), zeros(4, dtype=torch.float32), "bias"), (zeros(4, 8), zeros(4, device="meta"), "bias"),
])
def test_linear_weights_are_checked(w, bias, text):
    """A weight that is not bf16, a bias that is not, or is shorter than the output."""
    with pytest.raises(ValueError, match=text):
        qi.bf16_struct(w, bias)


def test_linear_weights_that_are_right_get_past_the_checks():
    for w, bias in ((zeros(4, 8), None), (zeros(4, 8), zeros(4)), (zeros(4, 8, dtype=torch.int16), zeros(4))):
        with pytest.raises(ValueError, match="takes CUDA tensors"):   # (host tensors: refused behind them)
            qi.bf16_struct(w, bias)


def test_gated_ffn_weights_on_two_devices():
    with pytest.raises(ValueError, match="one device"):
        qi.gated_ffn_struct(zeros(16, 8), zeros(16, 8, device="meta"), zeros(8, 16))


def test_weights_on_another_device_than_the_context():
    """Activations are checked against the context's device; so are the weights."""
    class Ctx:
        device, handle = 0, None

    class Stream:
        cuda_stream = 0

    lin, ffn = qi.qi_linear_bf16(), qi.qi_gated_ffn()
    lin.n, lin.k, ffn.hidden, ffn.mlp = 4, 8, 8, 16
    lin._keep, ffn._keep = (zeros(4, 8), None), (zeros(16, 8), zeros(16, 8), zeros(8, 16))
    lin._device = ffn._device = -1        # (a host tensor's)
    x, gu = zeros(2, 8), zeros(2, 32, dtype=torch.float32)
    for call in (lambda: qi.qi_linear_act(Ctx, x, lin, stream=Stream),
                 lambda: qi.qi_gated_ffn_forward(Ctx, ffn, x, stream=Stream),
                 lambda: qi.qi_gated_ffn_backward(Ctx, ffn, x, x, gu, stream=Stream)):
        with pytest.raises(ValueError, match="weights"):
            call()
