"""Refusals of the prompt-encoder layer calls: every bad argument is answered
with its status on the host, before anything is launched.  Run without a GPU:
the calls get a zeroed stand-in for a context (of which a check reads the SM
count only) and pointers that nothing may follow."""
import ctypes as C

import numpy as np
import pytest

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


def attn(L, ctx, spans=((0, 4, 0, 4),), **kw):
    t = None if spans is None else np.asarray(spans, np.int32).reshape(-1, 4)
    a = dict(q=P, ldq=512, q_rows=16, k=2 * P, ldk=256, v=3 * P, ldv=256, k_rows=16, heads=4,
             kv_heads=2, head_dim=128, spans=None if t is None else t.ctypes.data,
             n=1 if t is None else len(t), scale=0.1, o=4 * P, ldo=512,
             ws=None, ws_bytes=0)
    a.update(kw)
    return L.qi_attn_causal_packed(C.addressof(ctx) if ctx is not None else None, a["q"], a["ldq"],
                                   a["q_rows"], a["k"], a["ldk"], a["v"], a["ldv"], a["k_rows"],
                                   a["heads"], a["kv_heads"], a["head_dim"], a["spans"], a["n"],
                                   a["scale"], a["o"], a["ldo"], a["ws"], a["ws_bytes"], None)


@pytest.mark.parametrize("kw,code", [
    (dict(q=None), INV), (dict(o=None), INV), (dict(k=None), INV), (dict(v=None), INV),
    (dict(q=P + 2), ALIGN), (dict(o=4 * P + 8), ALIGN), (dict(ldq=516), ALIGN), (dict(ldk=250), INV),
    (dict(ldo=504), INV), (dict(heads=3), INV), (dict(heads=0), INV), (dict(kv_heads=0), INV),
    (dict(heads=258, kv_heads=2, ldq=258 * 128, ldo=258 * 128), SHAPE), (dict(head_dim=64), SHAPE),
    (dict(q_rows=-1), INV), (dict(k_rows=-1), INV), (dict(n=-1), INV), (dict(n=257), INV),
    (dict(spans=None), INV), (dict(scale=0.0), INV), (dict(scale=float("nan")), INV),
    (dict(scale=float("inf")), INV), (dict(o=P), INV), (dict(o=2 * P), INV), (dict(o=3 * P + 512), INV),
    (dict(spans=((0, 17, 0, 4),)), INV), (dict(spans=((0, 4, 13, 4),)), INV),
    (dict(spans=((0, 4, 0, 4), (3, 2, 4, 2))), INV), (dict(spans=((0, -1, 0, 4),)), INV),
    (dict(spans=((0, 4, -1, 4),)), INV), (dict(spans=((2 ** 31 - 1, 2 ** 31 - 1, 0, 4),)), INV),
])
def test_attention_refusals(L, dummy, kw, code):
    assert attn(L, dummy, **kw) == code
    assert qi.last_error()


def test_attention_needs_the_workspace_it_asks_for(L, dummy):
    """One token against 8192 keys is split over its keys: no workspace, one byte
    less than asked for and a misaligned one are refused."""
    t = np.array([[0, 1, 0, 8192]], np.int32)
    n = C.c_size_t()
    assert L.qi_attn_causal_packed_workspace_bytes(C.addressof(dummy), t.ctypes.data, 1, 4, 2,
                                                   C.byref(n)) == qi.QI_OK
    assert n.value > 0
    kw = dict(spans=t, k_rows=8192, k=P, ldk=256, v=P + (8 << 20), q=P + (16 << 20), o=P + (17 << 20))
    assert attn(L, dummy, **kw) == WS
    assert attn(L, dummy, ws=P + (20 << 20), ws_bytes=n.value - 1, **kw) == WS
    assert attn(L, dummy, ws=P + (20 << 20) + 4, ws_bytes=n.value, **kw) == ALIGN
    assert attn(L, None, **kw) == INV
    assert L.qi_attn_causal_packed_workspace_bytes(None, t.ctypes.data, 1, 4, 2, C.byref(n)) == INV
    assert L.qi_attn_causal_packed_workspace_bytes(C.addressof(dummy), t.ctypes.data, 1, 4, 2, None) == INV


def test_attention_with_nothing_to_do_launches_nothing(L, dummy):
    """No sequence, or sequences without queries: accepted, and nothing is launched
    (a launch would fail here)."""
    assert attn(L, dummy, n=0) == qi.QI_OK
    assert attn(L, dummy, n=0, spans=None) == qi.QI_OK
    assert attn(L, dummy, spans=((0, 0, 0, 5), (3, 0, 0, 0))) == qi.QI_OK
    assert attn(L, dummy, n=0, q=None, o=None, k=None, v=None, q_rows=0, k_rows=0) == qi.QI_OK


def linear(L, ctx, **kw):
    a = dict(a=P, M=4, lda=64, w=2 * P, bias=None, n=40, k=64, act=0, res=None, ldr=0, y=3 * P, ldy=40)
    a.update(kw)
    w = qi.qi_linear_bf16()
    w.w, w.bias, w.n, w.k = a["w"], a["bias"], a["n"], a["k"]
    return L.qi_linear_act(C.addressof(ctx) if ctx is not None else None, a["a"], a["M"], a["lda"],
                           C.byref(w), a["act"], a["res"], a["ldr"], a["y"], a["ldy"], None)


@pytest.mark.parametrize("kw,code", [
    (dict(a=None), INV), (dict(y=None), INV), (dict(w=None), INV), (dict(M=-1), INV), (dict(n=0), INV),
    (dict(k=0), INV), (dict(k=60, lda=64), SHAPE), (dict(lda=56), INV), (dict(lda=68), ALIGN),
    (dict(a=P + 2), ALIGN), (dict(w=2 * P + 8), ALIGN), (dict(bias=P + 4), ALIGN), (dict(act=3), INV),
    (dict(act=-1), INV), (dict(ldy=39), INV), (dict(res=4 * P, ldr=39), INV), (dict(y=P), INV),
    (dict(y=2 * P), INV), (dict(res=3 * P, ldr=48), INV), (dict(res=3 * P + 80, ldr=40), INV),
])
def test_linear_refusals(L, dummy, kw, code):
    assert linear(L, dummy, **kw) == code
    assert linear(L, None) == INV
    assert linear(L, dummy, M=0, a=None, y=None) == qi.QI_OK


def gated(**kw):
    w = qi.qi_gated_ffn()
    a = dict(gate=P, up=2 * P, down=3 * P, hidden=64, mlp=128, act=qi.QI_ACT_SILU)
    a.update(kw)
    for name, v in a.items():
        setattr(w, name, v)
    return w


@pytest.mark.parametrize("kw,code", [
    (dict(gate=None), INV), (dict(up=None), INV), (dict(down=None), INV), (dict(hidden=60), SHAPE),
    (dict(mlp=0), SHAPE), (dict(mlp=130), SHAPE), (dict(act=qi.QI_ACT_NONE), INV), (dict(act=7), INV),
    (dict(down=3 * P + 2), ALIGN),
])
def test_gated_ffn_weight_refusals(L, dummy, kw, code):
    w, n = gated(**kw), C.c_size_t()
    c = C.addressof(dummy)
    assert L.qi_gated_ffn_workspace_bytes(C.byref(w), 4, 0, C.byref(n)) == code
    assert L.qi_gated_ffn_forward(c, C.byref(w), 4 * P, 4, 64, None, 0, 5 * P, 64, None, 6 * P, 1 << 20,
                                  None) == code
    assert L.qi_gated_ffn_backward(c, C.byref(w), 4 * P, 4, 64, 5 * P, 64, 7 * P, None, 0, None, None,
                                   None, 6 * P, 1 << 20, None) == code


def test_gated_ffn_row_refusals(L, dummy):
    w, c, n = gated(), C.addressof(dummy), C.c_size_t()

    def fwd(ctx=c, x=4 * P, M=4, ldx=64, res=None, ldr=0, y=5 * P, ldy=64, gu=None, ws=6 * P, wsb=1 << 20):
        return L.qi_gated_ffn_forward(ctx, C.byref(w), x, M, ldx, res, ldr, y, ldy, gu, ws, wsb, None)

    assert L.qi_gated_ffn_workspace_bytes(C.byref(w), 4, 0, C.byref(n)) == qi.QI_OK and n.value > 0
    assert fwd(ctx=None) == INV and fwd(x=None) == INV and fwd(y=None) == INV and fwd(M=-1) == INV
    assert fwd(ldx=56) == INV and fwd(ldx=68) == ALIGN and fwd(ldy=68) == ALIGN and fwd(x=4 * P + 2) == ALIGN
    assert fwd(res=7 * P, ldr=68) == ALIGN and fwd(gu=7 * P + 4) == ALIGN
    assert fwd(ws=None) == WS and fwd(wsb=n.value - 1) == WS
    assert fwd(y=6 * P) == INV and fwd(gu=6 * P) == INV and fwd(gu=5 * P) == INV and fwd(gu=4 * P) == INV
    assert fwd(y=P) == INV and fwd(y=3 * P) == INV and fwd(res=5 * P + 128, ldr=64) == INV
    assert fwd(x=6 * P) == INV and fwd(res=6 * P, ldr=64) == INV
    assert fwd(M=0, x=None, y=None, ws=None, wsb=0) == qi.QI_OK
    assert L.qi_gated_ffn_workspace_bytes(C.byref(w), 4, 1, C.byref(n)) == qi.QI_OK
    assert L.qi_gated_ffn_workspace_bytes(C.byref(w), -1, 1, C.byref(n)) == INV

    def bwd(ctx=c, x=4 * P, M=4, ldx=64, dy=5 * P, ldd=64, gu=7 * P, dx=8 * P, ldo=64, dg=9 * P,
            du=10 * P, dd=11 * P, ws=6 * P, wsb=1 << 20):
        return L.qi_gated_ffn_backward(ctx, C.byref(w), x, M, ldx, dy, ldd, gu, dx, ldo, dg, du, dd, ws,
                                       wsb, None)

    assert bwd(ctx=None) == INV and bwd(x=None) == INV and bwd(dy=None) == INV and bwd(gu=None) == INV
    assert bwd(M=-1) == INV and bwd(ldd=68) == ALIGN and bwd(dg=9 * P + 2) == ALIGN and bwd(ldo=60) == INV
    assert bwd(dx=5 * P) == INV and bwd(dx=7 * P) == INV and bwd(dg=P) == INV and bwd(du=9 * P) == INV
    assert bwd(dd=6 * P) == INV and bwd(dx=9 * P) == INV and bwd(gu=6 * P) == INV


def test_binding_checks_tensors():
    """The binding refuses tensors that are not what a call takes (no GPU needed:
    host tensors are refused too)."""
    import torch

    class Ctx:
        device, handle = 0, None

    with pytest.raises(ValueError):
        qi._rows(Ctx, torch.zeros(4, 8, dtype=torch.bfloat16), "x", 8)
    with pytest.raises(ValueError):
        qi._spans(torch.zeros(3, 4))
    with pytest.raises(ValueError):
        qi._spans(torch.zeros(3, 3, dtype=torch.int32))
    with pytest.raises(ValueError):
        qi._spans(torch.zeros(4, 8, dtype=torch.int32)[:, ::2])
