"""Argument checks of the optimizer and 4-bit calls (CPU only: every call fails
validation or is a no-op, so nothing is launched and no address is read)."""
import ctypes

import pytest
import torch

import gradient_sync_amd as dps
from gradient_sync_amd import training as T

OK, INVALID, UNSUPPORTED, ALIAS = 0, 1, 2, 3
F32, BF16, I32 = 0, 1, 2
P = lambda ptrs: dps.ptr_array([p or 0 for p in ptrs])
B = [1 << s for s in range(40, 47)]
NAN, INF = float("nan"), float("inf")


def counts(*n):
    return (ctypes.c_int64 * max(1, len(n)))(*n)


def opts(lr=1e-3, b1=0.9, b2=0.99, eps=1e-8, wd=0.1, step=1, seed=0, flags=0, reserved=0):
    return dps.AdamWOpts(lr, b1, b2, eps, wd, step, seed, flags, reserved)


def adamw(n=100, p=B[0], pdt=F32, g=B[1], gdt=F32, m=B[2], v=B[3], copy=None, o=None, ctrl=None, nt=1):
    o = opts() if o is None else o
    return dps.lib().dp_adamw(nt, counts(n), P([p]), pdt, P([g]), gdt, P([m]), P([v]),
                              None if copy is None else P([copy]), ctypes.byref(o), ctrl, None)


def adamw8(n=100, p=B[0], g=B[1], m=B[2], v=B[3], s=B[4], o=None, copy=None, pdt=F32):
    o = opts() if o is None else o
    return dps.lib().dp_adamw8(1, counts(n), P([p]), pdt, P([g]), BF16, P([m]), P([v]), P([s]),
                               None if copy is None else P([copy]), ctypes.byref(o), None, None)


def norm(n=100, g=B[0], dt=F32, most=1.0, ctrl=B[1], ws=B[2], nt=1):
    return dps.lib().dp_grad_norm(nt, counts(n), P([g]), dt, most, ctrl, ws, None)


def test_constants_match_the_header():
    text = open(dps.LIB_PATH.rsplit("/", 2)[0] + "/include/dpsync.h").read()
    assert f"#define DP_STATE_BLOCK {T.STATE_BLOCK} " in text
    assert f"#define DP_GRAD_NORM_WS_BYTES {T.GRAD_NORM_WS_BYTES}\n" in text


def test_grad_norm_refusals():
    assert norm(nt=-1) == INVALID
    assert norm(nt=65537) == INVALID
    assert norm(n=-1) == INVALID
    assert norm(n=1 << 41) == INVALID
    assert norm(dt=I32) == UNSUPPORTED
    assert norm(g=None) == INVALID
    assert norm(g=B[0] + 2) == INVALID and norm(g=B[0] + 1, dt=BF16) == INVALID
    assert norm(ctrl=None) == INVALID and norm(ctrl=B[1] + 2) == INVALID
    assert norm(ws=None) == INVALID and norm(ws=B[2] + 4) == INVALID
    assert norm(most=-1.0) == INVALID and norm(most=NAN) == INVALID and norm(most=INF) == INVALID
    assert norm(ctrl=B[2] + 16) == ALIAS
    assert norm(g=B[1] - 396) == ALIAS and norm(g=B[2] + T.GRAD_NORM_WS_BYTES - 4) == ALIAS
    assert dps.lib().dp_grad_norm(1, None, P([B[0]]), F32, 1.0, B[1], B[2], None) == INVALID
    assert dps.lib().dp_grad_norm(1, counts(1), None, F32, 1.0, B[1], B[2], None) == INVALID


def test_adamw_refusals():
    assert adamw(pdt=I32) == UNSUPPORTED and adamw(gdt=5) == UNSUPPORTED
    assert adamw(pdt=BF16, copy=B[5]) == UNSUPPORTED
    assert adamw(o=opts(flags=1)) == UNSUPPORTED                  # nothing to round in fp32 states
    assert adamw(o=opts(flags=2)) == INVALID and adamw(o=opts(reserved=1)) == INVALID
    for bad in (dict(lr=-1), dict(lr=NAN), dict(lr=INF), dict(b1=1.0), dict(b1=-0.1), dict(b2=1.0),
                dict(b2=NAN), dict(eps=-1e-8), dict(eps=INF), dict(wd=-1), dict(wd=NAN),
                dict(step=-1), dict(step=0)):
        assert adamw(o=opts(**bad)) == INVALID, bad
        assert adamw8(o=opts(**bad)) == INVALID, bad
    for bad in (dict(p=None), dict(g=None), dict(m=None), dict(v=None), dict(p=B[0] + 2),
                dict(m=B[2] + 2), dict(copy=B[5] + 1), dict(n=-1), dict(nt=-1), dict(nt=1 << 20),
                dict(ctrl=B[6] + 2)):
        assert adamw(**bad) == INVALID, bad
    assert adamw8(s=B[4] + 4) == INVALID and adamw8(s=None) == INVALID
    for bad in (dict(g=B[0] + 396), dict(m=B[1] - 4), dict(v=B[2] + 4), dict(copy=B[3]), dict(p=B[3]),
                dict(ctrl=B[0] + 8)):
        assert adamw(**bad) == ALIAS, bad
    assert adamw8(s=B[2]) == ALIAS and adamw8(m=B[3] + 99) == ALIAS
    L = dps.lib()
    assert L.dp_adamw(1, counts(1), P([B[0]]), F32, P([B[1]]), F32, P([B[2]]), P([B[3]]), None, None,
                      None, None) == INVALID


def test_adamw_alias_among_many_tensors():
    k = 200
    base = lambda i: [B[i] + 4096 * j for j in range(k)]
    p, g, m, v = base(0), base(1), base(2), base(3)
    v[150] = m[7] + 8
    o = opts()
    assert dps.lib().dp_adamw(k, counts(*[5] * k), P(p), F32, P(g), F32, P(m), P(v), None,
                              ctypes.byref(o), None, None) == ALIAS


def test_empty_updates_are_no_ops():
    assert adamw(n=0) == OK and adamw8(n=0) == OK
    assert adamw(n=0, p=None, g=None, m=None, v=None) == OK
    assert adamw(nt=0) == OK


def quant(rows=64, cols=96, ld=96, dt=F32, src=B[0], q=B[1], s=B[2], qt=B[3], st=B[4]):
    return dps.lib().dp_mxfp4_quantize(src, rows, cols, ld, dt, q, s, qt, st, None)


def test_sizes():
    L = dps.lib()
    assert L.dp_mxfp4_code_bytes(3, 129) == 3 * 128 and L.dp_mxfp4_code_bytes(0, 5) == 0
    assert L.dp_mxfp4_scale_bytes(17, 513) == 2 * 2 * 256
    assert L.dp_mxfp4_code_bytes(-1, 5) == 0 and L.dp_mxfp4_scale_bytes(1, 1 << 25) == 0
    assert L.dp_mxfp4_linear_ws_bytes(16, 1000, 4096) == 0
    assert L.dp_mxfp4_linear_ws_bytes(1, 1 << 14, 14336) == 0
    assert L.dp_mxfp4_linear_ws_bytes(16, 1 << 15, 14336) == 16 * 7168 + 28 * 256
    assert L.dp_mxfp4_linear_ws_bytes(17, 1000, 100) == 17 * 64 + 192 + 512
    assert L.dp_mxfp4_linear_ws_bytes(-1, 10, 100) == 0


def test_quantize_refusals():
    assert quant(rows=-1) == INVALID and quant(cols=1 << 25, ld=1 << 25) == INVALID
    assert quant(ld=95) == INVALID and quant(ld=1 << 41) == INVALID
    assert quant(dt=I32) == UNSUPPORTED
    assert quant(q=None) == INVALID and quant(s=None) == INVALID          # half a pair
    assert quant(qt=None) == INVALID and quant(st=None) == INVALID
    assert quant(q=None, s=None, qt=None, st=None) == INVALID
    assert quant(src=None) == INVALID and quant(src=B[0] + 2) == INVALID
    assert quant(q=B[1] + 8) == INVALID and quant(s=B[2] + 2) == INVALID
    assert quant(q=B[0] + 64 * 96 * 4 - 16) == ALIAS and quant(st=B[1]) == ALIAS and quant(qt=B[1] + 16) == ALIAS
    assert quant(rows=0) == OK and quant(cols=0, ld=0) == OK


def test_dequantize_refusals():
    f = lambda q=B[0], s=B[1], r=64, c=96, d=B[2], ld=96, dt=F32: dps.lib().dp_mxfp4_dequantize(
        q, s, r, c, d, ld, dt, None)
    assert f(dt=I32) == UNSUPPORTED
    assert f(r=-1) == INVALID and f(ld=95) == INVALID and f(q=None) == INVALID and f(s=B[1] + 1) == INVALID
    assert f(d=B[2] + 1) == INVALID and f(d=None) == INVALID
    assert f(d=B[0]) == ALIAS and f(d=B[1] - 4) == ALIAS
    assert f(r=0) == OK and f(c=0, ld=0) == OK


def test_gemm_refusals():
    f = lambda a=B[0], sa=B[1], b=B[2], sb=B[3], c=B[4], m=64, n=32, k=96, dt=F32, acc=0: \
        dps.lib().dp_gemm_mxfp4(a, sa, b, sb, c, m, n, k, dt, acc, None)
    assert f(dt=I32) == UNSUPPORTED and f(dt=BF16, acc=1) == UNSUPPORTED
    assert f(m=-1) == INVALID and f(k=0) == INVALID and f(n=1 << 25) == INVALID
    assert f(m=1 << 24, n=1 << 24) == INVALID
    for bad in (dict(a=None), dict(sa=None), dict(b=B[2] + 4), dict(sb=B[3] + 1), dict(c=B[4] + 2)):
        assert f(**bad) == INVALID, bad
    for bad in (dict(c=B[0]), dict(c=B[1] + 4), dict(c=B[2] - 4), dict(c=B[3])):
        assert f(**bad) == ALIAS, bad
    assert f(m=0) == OK and f(n=0) == OK


def test_linear_refusals():
    f = lambda x=B[0], ldx=96, xdt=BF16, w=B[1], s=B[2], y=B[3], m=64, n=32, k=96, ydt=BF16, ws=B[4]: \
        dps.lib().dp_mxfp4_linear(x, ldx, xdt, w, s, y, m, n, k, ydt, ws, None)
    assert f(xdt=I32) == UNSUPPORTED and f(ydt=I32) == UNSUPPORTED
    assert f(ldx=95) == INVALID and f(k=0, ldx=0) == INVALID and f(m=-1) == INVALID
    for bad in (dict(x=B[0] + 1), dict(w=B[1] + 8), dict(s=None), dict(y=None), dict(ws=None), dict(ws=B[4] + 8)):
        assert f(**bad) == INVALID, bad
    for bad in (dict(y=B[0]), dict(y=B[1]), dict(ws=B[0]), dict(ws=B[3] - 16), dict(y=B[2])):
        assert f(**bad) == ALIAS, bad
    assert f(m=0) == OK and f(n=0) == OK


def test_binding_refusals():
    x = torch.zeros(4, 4)
    with pytest.raises(ValueError, match="GPU"):
        dps.GradNorm([x])
    with pytest.raises(TypeError):
        dps.GradNorm([x.double()])
    with pytest.raises(TypeError):
        dps.GradNorm([1.0])
    with pytest.raises(ValueError, match="GPU"):
        dps.AdamW([x], [x], [x], [x])
    with pytest.raises(ValueError):
        dps.AdamW.new_state([x], bits=4)
    with pytest.raises(ValueError, match="GPU"):
        dps.dp_mxfp4_quantize(x)
    with pytest.raises(ValueError):
        dps.dp_mxfp4_quantize(x, transposed="yes")
    with pytest.raises(TypeError):
        dps.dp_mxfp4_quantize(x.double())
    with pytest.raises(ValueError, match="GPU"):
        dps.Mxfp4(4, 4, device="cpu")
