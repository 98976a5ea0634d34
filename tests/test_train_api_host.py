"""Refusals of the training-step entry points, on the host: every call here
fails validation (or has nothing to do), so nothing reaches the device."""

import ctypes

import pytest

from moe_grouped_gemm_quantizer_amd import _lib
from tests.test_abi_host import STATUS, lib  # noqa: F401  (the library fixture)

P = 0x10000                                   # an aligned address that nothing uses


def _call(fn, base, **kw):
    assert set(kw) <= set(base), kw
    return fn(*{**base, **kw}.values())


def route_args(**kw):
    return dict(logits=P, type=0, T=256, E=8, ld=8, mask=None, k=2, renorm=0, coef=1.0, align=128, max_m=0,
                ids=P, weights=P, counts=P, routed=P, prob_sum=P, loss=P, offsets=P, slots=P, ws=P,
                ws_bytes=1 << 20, stream=None)


@pytest.mark.parametrize("kw,status", [
    (dict(T=-1), "SHAPE"), (dict(E=0), "SHAPE"), (dict(k=0), "SHAPE"), (dict(k=9), "SHAPE"),
    (dict(align=0), "SHAPE"), (dict(max_m=-1), "SHAPE"),
    (dict(type=3), "UNSUPPORTED"), (dict(type=-1), "UNSUPPORTED"), (dict(E=1025, ld=1025), "UNSUPPORTED"),
    (dict(E=32, ld=32, k=17), "UNSUPPORTED"), (dict(max_m=1 << 40), "UNSUPPORTED"),
    (dict(align=1 << 30), "UNSUPPORTED"), (dict(T=1 << 40), "UNSUPPORTED"),
    (dict(T=(1 << 30) - 1), "UNSUPPORTED"),
    (dict(ld=7), "STRIDE"),
    (dict(logits=None), "NULL"), (dict(ids=None), "NULL"), (dict(weights=None), "NULL"),
    (dict(counts=None), "NULL"), (dict(routed=None), "NULL"), (dict(prob_sum=None), "NULL"),
    (dict(loss=None), "NULL"), (dict(offsets=None), "NULL"), (dict(slots=None), "NULL"), (dict(ws=None), "NULL"),
    (dict(logits=P + 2), "ALIGN"), (dict(type=1, logits=P + 1), "ALIGN"), (dict(ids=P + 2), "ALIGN"),
    (dict(weights=P + 1), "ALIGN"), (dict(counts=P + 2), "ALIGN"), (dict(slots=P + 2), "ALIGN"),
    (dict(ws=P + 8), "ALIGN"),
    (dict(ws_bytes=16), "WORKSPACE"), (dict(ws=None, ws_bytes=0), "WORKSPACE"),
])
def test_moe_route(lib, kw, status):  # noqa: F811
    assert _call(lib.moe_route, route_args(), **kw) == STATUS[status]


def test_moe_route_workspace_size(lib):  # noqa: F811
    n = ctypes.c_size_t(7)
    assert lib.moe_route_workspace_size(64, 8, ctypes.byref(n)) == 0 and n.value == 0
    assert lib.moe_route_workspace_size(65, 8, ctypes.byref(n)) == 0 and n.value > 0
    small = n.value
    assert lib.moe_route_workspace_size(4096, 8, ctypes.byref(n)) == 0 and n.value > small
    assert lib.moe_route_workspace_size(-1, 8, ctypes.byref(n)) == STATUS["SHAPE"] and n.value == 0
    assert lib.moe_route_workspace_size(1, 0, ctypes.byref(n)) == STATUS["SHAPE"]
    assert lib.moe_route_workspace_size(1, 1025, ctypes.byref(n)) == STATUS["UNSUPPORTED"]
    assert lib.moe_route_workspace_size(1, 1, None) == STATUS["NULL"]


@pytest.mark.parametrize("kw,status", [
    (dict(T=-1), "SHAPE"), (dict(k=0), "SHAPE"), (dict(k=9), "SHAPE"), (dict(E=0), "SHAPE"),
    (dict(type=5), "UNSUPPORTED"), (dict(E=2000, ld=2000, ldd=2000), "UNSUPPORTED"),
    (dict(ld=7), "STRIDE"), (dict(ldd=7), "STRIDE"),
    (dict(logits=None), "NULL"), (dict(ids=None), "NULL"), (dict(counts=None), "NULL"),
    (dict(routed=None), "NULL"), (dict(d_logits=None), "NULL"),
    (dict(logits=P + 2), "ALIGN"), (dict(d_logits=P + 2), "ALIGN"), (dict(dw=P + 2), "ALIGN"),
    (dict(dloss=P + 1), "ALIGN"), (dict(ids=P + 1), "ALIGN"),
    (dict(T=0, logits=None, ids=None, d_logits=None), "OK"),
])
def test_moe_route_backward(lib, kw, status):  # noqa: F811
    base = dict(logits=P, type=0, T=256, E=8, ld=8, ids=P, k=2, renorm=0, coef=1.0, dw=P, dloss=P, counts=P,
                routed=P, d_logits=P, ldd=8, stream=None)
    assert _call(lib.moe_route_backward, base, **kw) == STATUS[status]


@pytest.mark.parametrize("kw,status", [
    (dict(rows=-1), "SHAPE"), (dict(cols=0), "SHAPE"), (dict(cols=24, ldx=24), "SHAPE"),
    (dict(type=3), "UNSUPPORTED"), (dict(fmt=2), "UNSUPPORTED"),
    (dict(rows=1 << 30, ldq=1 << 30), "UNSUPPORTED"),
    (dict(ldx=16), "STRIDE"), (dict(ldq=128), "STRIDE"),
    (dict(x=None), "NULL"), (dict(qt=None), "NULL"), (dict(st=None), "NULL"),
    (dict(x=P + 2), "ALIGN"), (dict(type=1, x=P + 1), "ALIGN"), (dict(qt=P + 8), "ALIGN"),
    (dict(ldq=260), "ALIGN"), (dict(st=P + 2), "ALIGN"),
    (dict(rows=0, x=None, qt=None, st=None), "OK"),
])
def test_fp8_quantize_transpose(lib, kw, status):  # noqa: F811
    base = dict(x=P, type=0, rows=200, cols=32, ldx=32, fmt=0, qt=P, ldq=256, st=P, stream=None)
    assert _call(lib.fp8_quantize_transpose, base, **kw) == STATUS[status]


@pytest.mark.parametrize("kw,status", [
    (dict(G=-1), "SHAPE"), (dict(T=-128), "SHAPE"), (dict(T=200), "SHAPE"), (dict(M=0), "SHAPE"),
    (dict(N=24), "SHAPE"), (dict(M=-16), "SHAPE"),
    (dict(fa=2), "UNSUPPORTED"), (dict(fb=-1), "UNSUPPORTED"), (dict(G=1025), "UNSUPPORTED"),
    (dict(lda=1 << 25), "UNSUPPORTED"), (dict(M=1 << 40, N=1 << 40), "UNSUPPORTED"),
    (dict(lda=128), "STRIDE"), (dict(ldb=240), "STRIDE"),
    (dict(a=None), "NULL"), (dict(sa=None), "NULL"), (dict(b=None), "NULL"), (dict(sb=None), "NULL"),
    (dict(d=None), "NULL"), (dict(group=None), "NULL"),
    (dict(a=P + 8), "ALIGN"), (dict(b=P + 4), "ALIGN"), (dict(d=P + 2), "ALIGN"), (dict(sa=P + 1), "ALIGN"),
    (dict(sb=P + 2), "ALIGN"), (dict(group=P + 2), "ALIGN"), (dict(lda=264), "ALIGN"), (dict(ldb=257), "ALIGN"),
    (dict(G=0, a=None, b=None, d=None), "OK"),
])
def test_grouped_gemm_fp8_wgrad(lib, kw, status):  # noqa: F811
    base = dict(a=P, fa=0, lda=256, sa=P, b=P, fb=0, ldb=256, sb=P, d=P, group=P, G=2, T=256, M=32, N=48,
                stream=None)
    assert _call(lib.grouped_gemm_fp8_wgrad, base, **kw) == STATUS[status]


def _list(ptrs, sizes, types):
    n = len(sizes)
    return (ctypes.c_void_p * n)(*ptrs), (ctypes.c_int64 * n)(*sizes), (ctypes.c_int * n)(*types)


@pytest.mark.parametrize("ptrs,sizes,types,kw,status", [
    ([P], [10], [0], dict(n=-1), "SHAPE"), ([P], [-1], [0], {}, "SHAPE"), ([P], [10], [3], {}, "UNSUPPORTED"),
    ([P], [1 << 50], [0], {}, "UNSUPPORTED"), ([None], [10], [0], {}, "NULL"), ([P + 2], [10], [0], {}, "ALIGN"),
    ([P, P + 1], [10, 10], [0, 1], {}, "ALIGN"), ([P], [10], [0], dict(sumsq=None), "NULL"),
    ([P], [10], [0], dict(sumsq=P + 4), "ALIGN"), ([P], [10], [0], dict(ws=P + 4), "ALIGN"),
    ([P], [10], [0], dict(ws_bytes=7), "WORKSPACE"), ([P], [10], [0], dict(ws=None, ws_bytes=0), "WORKSPACE"),
    ([P], [10], [0], dict(ws=None), "NULL"), ([P], [10], [0], dict(grads=None), "NULL"),
])
def test_grad_norm_sq(lib, ptrs, sizes, types, kw, status):  # noqa: F811
    g, s, t = _list(ptrs, sizes, types)
    base = dict(grads=g, numels=s, types=t, n=len(sizes), sumsq=P, ws=P, ws_bytes=1 << 20, stream=None)
    assert _call(lib.grad_norm_sq, base, **kw) == STATUS[status]


def test_grad_norm_sq_workspace_size(lib):  # noqa: F811
    n = ctypes.c_size_t(7)
    _, s, _ = _list([P] * 300, [5000] * 300, [0] * 300)
    assert lib.grad_norm_sq_workspace_size(s, 300, ctypes.byref(n)) == 0 and n.value == 300 * 8
    assert lib.grad_norm_sq_workspace_size(s, 0, ctypes.byref(n)) == 0 and n.value == 0
    assert lib.grad_norm_sq_workspace_size(s, -1, ctypes.byref(n)) == STATUS["SHAPE"]
    assert lib.grad_norm_sq_workspace_size(None, 1, ctypes.byref(n)) == STATUS["NULL"]
    assert lib.grad_norm_sq_workspace_size(s, 1, None) == STATUS["NULL"]


@pytest.mark.parametrize("outs,kw,status", [
    ([None], {}, "NULL"), ([P + 2], {}, "ALIGN"), ([P], dict(max_norm=0.0), "SHAPE"),
    ([P], dict(max_norm=-1.0), "SHAPE"), ([P], dict(max_norm=float("nan")), "SHAPE"),
    ([P], dict(sumsq=None), "NULL"), ([P], dict(norm=None), "NULL"), ([P], dict(norm=P + 2), "ALIGN"),
    ([P], dict(sumsq=P + 4), "ALIGN"), ([P], dict(outs=None), "NULL"), ([P], dict(n=-1), "SHAPE"),
])
def test_grad_clip(lib, outs, kw, status):  # noqa: F811
    g, s, t = _list([P], [10], [0])
    o, _, _ = _list(outs, [10], [0])
    base = dict(grads=g, outs=o, numels=s, types=t, n=1, sumsq=P, max_norm=1.0, norm=P, stream=None)
    assert _call(lib.grad_clip, base, **kw) == STATUS[status]


def test_binding_refuses_what_would_be_misread():
    import torch
    import moe_grouped_gemm_quantizer_amd as fp8g
    x = torch.zeros(4, 16)                                # not on the GPU
    u8 = torch.zeros(16, 128, dtype=torch.uint8)
    with pytest.raises(ValueError):
        fp8g.fp8_quantize_transpose(x, "e4m3", u8, torch.zeros(1, 16, dtype=torch.uint8))
    with pytest.raises(ValueError):
        fp8g.grad_norm_sq([x], torch.zeros(1, dtype=torch.float64), None)
    with pytest.raises(ValueError):
        fp8g.grad_norm_sq([x.double()], torch.zeros(1, dtype=torch.float64), None)
    with pytest.raises(ValueError):
        fp8g.moe_route_backward(x, torch.zeros(4, 2, dtype=torch.int32), None, None,
                                torch.zeros(16, dtype=torch.int32), torch.zeros(1, dtype=torch.int32), x)
    with pytest.raises(ValueError):
        fp8g.grouped_gemm_fp8_wgrad(u8, "e4m3", u8, u8, "e4m3", u8, u8)
    assert _lib.moe_route_workspace_size(1, 8) == 0
