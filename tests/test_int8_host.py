"""Refusals of the 8-bit integer entry points, on the host: every call here fails
validation (or has nothing to do), so nothing reaches the device."""

import numpy as np
import pytest

from tests import int8_ref as ref
from tests.test_abi_host import STATUS, lib  # noqa: F401  (the library fixture)
from tests.test_train_api_host import P, _call


def quant_args(**kw):
    return dict(x=P, type=1, rows=4, cols=64, ldx=64, q=P, ldq=64, scales=P, stream=None)


@pytest.mark.parametrize("kw,status", [
    (dict(rows=-1), "SHAPE"), (dict(cols=0), "SHAPE"), (dict(cols=24), "SHAPE"), (dict(type=3), "UNSUPPORTED"),
    (dict(type=-1), "UNSUPPORTED"), (dict(x=None), "NULL"), (dict(q=None), "NULL"), (dict(scales=None), "NULL"),
    (dict(ldx=63), "STRIDE"), (dict(ldq=48), "STRIDE"), (dict(x=P + 1), "ALIGN"), (dict(type=0, x=P + 2), "ALIGN"),
    (dict(q=P + 8), "ALIGN"), (dict(ldq=72), "ALIGN"), (dict(scales=P + 2), "ALIGN"), (dict(rows=0, x=None), "OK")])
def test_quantize(lib, kw, status):  # noqa: F811
    assert _call(lib.int8_quantize, quant_args(), **kw) == STATUS[status]


def dense_args(**kw):
    return dict(a=P, sa=P, b=P, sb=P, d=P, M=64, N=64, K=64, stream=None)


SHARED = [(dict(N=0), "SHAPE"), (dict(N=24), "SHAPE"), (dict(K=0), "SHAPE"), (dict(K=8), "SHAPE"),
          (dict(K=131072), "UNSUPPORTED"), (dict(N=(1 << 27) + 16), "UNSUPPORTED"),
          (dict(a=None), "NULL"), (dict(sa=None), "NULL"), (dict(b=None), "NULL"), (dict(sb=None), "NULL"),
          (dict(d=None), "NULL"), (dict(a=P + 8), "ALIGN"), (dict(b=P + 4), "ALIGN"), (dict(d=P + 2), "ALIGN"),
          (dict(sa=P + 2), "ALIGN"), (dict(sb=P + 1), "ALIGN")]


@pytest.mark.parametrize("kw,status", SHARED + [
    (dict(M=-1), "SHAPE"), (dict(M=(1 << 30) + 1), "UNSUPPORTED"), (dict(M=1 << 30, N=1 << 20), "UNSUPPORTED"),
    (dict(M=0, a=None), "OK")])
def test_dense(lib, kw, status):  # noqa: F811
    assert _call(lib.gemm_int8, dense_args(), **kw) == STATUS[status]


@pytest.mark.parametrize("kw,status", SHARED + [
    (dict(G=-1), "SHAPE"), (dict(M=-1), "SHAPE"), (dict(G=1025), "UNSUPPORTED"), (dict(off=None), "NULL"),
    (dict(off=P + 2), "ALIGN"), (dict(M=1 << 30, N=1 << 20), "UNSUPPORTED"), (dict(G=0, a=None), "OK"),
    (dict(M=0, a=None), "OK")])
def test_contiguous(lib, kw, status):  # noqa: F811
    base = dict(a=P, sa=P, b=P, sb=P, d=P, off=P, G=4, M=64, N=64, K=64, stream=None)
    assert _call(lib.grouped_gemm_int8_contiguous, base, **kw) == STATUS[status]


@pytest.mark.parametrize("kw,status", SHARED + [
    (dict(G=-1), "SHAPE"), (dict(max_m=-1), "SHAPE"), (dict(G=1025), "UNSUPPORTED"), (dict(m=None), "NULL"),
    (dict(m=P + 1), "ALIGN"), (dict(max_m=1 << 30, N=1 << 16, G=64), "UNSUPPORTED"), (dict(G=0, a=None), "OK"),
    (dict(max_m=0, a=None), "OK")])
def test_masked(lib, kw, status):  # noqa: F811
    base = dict(a=P, sa=P, b=P, sb=P, d=P, m=P, G=4, max_m=64, N=64, K=64, hint=0, stream=None)
    assert _call(lib.grouped_gemm_int8_masked, base, **kw) == STATUS[status]


def test_plain_quantiser_by_hand():
    q, s = ref.quantise(np.float32([[1, -2, 127, 0.5], [0, 0, 0, 0], [1, np.nan, 2, 3], [-254, 127, 3, 1]]))
    assert q.tolist() == [[1, -2, 127, 0], [0] * 4, [0] * 4, [-127, 64, 2, 0]]
    assert s[0] == 1 and s[1] == 0 and np.isnan(s[2]) and s[3] == 2


def test_plain_product_by_hand():
    d = ref.product(np.int8([[1, 2], [-3, 4]]), [2, 1], np.int8([[5, 6], [0, -128]]), [1, 0.5])
    want = np.float32([[34, -256], [9, -256]])
    assert np.array_equal(d, (want.view(np.uint32) >> 16).astype(np.uint16))
