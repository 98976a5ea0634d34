"""Refusals of the AdamW step on the host (nothing reaches the device), and its plain forms."""

import ctypes

import numpy as np
import pytest

from moe_grouped_gemm_quantizer_amd._lib import load
from oracle.formats import e4m3_decode_table
from tests import adamw_ref as ref
from tests.test_abi_host import STATUS, lib  # noqa: F401  (the library fixture)
from tests.test_train_api_host import P


def call(lib, n=2, sizes=(5, 300), eight=False, **kw):  # noqa: F811
    held = []

    def ptrs(v=P):
        a = (ctypes.c_uint64 * n)(*([v] * n))
        held.append(a)
        return ctypes.addressof(a)

    def ints(v, kind=ctypes.c_int):
        a = (kind * n)(*(v if isinstance(v, (tuple, list)) else [v] * n))
        held.append(a)
        return ctypes.addressof(a)
    base = dict(p=ptrs(), pt=ints(0), g=ptrs(), gt=ints(1), m=ptrs(), v=ptrs(), ms=ptrs() if eight else None,
                vs=ptrs() if eight else None, c=None, ct=None, numels=ints(list(sizes), ctypes.c_int64), n=n, step=None,
                step_value=1, lr=None, lr_value=0.1, b1=0.9, b2=0.99, eps=1e-8, wd=0.0, sumsq=None, max_norm=0.0,
                norm=None, seed=0, table=None, stream=None)
    for k, v in kw.items():
        if isinstance(v, tuple):
            v = ptrs(v[1]) if v[0] == "ptr" else ints(v[1], ctypes.c_int64 if k == "numels" else ctypes.c_int)
        base[k] = v
    return lib.adamw_step(*base.values())


NAN, INF = float("nan"), float("inf")


@pytest.mark.parametrize("kw,status", [
    (dict(numels=("int", [5, -1])), "SHAPE"), (dict(step_value=0), "SHAPE"), (dict(b1=1.0), "SHAPE"),
    (dict(b1=-0.1), "SHAPE"), (dict(b2=NAN), "SHAPE"), (dict(b2=1.5), "SHAPE"), (dict(eps=-1e-9), "SHAPE"),
    (dict(eps=INF), "SHAPE"), (dict(wd=NAN), "SHAPE"), (dict(lr_value=INF), "SHAPE"),
    (dict(sumsq=P, max_norm=0.0), "SHAPE"), (dict(sumsq=P, max_norm=NAN), "SHAPE"),
    (dict(pt=("int", 3)), "UNSUPPORTED"), (dict(gt=("int", -1)), "UNSUPPORTED"),
    (dict(c=("ptr", P), ct=("int", 0)), "UNSUPPORTED"), (dict(numels=("int", [5, (1 << 43) + 1])), "UNSUPPORTED"),
    (dict(eight=True, numels=("int", [5, (1 << 38) + 1])), "UNSUPPORTED"),
    (dict(p=None), "NULL"), (dict(pt=None), "NULL"), (dict(g=None), "NULL"), (dict(gt=None), "NULL"),
    (dict(m=None), "NULL"), (dict(v=None), "NULL"), (dict(numels=None), "NULL"), (dict(p=("ptr", 0)), "NULL"),
    (dict(g=("ptr", 0)), "NULL"), (dict(m=("ptr", 0)), "NULL"), (dict(v=("ptr", 0)), "NULL"),
    (dict(eight=True, ms=None), "NULL"), (dict(eight=True, vs=None), "NULL"), (dict(eight=True, vs=("ptr", 0)), "NULL"),
    (dict(c=("ptr", P)), "NULL"), (dict(norm=P), "NULL"),
    (dict(p=("ptr", P + 2)), "ALIGN"), (dict(g=("ptr", P + 1)), "ALIGN"), (dict(m=("ptr", P + 2)), "ALIGN"),
    (dict(v=("ptr", P + 1)), "ALIGN"), (dict(c=("ptr", P + 1), ct=("int", 1)), "ALIGN"), (dict(step=P + 4), "ALIGN"),
    (dict(lr=P + 2), "ALIGN"), (dict(sumsq=P + 4, max_norm=1.0), "ALIGN"), (dict(sumsq=P, max_norm=1.0, norm=P + 1), "ALIGN"),
    (dict(table=P + 4), "ALIGN"),
])
def test_refusals(lib, kw, status):  # noqa: F811
    assert call(lib, **kw) == STATUS[status]


def test_table():
    """Ends and entries of a list with an empty tensor, as the header's sizes say; refusals."""
    lib = load()
    size = ctypes.c_size_t(7)
    assert lib.adamw_table_size(-1, ctypes.byref(size)) == STATUS["SHAPE"] and size.value == 0
    assert lib.adamw_table_size(3, None) == STATUS["NULL"]
    assert lib.adamw_table_size(0, ctypes.byref(size)) == 0 and size.value == 0
    assert lib.adamw_table_size(3, ctypes.byref(size)) == 0 and size.value == 16 + 3 * 72
    numels = [5000, 0, 2048]
    ptr = [(ctypes.c_uint64 * 3)(*[P + 4096 * (3 * j + i) for i in range(3)]) for j in range(4)]
    typ = (ctypes.c_int * 3)(0, 1, 2)
    sizes = (ctypes.c_int64 * 3)(*numels)
    lists = [ptr[0], typ, ptr[1], typ, ptr[2], ptr[3], None, None, None, None, sizes]
    at = lambda t: None if t is None else ctypes.addressof(t)  # noqa: E731
    out = np.full(size.value + 8, 0xAB, np.uint8)
    call = lambda ls, table=None: lib.adamw_table(*map(at, ls), 3, out.ctypes.data if table is None else table)  # noqa: E731
    assert out.ctypes.data % 8 == 0 and call(lists) == 0
    assert (out[-8:] == 0xAB).all()
    assert list(out[:16].view(np.int32)[:3]) == [3, 3, 4]
    for i, n in enumerate(numels):
        e = out[16 + 72 * i:16 + 72 * (i + 1)]
        assert list(e[:64].view(np.uint64)) == [ptr[j][i] for j in range(4)] + [0, 0, 0, n]
        assert e[64:68].view(np.int32)[0] == [0, 3, 3][i] and e[68] == 4 * i and e[69] == 0
    assert call(lists, 0) == STATUS["NULL"] and call(lists, out.ctypes.data + 4) == STATUS["ALIGN"]
    assert call([None] + lists[1:]) == STATUS["NULL"]
    assert call(lists[:10] + [(ctypes.c_int64 * 3)(5, -1, 3)]) == STATUS["SHAPE"]
    lists[10] = (ctypes.c_int64 * 3)(*[(1 << 35) - 2048] * 3)
    assert call(lists) == 0


def test_plain_codes():
    """The plain encoder against the format's own table: without random bits the value below,
    with the largest ones the value above unless it is exact; blocks' scales."""
    table = e4m3_decode_table()
    rng = np.random.default_rng(0)
    x = np.concatenate([np.exp(rng.uniform(-25, 6, 500)) * rng.choice([-1, 1], 500), [448.0, -448.0, 0.0, -0.0],
                        table[:127], -table[:127]]).astype(np.float32)
    x = np.concatenate([x, np.zeros(-len(x) % 128, np.float32)])
    down, s = ref.encode(x, np.zeros(len(x)), False)
    up, _ = ref.encode(x, np.full(len(x), 65535.0), False)
    a, b = np.abs(ref.decode(down, s)), np.abs(ref.decode(up, s))
    assert (np.sign(ref.decode(up, s)) * np.sign(x) >= 0).all()
    y = np.abs(x.astype(np.float64))
    unit = np.where(y > 0, np.maximum(2.0 ** (np.frexp(y)[1] - 4.0), np.repeat(2.0 ** (s - 136.0), 128)), 0.0)
    assert (a <= y * (1 + 2.0 ** -20) + unit * 2.0 ** -19).all() and (b >= y * (1 - 2.0 ** -15) - unit * 2.0 ** -15).all()
    assert (b - a <= unit * 2).all()
    tops = np.abs(x).reshape(-1, 128).max(1)
    assert all(t <= 448.0 * 2.0 ** (k - 127) and (t > 224.0 * 2.0 ** (k - 127) or t == 0) for t, k in
               zip(tops, s.astype(float)))
    assert np.array_equal(ref.decode(np.arange(127, dtype=np.uint8), np.array([127], np.uint8)), table[:127])


def test_plain_root_is_never_zero():
    x = np.float32([1e-30, 0.0, 1.0] + [0] * 125)
    c, s = ref.encode(x, np.zeros(128), True)
    assert c[0] == 1 and c[1] == 0 and s[0] == 127 - 8
