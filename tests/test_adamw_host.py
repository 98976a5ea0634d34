"""Refusals of the AdamW step on the host (nothing reaches the device), and its plain forms."""

import ctypes

import numpy as np
import pytest

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
                norm=None, seed=0, stream=None)
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
])
def test_refusals(lib, kw, status):  # noqa: F811
    assert call(lib, **kw) == STATUS[status]


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
