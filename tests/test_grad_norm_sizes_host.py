"""Tensor sizes that grad_norm_sq refuses are refused by its workspace size
too, before anything is added up: on the host."""

import ctypes

import pytest

from tests.test_abi_host import STATUS, lib  # noqa: F401  (the library fixture)


@pytest.mark.parametrize("sizes", [[(1 << 45) + 1], [1 << 62], [(1 << 63) - 1], [5, (1 << 63) - 1, (1 << 63) - 1],
                                   [0, (1 << 63) - 4096]])
def test_too_large_tensors(lib, sizes):  # noqa: F811
    n = ctypes.c_size_t(7)
    a = (ctypes.c_int64 * len(sizes))(*sizes)
    assert lib.grad_norm_sq_workspace_size(a, len(sizes), ctypes.byref(n)) == STATUS["UNSUPPORTED"] and n.value == 0


def test_the_largest_tensors(lib):  # noqa: F811
    n = ctypes.c_size_t(7)
    a = (ctypes.c_int64 * 3)(1 << 45, 1 << 45, 1)
    assert lib.grad_norm_sq_workspace_size(a, 3, ctypes.byref(n)) == 0 and 0 < n.value <= 3 * 2048 * 8
