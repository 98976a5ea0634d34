"""Sizes that no launch can hold are refused before one is tried: on the host,
nothing reaches the device."""

import pytest

from tests.test_abi_host import STATUS, lib  # noqa: F401  (the library fixture)
from tests.test_train_api_host import P

LAST = ((1 << 24) - 1) * 128                  # 2^24 - 1 workgroups of 256 threads


@pytest.mark.parametrize("cols", [LAST + 16, 1 << 31, (1 << 31) + 128, 1 << 40])
def test_columns_of_the_transposing_quantiser(lib, cols):  # noqa: F811
    args = (P, 1, 1, cols, cols, 0, P, 128, P, None)
    assert lib.fp8_quantize_transpose(*args) == STATUS["UNSUPPORTED"]


def test_columns_up_to_the_bound_pass_it(lib):  # noqa: F811
    # (refused for the next reason in line: the row stride)
    assert lib.fp8_quantize_transpose(P, 1, 1, LAST, LAST - 1, 0, P, 128, P, None) == STATUS["STRIDE"]
