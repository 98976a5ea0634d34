"""Integer products that no launch holds, refused on the host."""

import pytest

from tests.test_abi_host import STATUS, lib  # noqa: F401  (the library fixture)
from tests.test_int8_host import dense_args
from tests.test_train_api_host import P, _call


@pytest.mark.parametrize("M,N", [(1 << 30, 144), ((1 << 30) - 127, 256), (1 << 17, 1 << 21), ((1 << 17) - 127, 1 << 21),
                                 (1 << 21, (1 << 17) - 112), (129 << 4, 1 << 27)])
def test_dense_of_too_many_tiles(lib, M, N):  # noqa: F811
    assert -(-M // 128) * -(-N // 128) >= 1 << 24
    assert _call(lib.gemm_int8, dense_args(), M=M, N=N, K=16) == STATUS["UNSUPPORTED"]


@pytest.mark.parametrize("M,N,G", [(1 << 30, 128 * 2, 1), ((1 << 30) - 128, 256, 1), (1, 1 << 27, 15), (1 << 20, 1 << 18, 1)])
def test_contiguous_of_too_many_tiles(lib, M, N, G):  # noqa: F811
    assert (-(-M // 128) + G) * -(-N // 128) >= 1 << 24
    base = dict(a=P, sa=P, b=P, sb=P, d=P, off=P, G=G, M=M, N=N, K=16, stream=None)
    assert _call(lib.grouped_gemm_int8_contiguous, base) == STATUS["UNSUPPORTED"]


@pytest.mark.parametrize("max_m,N,G", [(1, 1 << 21, 1024), (129, 1 << 20, 1024), (1 << 30, 16, 2), (1 << 27, 256, 8)])
def test_masked_of_too_many_tiles(lib, max_m, N, G):  # noqa: F811
    assert -(-max_m // 128) * -(-N // 128) * G >= 1 << 24
    base = dict(a=P, sa=P, b=P, sb=P, d=P, m=P, G=G, max_m=max_m, N=N, K=16, hint=0, stream=None)
    assert _call(lib.grouped_gemm_int8_masked, base) == STATUS["UNSUPPORTED"]
