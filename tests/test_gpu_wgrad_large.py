"""The weight gradient where 256x256 tiles serve it: chains of tiles in one
workgroup, every pair of formats, strides, offsets outside their contract, NaN."""

import pytest
import torch

import moe_grouped_gemm_quantizer_amd as fp8g
from tests.gpu_util import dev, banner

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("G,M,N", [(200, 16, 32), (3, 2064, 1552)])
def test_no_tokens_and_many_tiles(G, M, N):
    banner(f"wgrad T=0 G={G} M={M} N={N}")
    e = torch.empty(0, dtype=torch.uint8, device=dev())
    off = torch.zeros(G + 1, dtype=torch.int32, device=dev())
    d = torch.full((G, M, N), float("nan"), dtype=torch.bfloat16, device=dev())
    fp8g.grouped_gemm_fp8_wgrad(e.view(M, 0), "e4m3", e.view(0, M), e.view(N, 0), "e4m3", e.view(0, N), d,
                                group_offsets=off)
    assert (d.view(torch.int16) == 0).all()
