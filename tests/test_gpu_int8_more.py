"""Integer products on the GPU at sizes that the other tests leave out."""

import pytest
import torch

import moe_grouped_gemm_quantizer_amd as fp8g
from tests.gpu_util import dev

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("M", [1 << 30, (1 << 30) - 70])
def test_more_rows_than_a_launch_of_small_tiles_holds(M):
    """2^30 rows of 16: a workgroup for each 64 of them would be 2^32 threads."""
    N = K = 16
    gen = torch.Generator(dev()).manual_seed(5)
    step = 1 << 22
    base = torch.randint(-128, 128, (step, K), dtype=torch.int8, device=dev(), generator=gen)
    b = torch.randint(-128, 128, (N, K), dtype=torch.int8, device=dev(), generator=gen)
    sb = torch.rand(N, device=dev(), generator=gen)
    a = torch.empty(M, K, dtype=torch.int8, device=dev())
    sa = torch.empty(M, device=dev())
    for i, at in enumerate(range(0, M, step)):
        n = min(step, M - at)
        a[at:at + n] = base.roll(i * 1001, 0)[:n]
        sa[at:at + n] = (i + 1) * 1e-3
    d = torch.full((M, N), -1, dtype=torch.int16, device=dev())
    fp8g.gemm_int8(a, sa, b, sb, d)
    for at in range(0, M, step):
        n = min(step, M - at)
        want = (a[at:at + n].float() @ b.float().t() * sa[at:at + n, None] * sb).to(torch.bfloat16)   # (sums below 2^24)
        assert torch.equal(d[at:at + n], want.view(torch.int16)), at
