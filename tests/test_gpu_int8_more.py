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


@pytest.mark.parametrize("kind", [torch.float32, torch.bfloat16, torch.float16])
def test_codes_are_the_nearest_whole_numbers(kind):
    """Of x 127 / amax in 64 bits. Its fp32 form is off by half a step of the quotient and half a one of the
    product, 127 2^-23 in all: by that much a code may be on the other side of a half."""
    gen = torch.Generator(dev()).manual_seed(6)
    x = (torch.randn(2000, 4096, device=dev(), generator=gen) * torch.randn(2000, 1, device=dev(), generator=gen).exp()).to(kind)
    # (halves themselves are common where amax and x have few bits)
    x[::2, ::3] = (x[::2].abs().amax(1, keepdim=True) * 0.5).to(kind)
    q, s = torch.empty(x.shape, dtype=torch.int8, device=dev()), torch.empty(2000, device=dev())
    fp8g.int8_quantize(x, q, s)
    y = x.double() * 127 / x.double().abs().amax(1, keepdim=True)
    assert float((y - q).abs().max()) <= 0.5 + 127 * 2.0 ** -23
    assert int((q.abs() == 127).any(1).sum()) == 2000
    again = torch.empty_like(q)
    fp8g.int8_quantize(x, again, s)
    assert torch.equal(q, again)
