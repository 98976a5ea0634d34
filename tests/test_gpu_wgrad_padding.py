"""Rows between an expert's last token and the next offset: zeros there are no
part of the weight gradient, and nothing from the last offset on is."""

import pytest
import torch

import moe_grouped_gemm_quantizer_amd as fp8g
from tests.gpu_util import dev

pytestmark = pytest.mark.gpu


def quantised(x, fmt):
    nb = -(-x.shape[0] // 128)
    qt = torch.full((x.shape[1], nb * 128), 0x55, dtype=torch.uint8, device=dev())
    st = torch.full((nb, x.shape[1]), 0x55, dtype=torch.uint8, device=dev())
    fp8g.fp8_quantize_transpose(x, fmt, qt, st)
    return qt, st


def gradient(dy, x, offsets):
    G, M, N = len(offsets) - 1, dy.shape[1], x.shape[1]
    (qa, sa), (qb, sb) = quantised(dy, "e5m2"), quantised(x, "e4m3")
    d = torch.full((G, M, N), float("nan"), dtype=torch.bfloat16, device=dev())
    fp8g.grouped_gemm_fp8_wgrad(qa, "e5m2", sa, qb, "e4m3", sb, d,
                                group_offsets=torch.tensor(offsets, dtype=torch.int32, device=dev()))
    return d


@pytest.mark.parametrize("max_m", [0, 256])
def test_rows_without_a_token(max_m):
    counts, M, N = [130, 0, 1, 255], 48, 80
    g = torch.Generator(dev()).manual_seed(3)
    dy = [torch.randn(n, M, device=dev(), generator=g) for n in counts]
    x = [torch.randn(n, N, device=dev(), generator=g) for n in counts]
    ends = [0]
    for n in counts:
        ends.append(ends[-1] + (max_m or (n + 127) // 128 * 128))
    rows = ends[-1] + 128
    by, bx = torch.zeros(rows, M, device=dev()), torch.zeros(rows, N, device=dev())
    for n, e, u, v in zip(counts, ends, dy, x):
        by[e:e + n], bx[e:e + n] = u, v
    by[ends[-1]:], bx[ends[-1]:] = float("nan"), float("inf")
    d = gradient(by, bx, ends)
    for e, n in enumerate(counts):
        # the expert's tokens alone, bit for bit
        one = gradient(dy[e], x[e], [0, (n + 127) // 128 * 128])[0] if n else torch.zeros_like(d[e])
        assert torch.equal(d[e].view(torch.int16), one.view(torch.int16)), e
    # and a row that is not zero is summed: the caller clears them
    by[ends[1] - 1], bx[ends[1] - 1] = 1.0, 1.0
    assert not torch.equal(gradient(by, bx, ends)[0], d[0])
