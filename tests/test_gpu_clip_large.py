"""Norm and clipping of lists as large as a model's gradients: more chunks than
workgroups, both chunk sizes, and lists that outgrow the caches."""

import pytest
import torch

import moe_grouped_gemm_quantizer_amd as fp8g
from tests.gpu_util import dev, banner

pytestmark = pytest.mark.gpu

F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16


def check(grads, max_norm):
    """Norm, then clipping out of place and in place, against torch in float64."""
    total = sum(float(x.double().square().sum()) for x in grads)
    ws = torch.full((fp8g.grad_norm_sq_workspace_size(grads),), 0x5A, dtype=torch.uint8, device=dev())
    s, norm = torch.empty(1, dtype=torch.float64, device=dev()), torch.empty(1, device=dev())
    fp8g.grad_norm_sq(grads, s, ws)
    # fp64 sums of at most 2^28 squares, in whatever order: each addition is off by
    # 2^-53 of the total at most, and trees and runs are far shorter than 2^13
    assert abs(s.item() - total) <= 2.0 ** -40 * total
    # (outputs with a guard behind them)
    bufs = [torch.full((x.numel() + 8,), 3.0, dtype=x.dtype, device=dev()) for x in grads]
    outs = [b[:x.numel()] for b, x in zip(bufs, grads)]
    fp8g.grad_clip(grads, outs, s, max_norm, norm)
    n = total ** 0.5
    assert abs(norm.item() - n) <= 2.0 ** -23 * n
    f = min(1.0, max_norm / (n + 1e-6))
    for x, o, b in zip(grads, outs, bufs):
        eps = torch.finfo(o.dtype).eps / 2
        for i in range(0, x.numel(), 1 << 24):
            w = x[i:i + (1 << 24)].double() * f
            off = (o[i:i + (1 << 24)].double() - w).abs()
            # the factor's and the product's rounding to fp32, the type's
            tol = w.abs() * (eps + 2 * 2.0 ** -24 + 2.0 ** -30) + torch.finfo(o.dtype).smallest_normal * eps * 2
            assert bool((off <= tol).all())
        assert (b[x.numel():] == 3).all()
    fp8g.grad_clip(grads, grads, s, max_norm, norm)
    assert all(torch.equal(x, o) for x, o in zip(grads, outs))


def tensors(sizes, types, seed):
    g = torch.Generator(dev()).manual_seed(seed)
    return [(torch.randn(n, device=dev(), generator=g) * 10.0 ** -(i % 3)).to(t)
            for i, (n, t) in enumerate(zip(sizes, types))]


@pytest.mark.parametrize("sizes,types", [
    ([16_777_217, 1, 3_000_001, 8191, 8193], [F32, BF16, F16, F32, BF16]),       # 2,417 chunks of 8192: a second round
    ([7_000_003] * 9, [BF16, F32, F16] * 3),                                     # 63M values, 168 MB
    ([60_000_011, 12_345], [F32, F16]),                                          # over 192 MiB in small chunks
    ([140_000_033, 32_769], [BF16, F32]),                                        # over 134M values: large chunks
    ([1_200_007] * 130, [BF16, F16] * 65),                                       # the same in two launches
])
@pytest.mark.parametrize("max_norm", [0.5, 1e9])
def test_large_lists(sizes, types, max_norm):
    banner(f"clip list of {sum(sizes)} values, max_norm {max_norm}")
    check(tensors(sizes, types, len(sizes)), max_norm)


def test_a_large_list_of_unaligned_views():
    base = tensors([70_000_003, 30_000_001], [F32, BF16], 5)
    check([base[0][1:69_000_000], base[1][3:], base[0][69_000_001:69_999_990]], 0.25)


@pytest.mark.parametrize("total", [65_535, 65_536, 65_537, 131_072, 1_000_000, 1_048_577])
def test_around_the_single_launch(total):
    """Up to 32 chunks of 2048 values are summed by one workgroup."""
    check(tensors([total], [F32], total), 0.5)
    check(tensors([total // 32] * 31 + [total - total // 32 * 31], [BF16] * 32, total), 0.5)
    check(tensors([total // 33] * 32 + [total - total // 33 * 32], [BF16] * 33, total), 0.5)
    check(tensors([total - 4097, 4096, 1], [F32, BF16, F32], total), 0.5)
    check(tensors([total // 112] * 111 + [total - total // 112 * 111], [F16] * 112, total), 0.5)
    check(tensors([total // 113] * 112 + [total - total // 113 * 112], [F16] * 113, total), 0.5)
