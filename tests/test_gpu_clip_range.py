"""Clipping where the factor is below fp32's normal numbers and the clipped
values are not: norms near the end of the types' range."""

import numpy as np
import pytest
import torch

import moe_grouped_gemm_quantizer_amd as fp8g
from oracle import train
from tests.gpu_util import dev

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("t", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("n,max_norm", [(3000, 1.0), (3000, 1e-3), (200_001, 1e-6), (9, 2.0 ** -100), (1, 1e-30)])
def test_factors_below_the_normal_numbers(n, max_norm, t, in_place):
    g = np.random.default_rng(n)
    x = torch.from_numpy(g.uniform(1e38, 3e38, size=n) * g.choice([-1.0, 1.0], size=n)).to(t).to(dev())
    y = torch.tensor([2.0 ** -10, 0.0, -1.0], device=dev())              # clips to nothing
    host = [x.double().cpu().numpy(), y.double().cpu().numpy()]
    total, norm, want = train.grad_clip(host, max_norm)
    s, nrm = torch.empty(1, dtype=torch.float64, device=dev()), torch.empty(1, device=dev())
    ws = torch.empty(fp8g.grad_norm_sq_workspace_size([x, y]), dtype=torch.uint8, device=dev())
    fp8g.grad_norm_sq([x, y], s, ws)
    assert abs(s.item() - total) <= 2.0 ** -40 * total
    outs = [x, y] if in_place else [torch.full_like(x, 3), torch.full_like(y, 3)]
    fp8g.grad_clip([x, y], outs, s, max_norm, nrm)
    for o, w in zip(outs, want):
        eps = torch.finfo(o.dtype).eps / 2
        # the factor's and the product's rounding to fp32, the type's; half a
        # step of the subnormal numbers, once for fp32 and once for the type
        tol = np.abs(w) * (eps + 2 * 2.0 ** -24) * (1 + 2.0 ** -7) + 2.0 ** -150 + 2.0 ** -126 * eps
        off = np.abs(o.double().cpu().numpy() - w)
        assert (off <= tol).all(), float((off / tol).max())
