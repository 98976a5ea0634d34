"""Routing of more tokens than one launch of the rows' kernel holds."""

import pytest
import torch

import moe_grouped_gemm_quantizer_amd as fp8g
from tests.gpu_util import dev, banner

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("E,T", [(2, (1 << 28) + 12345)])
def test_more_tokens_than_a_launch_holds(E, T):
    """64 tokens a workgroup of 1024 threads: from 2^28 tokens on more than the
    2^32 threads that a launch may have."""
    banner(f"route T={T} E={E}")
    g = torch.Generator(dev()).manual_seed(1)
    x = torch.randn(T, E, device=dev(), generator=g, dtype=torch.bfloat16)

    def new(shape, dtype):
        return torch.full(shape, 77, dtype=dtype, device=dev())
    i, f = torch.int32, torch.float32
    out = dict(expert_ids=new((T, 1), i), weights=new((T, 1), f), counts=new((E,), i), routed=new((1,), i),
               prob_sum=new((E,), f), loss=new((1,), f), group_offsets=new((E + 1,), i), slots=new((T, 1), i))
    ws = torch.full((fp8g.moe_route_workspace_size(T, E),), 0x5A, dtype=torch.uint8, device=dev())
    fp8g.moe_route(x, 1, *out.values(), ws)
    second = x[:, 1] > x[:, 0]                            # (ties to the lower expert)
    ids = out["expert_ids"][:, 0]
    assert torch.equal(ids == 1, second) and bool(((ids == 0) | (ids == 1)).all())
    n1 = int(second.sum())
    assert out["counts"].tolist() == [T - n1, n1] and out["routed"].item() == T
    ends = [0, (T - n1 + 127) // 128 * 128]
    ends.append(ends[1] + (n1 + 127) // 128 * 128)
    assert out["group_offsets"].tolist() == ends
    rank = torch.cumsum(second, 0)                        # tokens of expert 1 up to here
    at = torch.arange(T, device=dev())
    assert torch.equal(out["slots"][:, 0].long(), torch.where(second, ends[1] + rank - 1, at - rank))
    del rank, at
    p1 = torch.sigmoid(x[:, 1].double() - x[:, 0].double())
    want = torch.stack([(1 - p1).sum(), p1.sum()])
    # (a probability's roundings, and those of the sums over a block: below 32 halves of an ulp)
    assert ((out["prob_sum"].double() - want).abs() <= 32 * 2.0 ** -24 * want).all()
    top = torch.where(second, p1, 1 - p1)
    assert ((out["weights"][:, 0].double() - top).abs() <= 32 * 2.0 ** -24 * top).all()
