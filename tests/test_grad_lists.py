"""Lists of gradients given as iterators: gone through once, so that what is
checked is what is used."""

import pytest
import torch

import moe_grouped_gemm_quantizer_amd as fp8g


def _kinds(ts):
    """The same tensors as iterables of every kind."""
    return [list(ts), tuple(ts), (t for t in ts), map(lambda t: t, ts), iter(ts), {i: t for i, t in enumerate(ts)}.values()]


def test_iterators_of_tensors_off_the_gpu_are_refused():
    ts = [torch.zeros(4), torch.zeros(5)]
    total, norm = torch.zeros(1, dtype=torch.float64), torch.zeros(1)
    for g in _kinds(ts):
        with pytest.raises(ValueError, match="grads must be contiguous and on the GPU"):
            fp8g.grad_norm_sq(g, total, None)
    for g in _kinds(ts):
        with pytest.raises(ValueError, match="grads must be contiguous and on the GPU"):
            fp8g.grad_clip(g, g, total, 1.0, norm)


def test_workspace_size_of_an_iterator():
    ts = [torch.zeros(200_000), torch.zeros(7)]
    want = fp8g.grad_norm_sq_workspace_size(ts)
    assert want > 0
    assert all(fp8g.grad_norm_sq_workspace_size(g) == want for g in _kinds(ts))


@pytest.mark.gpu
def test_iterators_give_the_lists_results():
    g = torch.Generator("cuda").manual_seed(1)
    ts = [torch.randn(n, device="cuda", generator=g) for n in (5000, 1, 300_001)]
    ws = torch.empty(fp8g.grad_norm_sq_workspace_size(ts), dtype=torch.uint8, device="cuda")
    total, norm = torch.empty(1, dtype=torch.float64, device="cuda"), torch.empty(1, device="cuda")
    want = sum(float(t.double().square().sum()) for t in ts)
    f = min(1.0, 3.0 / (want ** 0.5 + 1e-6))
    for grads, again, outs in zip(_kinds(ts), _kinds(ts), range(6)):
        total.fill_(-1)
        fp8g.grad_norm_sq(grads, total, ws)
        assert abs(float(total) - want) <= 2.0 ** -40 * want
        dst = [torch.zeros_like(t) for t in ts]
        fp8g.grad_clip(again, _kinds(dst)[outs], total, 3.0, norm)
        for t, d in zip(ts, dst):
            # (the factor's and the product's rounding to fp32)
            assert (d.double() - t.double() * f).abs().max() <= 2 ** -22 * float(t.abs().max()) * f
    # one iterator as both: in place
    for k in range(6):
        mine = [t.clone() for t in ts]
        it = _kinds(mine)[k]
        fp8g.grad_clip(it, it, total, 3.0, norm)
        assert all(torch.equal(m, d) for m, d in zip(mine, dst))
