"""Global gradient norm and clipping on the GPU against float64."""

import numpy as np
import pytest
import torch

import moe_grouped_gemm_quantizer_amd as fp8g
from oracle import train
from tests.gpu_util import dev

pytestmark = pytest.mark.gpu

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


def tensors(sizes, types, seed, scale=1.0):
    g = np.random.default_rng(seed)
    return [torch.from_numpy(g.normal(size=n) * scale).to(TYPES[t]).to(dev()) for n, t in zip(sizes, types)]


def norm_sq(grads, **kw):
    n = fp8g.grad_norm_sq_workspace_size(grads)
    ws = torch.full((max(n, 8),), 0x5A, dtype=torch.uint8, device=dev())
    s = torch.full((1,), -1.0, dtype=torch.float64, device=dev())
    fp8g.grad_norm_sq(grads, s, ws, **kw)
    return s


def check(grads, max_norm, in_place=False):
    host = [g.double().cpu().numpy() for g in grads]
    total, norm, want = train.grad_clip(host, max_norm)
    s = norm_sq(grads)
    n = torch.full((1,), -1.0, device=dev())
    outs = grads if in_place else [torch.full_like(g, 3.0) for g in grads]
    fp8g.grad_clip(grads, outs, s, max_norm, n)
    # squares of fp32 values are exact in fp64 up to one rounding; chunks of
    # at most 2^31 / 2^8 of them a lane, then trees
    assert abs(s.item() - total) <= 2.0 ** -40 * total
    assert abs(n.item() - norm) <= 2.0 ** -23 * norm
    for o, w in zip(outs, want):
        eps, tiny = torch.finfo(o.dtype).eps / 2, torch.finfo(o.dtype).smallest_normal
        # the factor's rounding to fp32, the product's, and the type's
        tol = np.abs(w) * (eps + 2 * 2.0 ** -24 + 2.0 ** -30) + tiny * eps * 2
        assert (np.abs(o.double().cpu().numpy() - w) <= tol).all()
    if not in_place:
        for g, h in zip(grads, host):
            assert np.array_equal(g.double().cpu().numpy(), h)


@pytest.mark.parametrize("t", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("sizes", [[1], [0], [], [7, 0, 8, 9, 1], [32768], [32767, 32769, 65536 + 5], [3] * 250,
                                   [1000003]])
def test_sizes(sizes, t):
    g = tensors(sizes, [t] * len(sizes), seed=len(sizes))
    check(g, 0.7)
    check(g, 1e6)
    check(g, 0.7, in_place=True)


def test_mixed_types_and_unaligned_views():
    base = tensors([5000, 5000, 5000], ["f32", "bf16", "f16"], 1)
    g = [base[0][1:4001], base[1][3:4900], base[2][8:], base[0][4001:4999], base[1][:3]]
    check(g, 1.0)
    outs = [torch.empty(x.numel() + 1, dtype=x.dtype, device=dev())[1:] for x in g]     # unaligned outputs
    s = norm_sq(g)
    n = torch.empty(1, device=dev())
    fp8g.grad_clip(g, outs, s, 1.0, n)
    again = [torch.empty_like(x) for x in g]
    fp8g.grad_clip(g, again, s, 1.0, n)
    assert all(torch.equal(a, b) for a, b in zip(outs, again))


def test_squares_outside_fp32():
    check(tensors([3000, 40], ["f32", "f32"], 2, 1e30), 1.0)
    check(tensors([3000, 40], ["f32", "bf16"], 3, 1e-30), 1e-32)
    check([torch.zeros(100, device=dev())], 1.0)


def test_nothing_to_clip_leaves_the_gradients_as_they_are():
    g = tensors([4097], ["bf16"], 4, 1e-3)
    h = g[0].clone()
    check(g, 100.0, in_place=True)
    assert torch.equal(g[0].view(torch.int16), h.view(torch.int16))


def test_infinite_and_nan_norms_follow_the_formula():
    g = tensors([500, 500], ["f32", "f32"], 5)
    g[1][7] = float("inf")
    s, n = norm_sq(g), torch.empty(1, device=dev())
    outs = [torch.empty_like(x) for x in g]
    fp8g.grad_clip(g, outs, s, 1.0, n)
    assert n.item() == float("inf") and (outs[0] == 0).all() and torch.isnan(outs[1][7])
    g[1][7] = float("nan")
    fp8g.grad_clip(g, outs, norm_sq(g), 1.0, n)
    assert np.isnan(n.item()) and all(torch.isnan(o).all() for o in outs)


def test_refusals():
    g = tensors([100], ["f32"], 6)
    n, s = torch.empty(1, device=dev()), torch.empty(1, dtype=torch.float64, device=dev())
    with pytest.raises(fp8g.Fp8GemmError):
        fp8g.grad_norm_sq(g, s, None)
    with pytest.raises(fp8g.Fp8GemmError):
        fp8g.grad_clip(g, g, s, 0.0, n)
    with pytest.raises(ValueError):
        fp8g.grad_clip(g, [g[0][:50]], s, 1.0, n)
    with pytest.raises(ValueError):
        fp8g.grad_norm_sq([g[0][::2]], s, None)


def test_the_same_bits_again_on_another_stream_and_in_a_graph():
    g = tensors([40000, 13, 70001], ["f32", "bf16", "f16"], 7)
    outs = [torch.empty_like(x) for x in g]
    ws = torch.empty(fp8g.grad_norm_sq_workspace_size(g), dtype=torch.uint8, device=dev())
    s, n = torch.empty(1, dtype=torch.float64, device=dev()), torch.empty(1, device=dev())

    def step():
        fp8g.grad_norm_sq(g, s, ws)
        fp8g.grad_clip(g, outs, s, 1.0, n)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(4):
        for x, y in zip(g, tensors([40000, 13, 70001], ["f32", "bf16", "f16"], 40 + i, 2.0 + i)):
            x.copy_(y)
        step()
        want = [v.clone() for v in (*outs, s, n)]
        for v in (*outs, s, n):
            v.fill_(9)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, (*outs, s, n))), i
