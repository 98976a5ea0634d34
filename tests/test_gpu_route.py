"""Routing, balance loss and their gradient on the GPU against the float64
oracle: choices, counts, offsets and slots equal; weights, sums, loss and
gradients within bounds that are derived from fp32's rounding."""

import numpy as np
import pytest
import torch

import moe_grouped_gemm_quantizer_amd as fp8g
from oracle import train
from tests.gpu_util import dev

pytestmark = pytest.mark.gpu

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}

# A probability's relative error in fp32: x - max rounds (2^-24 |x - max|, below
# 40 in these tests but for what vanishes), exp is good to 2 ulp, the sum of up
# to 1024 terms takes at most 16 + 6 roundings in a row, a division or product
# two: below 128 half-ulps.
P_REL = 128 * 2.0 ** -24
# a sum over tokens adds at most 4 + 3 roundings in a block, the rest is fp64
S_REL = P_REL + 8 * 2.0 ** -24


def buffers(T, E, k):
    def new(shape, dtype):
        return torch.full(shape, 77, dtype=dtype, device=dev())
    i, f = torch.int32, torch.float32
    return dict(expert_ids=new((T, k), i), weights=new((T, k), f), counts=new((E,), i), routed=new((1,), i),
                prob_sum=new((E,), f), loss=new((1,), f), group_offsets=new((E + 1,), i), slots=new((T, k), i))


def run(x, k, out=None, ws=None, **kw):
    T, E = x.shape
    out = out or buffers(T, E, k)
    n = fp8g.moe_route_workspace_size(T, E)
    ws = ws if ws is not None else (torch.full((n,), 0x5A, dtype=torch.uint8, device=dev()) if n else None)
    fp8g.moe_route(x, k, *out.values(), ws, **kw)
    return out


def logits(T, E, t, seed, closed=0, steps=0):
    g = np.random.default_rng(seed)
    x = g.normal(size=(T, E)) * 2 + g.normal(size=(1, E))
    if steps:                                    # few different values: ties everywhere
        x = np.round(x * steps) / steps
    if closed:
        x[:, g.permutation(E)[:closed]] = -np.inf
    return torch.from_numpy(x).to(TYPES[t]).to(dev())


def check(x, k, got, mask=None, **kw):
    host = {n: v.cpu().numpy() for n, v in got.items()}
    ref = train.route(x.double().cpu().numpy(), k, mask=None if mask is None else mask.cpu().numpy(),
                      renormalise=kw.get("renormalise", False), coef=kw.get("loss_coef", 1.0),
                      align=kw.get("align", 128), max_m=kw.get("max_m", 0))
    for n in ("expert_ids", "counts", "group_offsets", "slots"):
        assert np.array_equal(host[n], ref[n]), n
    assert host["routed"][0] == ref["routed"]
    for n, rel in (("weights", P_REL), ("prob_sum", S_REL), ("loss", S_REL + 2.0 ** -24)):
        # (2^-126: what is below the smallest normal fp32 has fewer bits)
        np.testing.assert_allclose(host[n].astype(np.float64).reshape(np.shape(ref[n]) or (1,)),
                                   ref[n], rtol=rel, atol=2.0 ** -126 * 64, err_msg=n)
    return ref


@pytest.mark.parametrize("t", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (1, 256, 8), (2, 8, 2), (63, 16, 16), (64, 17, 3), (65, 33, 5),
                                   (129, 64, 6), (200, 65, 7), (1000, 128, 8), (77, 255, 16), (300, 257, 4),
                                   (130, 512, 8), (66, 1000, 16), (5, 1024, 16)])
def test_sizes(T, E, k, t):
    x = logits(T, E, t, seed=T * 7 + E)
    check(x, k, run(x, k))
    check(x, k, run(x, k, renormalise=True, loss_coef=0.01), renormalise=True, loss_coef=0.01)


@pytest.mark.parametrize("t", ["f32", "bf16", "f16"])
def test_ties_go_to_the_lower_expert(t):
    x = logits(300, 96, t, seed=1, steps=1)
    x[::3] = 0.25                                # whole rows of one value
    x[1::7, ::2] = -0.0
    x[1::7, 1::2] = 0.0
    check(x, 8, run(x, 8))


@pytest.mark.parametrize("E", [8, 200, 256, 700])
def test_neighbours_that_differ_in_their_last_bits_only(E):
    """fp32 values one or a few ulps apart, equal ones among them, around the
    k-th place too."""
    g = np.random.default_rng(E)
    x = (1.0 + g.integers(0, 40, size=(300, E)) * 2.0 ** -23).astype(np.float32)
    x[1::4] *= -1
    x[2::4] = (g.normal(size=x[2::4].shape) * 2.0 ** g.integers(-60, 60, size=(x[2::4].shape[0], 1))).astype(np.float32)
    x[3::8, : E // 2] = 3.0
    x = torch.from_numpy(x).to(dev())
    for k in (1, min(E, 7), min(E, 16)):
        check(x, k, run(x, k))
    check(x[:3], min(E, 16), run(x[:3], min(E, 16)))


def test_every_expert_is_chosen_when_k_is_all_of_them():
    for E in (1, 2, 15, 16):
        x = logits(70, E, "f32", seed=E)
        check(x, E, run(x, E, renormalise=True), renormalise=True)
        x = logits(3, E, "bf16", seed=E, steps=1)
        check(x, E, run(x, E))


@pytest.mark.parametrize("t", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("T", [50, 500])
def test_masks_closed_experts_and_empty_rows(T, t):
    x = logits(T, 24, t, seed=2, closed=9)
    x[3::11] = -float("inf")                     # nothing to choose
    x[4::11, 1:] = -float("inf")                 # at most one
    x[5::11] = torch.finfo(TYPES[t]).min         # masks of the type's lowest value
    x[6::11, :20] = torch.finfo(TYPES[t]).min
    mask = torch.rand(T, device=dev(), generator=torch.Generator(dev()).manual_seed(3)) > 0.3
    mask[:2] = False
    for kw in (dict(), dict(renormalise=True, max_m=16), dict(align=1), dict(align=16, max_m=3)):
        check(x, 6, run(x, 6, token_mask=mask, **kw), mask=mask, **kw)
    nobody = torch.zeros(T, dtype=torch.uint8, device=dev())
    check(x, 6, run(x, 6, token_mask=nobody), mask=nobody)
    # what a masked token's logits hold does not matter
    y = x.clone()
    y[~mask] = float("nan")
    a, b = run(x, 6, token_mask=mask), run(y, 6, token_mask=mask)
    assert all(torch.equal(a[n], b[n]) for n in a)


@pytest.mark.parametrize("t", ["f32", "bf16", "f16"])
def test_nan_and_infinite_logits(t):
    x = logits(100, 40, t, seed=4)
    x[7, 3] = x[50] = float("nan")
    x[90, 5] = float("inf")
    got = run(x, 4, renormalise=True)
    ref = train.route(x.double().cpu().numpy(), 4, renormalise=True)
    for n in ("expert_ids", "counts", "group_offsets", "slots"):
        assert np.array_equal(got[n].cpu().numpy(), ref[n]), n
    w = got["weights"].cpu().numpy()
    bad = np.isin(np.arange(100), [7, 50, 90])
    assert np.isnan(w[bad]).all() and np.isfinite(w[~bad]).all()
    assert np.isnan(got["loss"].item()) and torch.isnan(got["prob_sum"]).all()


def test_no_tokens():
    x = torch.empty(0, 8, device=dev())
    for kw in (dict(), dict(max_m=5)):
        check(x, 2, run(x, 2, **kw), **kw)


@pytest.mark.parametrize("t", ["f32", "bf16"])
def test_strided_and_unaligned_rows(t):
    big = logits(200, 61, t, seed=5)
    x = big[:, 1:38]                             # rows 61 apart, an odd start
    check(x, 5, run(x, 5, renormalise=True), renormalise=True)
    out = torch.full((200, 61), 9.0, device=dev(), dtype=TYPES[t])
    got = run(x, 5)
    dw = torch.randn(200, 5, device=dev())
    dl = torch.ones(1, device=dev())
    fp8g.moe_route_backward(x, got["expert_ids"], dw, dl, got["counts"], got["routed"], out[:, 3:40])
    dense = torch.empty(200, 37, device=dev(), dtype=TYPES[t])
    fp8g.moe_route_backward(x.contiguous(), got["expert_ids"], dw, dl, got["counts"], got["routed"], dense)
    assert torch.equal(out[:, 3:40], dense)
    assert (out[:, :3] == 9).all() and (out[:, 40:] == 9).all()


def test_many_tokens_and_the_same_bits_again():
    x = logits(20011, 72, "bf16", seed=6, closed=2, steps=4)
    a = run(x, 8, renormalise=True, loss_coef=0.01)
    check(x, 8, a, renormalise=True, loss_coef=0.01)
    b = run(x, 8, renormalise=True, loss_coef=0.01)
    assert all(torch.equal(a[n], b[n]) for n in a)


def test_too_small_a_workspace_is_refused():
    x = logits(300, 8, "f32", seed=7)
    with pytest.raises(fp8g.Fp8GemmError):
        run(x, 2, ws=torch.empty(16, dtype=torch.uint8, device=dev()))
    with pytest.raises(ValueError):
        run(x, 2, out={**buffers(300, 8, 2), "slots": torch.empty(300, 3, dtype=torch.int32, device=dev())})


def test_on_another_stream_and_in_a_graph():
    x = logits(700, 40, "f32", seed=8)
    k = 4
    out, ws = buffers(700, 40, k), torch.empty(fp8g.moe_route_workspace_size(700, 40), dtype=torch.uint8,
                                               device=dev())
    dx, dw, dl = torch.empty_like(x), torch.randn(700, k, device=dev()), torch.ones(1, device=dev())

    def both():
        run(x, k, out, ws)
        fp8g.moe_route_backward(x, out["expert_ids"], dw, dl, out["counts"], out["routed"], dx)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        both()
    torch.cuda.synchronize()
    check(x, k, out)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        both()
    for i in range(4):
        x.copy_(logits(700, 40, "f32", seed=20 + i))
        both()
        want = [v.clone() for v in out.values()] + [dx.clone()]
        for v in (*out.values(), dx):
            v.fill_(3)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, (*out.values(), dx))), i


@pytest.mark.parametrize("t", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (1, 256, 8), (3, 8, 2), (65, 17, 16), (200, 65, 7), (1000, 128, 8),
                                   (300, 257, 4), (66, 1000, 16)])
@pytest.mark.parametrize("renorm", [False, True])
def test_gradient(T, E, k, t, renorm):
    x = logits(T, E, t, seed=T + E, closed=E // 3)
    if T > 10:
        x[3::7] = -float("inf")
        x[4::7, 2:] = -float("inf")
    g = np.random.default_rng(T)
    dw, dl = torch.from_numpy(g.normal(size=(T, k)).astype(np.float32)), 2.5
    ref = train.route(x.double().cpu().numpy(), k, renormalise=renorm)
    ids, counts = torch.from_numpy(ref["expert_ids"]).to(dev()), torch.from_numpy(ref["counts"]).to(dev())
    routed = torch.tensor([ref["routed"]], dtype=torch.int32, device=dev())
    dx = torch.full_like(x, 5.0)
    fp8g.moe_route_backward(x, ids, dw.to(dev()), torch.tensor([dl], device=dev()), counts, routed, dx,
                            renormalise=renorm, loss_coef=0.3)
    want, size = train.route_backward(x.double().cpu().numpy(), ref["expert_ids"], dw.numpy(), dl, ref["counts"],
                                      ref["routed"], renorm, 0.3)
    # each of the terms of `size` carries a probability's error twice (its
    # own factor and the sum's), with renormalise twice more (division by a
    # sum of them, and the weights'); then one rounding to the type
    eps = torch.finfo(TYPES[t]).eps / 2
    tiny = torch.finfo(TYPES[t]).smallest_normal * eps
    tol = 4 * P_REL * size * (1 + eps) + eps * np.abs(want) + tiny
    off = np.abs(dx.double().cpu().numpy() - want)
    assert (off <= tol).all(), float((off / tol).max())
    # without one of the two gradients
    for a, b in ((None, torch.tensor([dl], device=dev())), (dw.to(dev()), None)):
        fp8g.moe_route_backward(x, ids, a, b, counts, routed, dx, renormalise=renorm, loss_coef=0.3)
        want, size = train.route_backward(x.double().cpu().numpy(), ref["expert_ids"],
                                          dw.numpy() * (a is not None), dl * (b is not None), ref["counts"],
                                          ref["routed"], renorm, 0.3)
        tol = 4 * P_REL * size * (1 + eps) + eps * np.abs(want) + tiny
        assert (np.abs(dx.double().cpu().numpy() - want) <= tol).all()
