"""Routing and its gradient in every kernel variant and at the sizes where a
loop inside a kernel goes round again, against the many-row reference."""

import numpy as np
import pytest
import torch

import moe_grouped_gemm_quantizer_amd as fp8g
from tests import route_ref
from tests.gpu_util import dev, banner
from tests.test_gpu_route import P_REL, S_REL, TYPES, run

pytestmark = pytest.mark.gpu


def logits(T, E, t, seed, closed=0, empty=False):
    g = torch.Generator(dev()).manual_seed(seed)
    x = torch.randn(T, E, device=dev(), generator=g) * 2 + torch.randn(1, E, device=dev(), generator=g)
    if closed:
        x[:, torch.randperm(E, device=dev(), generator=g)[:closed]] = -float("inf")
    if empty:
        x[3::11] = -float("inf")
        x[4::11, 2:] = -float("inf")
    return x.to(TYPES[t])


def token_mask(T, seed):
    return torch.rand(T, device=dev(), generator=torch.Generator(dev()).manual_seed(seed)) > 0.2


def check(x, k, got, mask=None, **kw):
    ref = route_ref.route(x.double().cpu().numpy(), k, mask=None if mask is None else mask.cpu().numpy(),
                          renormalise=kw.get("renormalise", False), coef=kw.get("loss_coef", 1.0),
                          align=kw.get("align", 128), max_m=kw.get("max_m", 0))
    host = {n: v.cpu().numpy() for n, v in got.items()}
    for n in ("expert_ids", "counts", "group_offsets", "slots"):
        assert np.array_equal(host[n], ref[n]), n
    assert host["routed"][0] == ref["routed"]
    for n, rel in (("weights", P_REL), ("prob_sum", S_REL), ("loss", S_REL + 2.0 ** -24)):
        np.testing.assert_allclose(host[n].astype(np.float64).reshape(np.shape(ref[n]) or (1,)), ref[n], rtol=rel,
                                   atol=2.0 ** -126 * 64, err_msg=n)
    return ref


def check_gradient(x, k, ref, t, renorm, seed):
    T, E = x.shape
    g = np.random.default_rng(seed)
    dw, dl = g.normal(size=(T, k)).astype(np.float32), 2.5
    ids, counts = torch.from_numpy(ref["expert_ids"]).to(dev()), torch.from_numpy(ref["counts"]).to(dev())
    dx = torch.full_like(x, 5.0)
    fp8g.moe_route_backward(x, ids, torch.from_numpy(dw).to(dev()), torch.tensor([dl], device=dev()), counts,
                            torch.tensor([ref["routed"]], dtype=torch.int32, device=dev()), dx, renormalise=renorm,
                            loss_coef=0.3)
    want, size = route_ref.route_backward(x.double().cpu().numpy(), ref["expert_ids"], dw, dl, ref["counts"],
                                          ref["routed"], renorm, 0.3)
    # (as for the small sizes: a probability's error in each term, renormalising
    # twice more, and one rounding to the type)
    eps = torch.finfo(TYPES[t]).eps / 2
    tol = 4 * P_REL * size * (1 + eps) + eps * np.abs(want) + torch.finfo(TYPES[t]).smallest_normal * eps
    off = np.abs(dx.double().cpu().numpy() - want)
    assert (off <= tol).all(), float((off / tol).max())


@pytest.mark.parametrize("t", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("T,E,k", [(4, 256, 8), (5, 256, 8), (4, 130, 3), (6, 129, 16), (300, 48, 5), (200, 130, 7),
                                   (333, 160, 6), (130, 192, 16), (130, 193, 2), (260, 200, 8), (129, 256, 8),
                                   (4, 300, 5), (200, 512, 4), (70, 513, 9)])
def test_every_kernel(T, E, k, t):
    x = logits(T, E, t, T * E, closed=E // 4, empty=T > 10)
    mask = token_mask(T, E) if T > 10 else None
    for renorm in (False, True):
        kw = dict(renormalise=renorm, loss_coef=0.3)
        ref = check(x, k, run(x, k, token_mask=mask, **kw), mask=mask, **kw)
        check_gradient(x, k, ref, t, renorm, T)


@pytest.mark.parametrize("T,E,k,t,renorm", [(20011, 24, 4, "bf16", True), (33001, 40, 3, "f32", False),
                                            (33001, 160, 6, "f32", True), (20011, 200, 8, "f16", False),
                                            (17003, 256, 2, "bf16", True), (9001, 300, 5, "f32", True),
                                            (5003, 1000, 16, "bf16", False)])
def test_rows_in_several_rounds(T, E, k, t, renorm):
    """The backward pass walks rows with the next ones' loads on their way:
    more rows than one round of its workgroups takes."""
    banner(f"route rounds T={T} E={E}")
    x = logits(T, E, t, T + E, closed=E // 8, empty=True)
    mask = token_mask(T, E)
    kw = dict(renormalise=renorm, loss_coef=0.3)
    ref = check(x, k, run(x, k, token_mask=mask, **kw), mask=mask, **kw)
    check_gradient(x, k, ref, t, renorm, T)


@pytest.mark.parametrize("T,E,k,max_m", [(30000, 24, 6, 0), (30000, 24, 6, 5000), (8000, 300, 4, 100),
                                         (3000, 256, 8, 0), (2100, 255, 8, 64), (70001, 20, 2, 0),
                                         (40003, 31, 3, 3000), (66001, 100, 1, 0), (131073, 8, 2, 20000)])
def test_scans_of_many_blocks(T, E, k, max_m):
    """Tables of counts too large for the joined launch, runs of more than one
    batch of blocks, and both layouts behind them."""
    banner(f"route blocks T={T} E={E}")
    x = logits(T, E, "bf16", T - E, empty=True)
    mask = token_mask(T, E)
    kw = dict(max_m=max_m, align=64)
    check(x, k, run(x, k, token_mask=mask, **kw), mask=mask, **kw)
