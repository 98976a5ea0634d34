"""Routing by scores on the GPU against NumPy in 64 bits."""

import numpy as np
import pytest
import torch

import moe_grouped_gemm_quantizer_amd as fp8g
from tests import route_scored_ref as ref
from tests.gpu_util import dev

pytestmark = pytest.mark.gpu

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


def outputs(T, E, k):
    i32 = torch.int32

    def new(shape, dtype=torch.float32):
        return torch.full(shape, 77, dtype=dtype, device=dev())
    return dict(expert_ids=new((T, k), i32), weights=new((T, k)), counts=new((E,), i32), routed=new((1,), i32),
                prob_sum=new((E,)), loss=new((1,)), group_offsets=new((E + 1,), i32), slots=new((T, k), i32))


def call(x, k, bias=None, score="sigmoid", groups=1, opened=1, best=1, mask=None, renorm=False, scale=1.0,
         coef=0.01, align=128, max_m=0, **kw):
    T, E = x.shape
    o = outputs(T, E, k)
    n = fp8g.moe_route_workspace_size(T, E)
    ws = torch.full((n,), 0x5A, dtype=torch.uint8, device=dev()) if n else None
    fp8g.moe_route_scored(x, k, *o.values(), ws, score=score, bias=bias, groups=groups, open_groups=opened,
                          group_best=best, token_mask=mask, renormalise=renorm, scale=scale, loss_coef=coef,
                          align=align, max_m=max_m, **kw)
    return o


def check(x, k, bias=None, score="sigmoid", groups=1, opened=1, best=1, mask=None, renorm=False, scale=1.0,
          coef=0.01, align=128, max_m=0):
    """x: a GPU tensor (rows may be strided); bias, mask: NumPy or None."""
    o = call(x, k, None if bias is None else torch.from_numpy(bias).to(dev()), score, groups, opened, best,
             None if mask is None else torch.from_numpy(mask).to(dev()), renorm, scale, coef, align, max_m)
    w = ref.route(x.double().cpu().numpy(), bias, score, groups, opened, best, k, renorm, scale, coef, align, max_m,
                  mask)
    got = {name: t.cpu().numpy() for name, t in o.items()}
    assert np.array_equal(got["expert_ids"], w["expert_ids"])
    for name in ("counts", "routed", "group_offsets", "slots"):
        assert np.array_equal(got[name].astype(np.int64).reshape(-1), np.asarray(w[name]).reshape(-1)), name
    # a score: 4 ulp of sigmoid; softmax's exponential 2, its sum's terms 2 and up to 22 additions, a
    # division and a product; the chosen ones' sum 5 additions more; division, scale
    u = 2.0 ** -24
    tol = (48 if score == "softmax" else 24) * u
    for name, more in (("weights", 0), ("prob_sum", 80), ("loss", 90)):     # rows of a block, waves, blocks
        a, b = got[name].astype(np.float64).reshape(-1), np.asarray(w[name], np.float64).reshape(-1)
        assert np.array_equal(np.isnan(a), np.isnan(b)), name
        ok = ~np.isnan(b)
        assert (np.abs(a - b)[ok] <= (tol + more * u) * np.abs(b[ok]) + 2.0 ** -126).all(), name
    return got


def logits(rng, T, E, kind="f32", spread=1.5, shift=-1.0):
    return torch.from_numpy(rng.standard_normal((T, E)) * spread + shift).to(TYPES[kind]).to(dev())


def some_bias(rng, E):
    return (np.round(rng.standard_normal(E) * 50) * 1e-3).astype(np.float32)


SHAPES = [(1, 1, 1), (2, 1, 2), (16, 4, 3), (20, 5, 4), (32, 8, 6), (60, 3, 8), (64, 16, 6), (100, 4, 8), (128, 32, 8),
          (160, 8, 6), (192, 12, 16), (250, 5, 8), (256, 8, 8), (300, 6, 7), (512, 32, 16), (1000, 25, 4), (1024, 16, 16)]


@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("E,groups,k", SHAPES)
@pytest.mark.parametrize("T", [1, 4, 5, 64, 65, 333])
def test_shapes(T, E, groups, k, kind):
    rng = np.random.default_rng(T * 7 + E)
    size = E // groups
    opened = max(-(-k // size), groups // 2, 1)
    check(logits(rng, T, E, kind), k, some_bias(rng, E), "sigmoid", groups, opened, min(2, size), renorm=True, scale=2.5)
    check(logits(rng, T, E, kind), k, some_bias(rng, E) * 0.1, "softmax", groups, opened, 1, scale=1.5)


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("with_bias", [False, True])
@pytest.mark.parametrize("groups,opened,best", [(1, 1, 1), (8, 8, 2), (8, 1, 1), (8, 3, 2), (32, 5, 1)])
@pytest.mark.parametrize("renorm,max_m", [(True, 0), (False, 40)])
def test_options(score, with_bias, groups, opened, best, renorm, max_m):
    rng = np.random.default_rng(groups + opened)
    T, E = 200, 96 if groups != 32 else 128
    k = min(6, opened * (E // groups))
    x = logits(rng, T, E)
    x[:, rng.permutation(E)[:9]] = -torch.inf
    mask = rng.random(T) > 0.3
    check(x, k, some_bias(rng, E) if with_bias else None, score, groups, opened, best, mask, renorm, 0.7, 1.0, 128, max_m)


def test_softmax_without_bias_and_groups_is_moe_route():
    rng = np.random.default_rng(4)
    for T, E, k in ((3, 40, 4), (500, 256, 8)):
        x = logits(rng, T, E)
        a = call(x, k, score="softmax", renorm=True)
        b = outputs(T, E, k)
        n = fp8g.moe_route_workspace_size(T, E)
        fp8g.moe_route(x, k, *b.values(), torch.empty(n, dtype=torch.uint8, device=dev()) if n else None,
                       renormalise=True, loss_coef=0.01)
        for name in ("expert_ids", "counts", "routed", "group_offsets", "slots"):
            assert torch.equal(a[name], b[name]), name
        assert torch.allclose(a["weights"], b["weights"], rtol=2.0 ** -20, atol=0)


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("E,groups", [(16, 1), (64, 8), (256, 8), (512, 16)])
def test_values_nearer_than_fp32_tells(E, groups, score):
    """Biases that bring many experts' values within an fp32 step of each other: the order
    is the one of 64 bits."""
    rng = np.random.default_rng(E)
    x = rng.standard_normal((1, E)).astype(np.float32).astype(np.float64)
    s = ref.scores(x, score)[0]
    bias = (1.5 - s).astype(np.float32)                # s + bias: 1.5 within half a step of 2^-24
    x = np.repeat(x, 70, 0)
    x[1::3] += np.float32(2.0 ** -20) * rng.integers(-2, 3, (len(x[1::3]), E))
    x = torch.from_numpy(x).float().to(dev())
    check(x, min(8, E // groups), bias, score, groups, max(1, groups // 2), 2)


@pytest.mark.parametrize("kind", ["f32", "bf16"])
def test_ties(kind):
    """Equal logits with equal biases, equal groups: the lower index first."""
    rng = np.random.default_rng(6)
    x = torch.from_numpy(rng.integers(-2, 3, (150, 64)).astype(np.float64)).to(TYPES[kind]).to(dev())
    bias = (rng.integers(-1, 2, 64) * 0.25).astype(np.float32)
    check(x, 8, bias, "sigmoid", 8, 3, 2)
    check(x, 8, None, "sigmoid", 8, 3, 2)
    check(torch.zeros(70, 64, device=dev()), 8, np.zeros(64, np.float32), "sigmoid", 8, 3, 2)
    check(torch.zeros(70, 64, device=dev()), 8, np.zeros(64, np.float32), "softmax", 8, 3, 1)
    check(torch.full((70, 300), 50.0, device=dev()), 4, None, "sigmoid", 10, 2, 2)


def test_large_and_odd_biases():
    rng = np.random.default_rng(7)
    x = logits(rng, 130, 64)
    check(x, 6, (rng.standard_normal(64) * 100).astype(np.float32), "sigmoid", 8, 4, 2)
    b = some_bias(rng, 64)
    b[3], b[9], b[20], b[21] = np.inf, -np.inf, np.nan, np.inf
    check(x, 6, b, "sigmoid", 1, 1, 1)
    check(x, 6, b, "sigmoid", 8, 4, 1)
    check(x, 6, np.full(64, -np.inf, np.float32), "sigmoid", 8, 4, 1)
    check(x, 6, np.full(64, 3e38, np.float32), "sigmoid", 1, 1, 1)
    check(x * 0 - 200, 6, np.zeros(64, np.float32), "sigmoid", 8, 2, 2)          # (scores of 0)
    check(x, 6, (b * 0 + 1e-38).astype(np.float32) * np.isfinite(b), "sigmoid", 8, 2, 1)


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("with_bias", [False, True])
def test_rows_that_are_not_finite(score, with_bias):
    rng = np.random.default_rng(8)
    x = logits(rng, 100, 32)
    x[3] = -torch.inf
    x[10, 5], x[11, 6], x[12] = torch.nan, torch.inf, torch.nan
    x[13, :31] = -torch.inf
    x[14, 4:8] = -torch.inf
    mask = np.ones(100, bool)
    mask[12] = mask[50] = False
    b = some_bias(rng, 32) if with_bias else None
    got = check(x, 4, b, score, 8, 8, 1, mask)
    assert (got["expert_ids"][3] == -1).all() and np.isnan(got["weights"][10]).all()
    check(x, 4, b, score, 8, 2, 2, mask)
    mask[10] = mask[11] = False
    got = check(x, 4, b, score, 8, 2, 2, mask, renorm=True)
    assert np.isfinite(got["loss"]).all()


def test_strided_and_unaligned_rows():
    rng = np.random.default_rng(9)
    for kind in TYPES:
        buf = torch.full((70, 130), 99.0, dtype=TYPES[kind], device=dev())
        view = buf[:, 3:103]
        view.copy_(logits(rng, 70, 100, kind))
        check(view, 5, some_bias(rng, 100), "sigmoid", 10, 4, 2)


def test_no_tokens():
    o = call(torch.empty(0, 16, device=dev()), 2, groups=4, opened=2, best=2)
    assert int(o["counts"].abs().sum()) == 0 and int(o["routed"]) == 0 and float(o["loss"]) == 0.0
    assert int(o["group_offsets"].abs().sum()) == 0


def test_many_tokens():
    """Blocks scanned in every way: few and many, large tables."""
    rng = np.random.default_rng(10)
    for T, E, groups, k in ((4096, 8, 2, 2), (5000, 256, 8, 8), (3001, 600, 12, 3)):
        x = logits(rng, T, E, "bf16")
        check(x, k, some_bias(rng, E), "sigmoid", groups, groups // 2, 2, rng.random(T) > 0.1, True, 2.5)


def gradient(x, o, dw, dloss, **kw):
    d = torch.full_like(x, 55.0)
    fp8g.moe_route_scored_backward(x, o["expert_ids"], dw, dloss, o["counts"], o["routed"], d, **kw)
    return d


@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("T,E,groups,k", [(1, 4, 1, 1), (3, 256, 8, 8), (70, 16, 4, 4), (130, 60, 3, 5), (40, 100, 4, 1),
                                          (33, 160, 8, 6), (300, 256, 8, 8), (20, 500, 4, 16), (9, 1024, 32, 16)])
def test_gradient(T, E, groups, k, score, renorm, kind):
    rng = np.random.default_rng(T + E + k)
    x = logits(rng, T, E, kind)
    if E > 8:
        x[:, 2] = -torch.inf
    mask = torch.from_numpy(rng.random(T) > 0.2).to(dev()) if T > 1 else None
    bias = torch.from_numpy(some_bias(rng, E)).to(dev())
    o = call(x, k, bias, score, groups, max(-(-k // (E // groups)), groups // 2, 1), 1, mask, renorm, 2.5)
    dw = torch.from_numpy(rng.standard_normal((T, k))).float().to(dev())
    dloss = torch.full((1,), 3.0, device=dev())
    coef = 100.0                                       # (the loss's part about as large as the weights')
    got = gradient(x, o, dw, dloss, score=score, renormalise=renorm, scale=2.5, loss_coef=coef)
    want, size = ref.backward(x.double().cpu().numpy(), o["expert_ids"].cpu().numpy(), dw.double().cpu().numpy(), 3.0,
                              o["counts"].cpu().numpy(), int(o["routed"]), score, renorm, 2.5, coef)
    fi = torch.finfo(x.dtype)
    # scores' errors (as above), sums of up to 22 additions twice, a dozen products
    tol = 96 * 2.0 ** -24 * size + fi.eps / 2 * np.abs(want) + fi.smallest_normal * fi.eps / 2
    assert (np.abs(got.double().cpu().numpy() - want) <= tol).all()
    # either gradient alone
    a = gradient(x, o, dw, None, score=score, renormalise=renorm, scale=2.5, loss_coef=coef)
    b = gradient(x, o, None, dloss, score=score, renormalise=renorm, scale=2.5, loss_coef=coef)
    wa, sa = ref.backward(x.double().cpu().numpy(), o["expert_ids"].cpu().numpy(), dw.double().cpu().numpy(), 0.0,
                          o["counts"].cpu().numpy(), int(o["routed"]), score, renorm, 2.5, coef)
    assert (np.abs(a.double().cpu().numpy() - wa) <= 96 * 2.0 ** -24 * sa + fi.eps / 2 * np.abs(wa)
            + fi.smallest_normal * fi.eps / 2).all()
    assert (np.abs(b.double().cpu().numpy() - (want - wa)) <= 96 * 2.0 ** -24 * size + fi.eps / 2 * np.abs(want - wa)
            + fi.smallest_normal * fi.eps / 2).all()


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
def test_gradient_far_from_the_middle(score):
    """Logits of +-30: s (1 - s) does not lose what 1 - s would."""
    x = torch.tensor([[30.0, -30.0, 12.0, 0.0], [25.0, 25.0, 25.0, 20.0]], device=dev())
    o = call(x, 2, None, score)
    dw = torch.tensor([[1.0, -2.0], [0.5, 1.0]], device=dev())
    got = gradient(x, o, dw, None, score=score).double().cpu().numpy()
    want, size = ref.backward(x.double().cpu().numpy(), o["expert_ids"].cpu().numpy(), dw.double().cpu().numpy(), 0.0,
                              o["counts"].cpu().numpy(), 2, score, False, 1.0, 1.0)
    tol = 96 * 2.0 ** -24 * (size if score == "softmax" else np.abs(want))
    assert (np.abs(got - want) <= tol + 2.0 ** -140).all()


def test_gradient_of_one_chosen_weight_is_zero():
    """A single renormalised weight is 1 whatever the logits."""
    rng = np.random.default_rng(12)
    x = logits(rng, 100, 24)
    o = call(x, 1, None, "sigmoid", renorm=True)
    got = gradient(x, o, torch.ones(100, 1, device=dev()), None, renormalise=True)
    assert (got == 0).all()


def test_gradient_strided_and_ids_out_of_range():
    rng = np.random.default_rng(13)
    buf = torch.zeros(50, 40, device=dev())
    x = buf[:, 1:25]
    x.copy_(logits(rng, 50, 24))
    o = call(x, 3, None, "sigmoid", 4, 2, 2)
    ids = o["expert_ids"].clone()
    ids[4] = torch.tensor([-7, 3, 4], dtype=torch.int32)
    ids[5, 2] = 1000
    o["expert_ids"] = ids
    out = torch.full((50, 40), 9.0, device=dev())
    dw = torch.ones(50, 3, device=dev())
    fp8g.moe_route_scored_backward(x, ids, dw, None, o["counts"], o["routed"], out[:, 2:26])
    ids = torch.where((ids < 0) | (ids >= 24), -1, ids).cpu().numpy()
    want, size = ref.backward(x.double().cpu().numpy(), ids, np.ones((50, 3)), 0.0, o["counts"].cpu().numpy(),
                              int(o["routed"]), "sigmoid", False, 1.0, 1.0)
    got = out.double().cpu().numpy()
    assert (np.abs(got[:, 2:26] - want) <= 97 * 2.0 ** -24 * size).all()
    assert (got[:, :2] == 9).all() and (got[:, 26:] == 9).all() and (got[4, 2:26] == 0).all()


def test_captured_and_replayed():
    rng = np.random.default_rng(14)
    T, E, k = 500, 64, 6
    x = logits(rng, T, E)
    bias = torch.from_numpy(some_bias(rng, E)).to(dev())
    ws = torch.empty(fp8g.moe_route_workspace_size(T, E), dtype=torch.uint8, device=dev())
    dw, dl = torch.randn(T, k, device=dev()), torch.ones(1, device=dev())

    def step(o, d):
        fp8g.moe_route_scored(x, k, *o.values(), ws, bias=bias, groups=8, open_groups=4, group_best=2, renormalise=True)
        fp8g.moe_route_scored_backward(x, o["expert_ids"], dw, dl, o["counts"], o["routed"], d, renormalise=True)
    a, b = outputs(T, E, k), outputs(T, E, k)
    da, db = torch.empty_like(x), torch.empty_like(x)
    step(a, da)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(a, da)
    for _ in range(4):
        x.normal_()
        bias.normal_(std=0.05)
        graph.replay()
        torch.cuda.synchronize()
        step(b, db)
        torch.cuda.synchronize()
        assert all(torch.equal(a[n], b[n]) for n in a) and torch.equal(da, db)


def test_same_bits_twice_and_another_stream():
    rng = np.random.default_rng(15)
    x = logits(rng, 3000, 128)
    bias = torch.from_numpy(some_bias(rng, 128)).to(dev())
    a = call(x, 8, bias, "sigmoid", 8, 4, 2, renorm=True)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        b = call(x, 8, bias, "sigmoid", 8, 4, 2, renorm=True)
    side.synchronize()
    assert all(torch.equal(a[n], b[n]) for n in a)


def test_binding_refuses():
    x = torch.zeros(8, 16, device=dev())
    call(x, 2, groups=4, opened=2, best=2)
    for kw in (dict(score="tanh"), dict(bias=torch.zeros(15, device=dev())), dict(bias=torch.zeros(16)),
               dict(bias=torch.zeros(16, device=dev()).double())):
        with pytest.raises(ValueError):
            call(x, 2, **kw)
    for kw in (dict(groups=3), dict(groups=0), dict(groups=4, opened=5), dict(groups=4, opened=0), dict(groups=16, best=2),
               dict(groups=4, opened=1, best=3), dict(groups=8, opened=1, k=3)):
        k = kw.pop("k", 2)
        with pytest.raises(fp8g.Fp8GemmError):
            call(x, k, **kw)


def test_more_tokens_than_a_launch_holds():
    """64 tokens a workgroup of 1024 threads: from 2^28 tokens on more than the 2^32 threads that a
    launch may have. Two experts, a bias that favours the second."""
    T, E = (1 << 28) + 12345, 2
    g = torch.Generator(dev()).manual_seed(1)
    x = torch.randint(-8, 9, (T, E), device=dev(), generator=g, dtype=torch.int8).to(torch.bfloat16)
    i, f = torch.int32, torch.float32
    new = lambda shape, t: torch.full(shape, 77, dtype=t, device=dev())  # noqa: E731
    out = dict(expert_ids=new((T, 1), i), weights=new((T, 1), f), counts=new((E,), i), routed=new((1,), i),
               prob_sum=new((E,), f), loss=new((1,), f), group_offsets=new((E + 1,), i), slots=new((T, 1), i))
    ws = torch.full((fp8g.moe_route_workspace_size(T, E),), 0x5A, dtype=torch.uint8, device=dev())
    bias = torch.tensor([0.0, 1e-5], device=dev())
    fp8g.moe_route_scored(x, 1, *out.values(), ws, bias=bias)
    # (scores of whole numbers up to 8 in size are alike or differ by 5.7e-4 and more)
    second = x[:, 1] >= x[:, 0]
    ids = out["expert_ids"][:, 0]
    assert torch.equal(ids == 1, second) and bool(((ids == 0) | (ids == 1)).all())
    n1 = int(second.sum())
    assert out["counts"].tolist() == [T - n1, n1] and out["routed"].item() == T
    ends = [0, (T - n1 + 127) // 128 * 128]
    rank = torch.cumsum(second, 0)
    at = torch.arange(T, device=dev())
    assert torch.equal(out["slots"][:, 0].long(), torch.where(second, ends[1] + rank - 1, at - rank))
    del rank, at
    top = torch.sigmoid(torch.where(second, x[:, 1], x[:, 0]).float())
    # (two exponentials of a few ulp and the quotients)
    assert bool(((out["weights"][:, 0] - top).abs() <= 16 * 2.0 ** -24 * top).all())


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("E,groups,k", [(16, 1, 1), (16, 1, 4), (64, 1, 6), (160, 1, 8), (256, 8, 8), (600, 1, 16)])
def test_one_near_pair_a_row(E, groups, k, score):
    """In each row two neighbours of the order, the k-th and the next in half of them, whose values differ
    by less than fp32's rounding of them, nothing else near: put in order as in 64 bits."""
    rng = np.random.default_rng(E + k)
    T = 400
    bias = some_bias(rng, E)
    x = (rng.standard_normal((T, E)) * 1.5 - 1).astype(np.float32)
    crossed = 0
    for t in range(T):
        j = k - 1 if t % 2 else int(rng.integers(0, k))
        for _ in range(12):                                # (softmax: what is moved moves the sum)
            row = x[t:t + 1].astype(np.float64)
            v = ref.scores(row, score)[0] + bias
            order = np.lexsort((np.arange(E), -v))
            p, q = order[j], order[j + 1]
            want = v[p] - bias[q]
            if not 1e-12 < want < 1:
                break
            if score == "sigmoid":
                x[t, q] = np.float32(np.log(want / (1 - want)))
                break
            z = np.exp(row[0]).sum() - np.exp(row[0, q])
            x[t, q] = np.float32(np.log(want * z / (1 - want)))
        v = np.sort(ref.scores(x[t:t + 1].astype(np.float64), score)[0] + bias)[::-1]
        crossed += v[j] - v[j + 1] < 2.0 ** -22
    assert crossed > T / 10                                # (softmax of few experts: one that is moved moves the others)
    for renorm in (False, True):
        check(torch.from_numpy(x).to(dev()), k, bias, score, groups, groups, 1, renorm=renorm)


@pytest.mark.parametrize("E,groups,opened,best", [(16, 4, 2, 1), (60, 3, 1, 2), (64, 8, 4, 2), (160, 8, 3, 2), (256, 8, 4, 2),
                                                  (256, 32, 5, 1), (600, 6, 3, 2), (1024, 16, 7, 2)])
def test_one_near_pair_of_groups_a_row(E, groups, opened, best):
    """In each row the last open and the first closed group's values differ by less than fp32's rounding
    of them."""
    rng = np.random.default_rng(E + groups)
    T, size, k = 300, E // groups, min(6, opened * (E // groups))
    bias = some_bias(rng, E)
    x = (rng.standard_normal((T, E)) * 1.5 - 1).astype(np.float32)
    near = 0
    for t in range(T):
        v = (ref.scores(x[t:t + 1].astype(np.float64), "sigmoid")[0] + bias).reshape(groups, size)
        value = np.sort(v, 1)[:, ::-1][:, :best].sum(1)
        order = np.lexsort((np.arange(groups), -value))
        a, b = order[opened - 1], order[opened]
        e = b * size + int(v[b].argmax())
        want = value[a] - (np.sort(v[b])[-2] if best == 2 else 0.0) - bias[e]
        if 1e-12 < want < 1 - 1e-7:
            x[t, e] = np.float32(np.log(want / (1 - want)))
            near += 1
    assert near > T / 2
    check(torch.from_numpy(x).to(dev()), k, bias, "sigmoid", groups, opened, best, renorm=True)


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("E,k", [(16, 4), (64, 6), (160, 8), (256, 8), (512, 8), (1000, 16)])
def test_logits_one_step_apart(E, k, score):
    """Without a bias: two neighbours of the order (three in every other row) one fp32 step apart or alike."""
    rng = np.random.default_rng(E + k)
    T = 300
    x = (rng.standard_normal((T, E)) * 1.5 - 1).astype(np.float32)
    for t in range(T):
        j = int(rng.integers(0, k))
        order = np.argsort(-x[t], kind="stable")
        p, q, r = order[j], order[j + 1], order[j + 2] if j + 2 < E else order[j - 1]
        x[t, q] = np.nextafter(x[t, p], np.float32(np.inf if t % 3 == 0 else -np.inf)) if t % 3 < 2 else x[t, p]
        if t % 2:
            x[t, r] = x[t, q]
    check(torch.from_numpy(x).to(dev()), k, None, score, renorm=True)


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("renorm", [False, True])
def test_gradient_against_differences(score, renorm):
    """Central differences in 64 bits of sum(dw weights) + dl loss, experts and counts held."""
    rng = np.random.default_rng(21)
    T, E, k, scale, coef, dl = 9, 20, 3, 2.5, 50.0, 1.5
    x = logits(rng, T, E)
    o = call(x, k, torch.from_numpy(some_bias(rng, E)).to(dev()), score, 4, 2, 2, None, renorm, scale, coef)
    dw = rng.standard_normal((T, k)).astype(np.float32)
    got = gradient(x, o, torch.from_numpy(dw).to(dev()), torch.full((1,), dl, device=dev()), score=score,
                   renormalise=renorm, scale=scale, loss_coef=coef).double().cpu().numpy()
    ids, counts = o["expert_ids"].cpu().numpy().astype(np.int64), o["counts"].cpu().numpy()
    base = x.double().cpu().numpy()

    def value(x):
        s = ref.scores(x, score)
        w = np.take_along_axis(s, ids, 1)
        w = scale * (w / w.sum(1, keepdims=True) if renorm else w)
        share = (s / s.sum(1, keepdims=True)).sum(0)
        return (dw * w).sum() + dl * coef * (E * counts / (k * T) * share / T).sum()
    h, want = 1e-4, np.zeros((T, E))
    for i in np.ndindex(T, E):
        up, down = base.copy(), base.copy()
        up[i] += h
        down[i] -= h
        want[i] = (value(up) - value(down)) / (2 * h)
    _, size = ref.backward(base, ids, dw.astype(np.float64), dl, counts, T, score, renorm, scale, coef)
    # differences: h^2 / 6 of a third derivative, which is below 8 of these sizes (each is a product of
    # at most three scores' slopes), and 2^-52 of the value over h
    tol = 96 * 2.0 ** -24 * size + h * h * 2 * size.max() + 2.0 ** -52 * abs(value(base)) * 4 / h
    assert (np.abs(got - want) <= tol).all()
