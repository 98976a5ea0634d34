"""The 8-bit weight gradient on the GPU: the transposing quantiser bit for bit
against the oracle, the product within a bound derived from its roundings."""

import numpy as np
import pytest
import torch

import moe_grouped_gemm_quantizer_amd as fp8g
from oracle import train
from oracle.formats import bf16_bits_to_f64
from tests.gpu_util import dev, to_dev, banner

pytestmark = pytest.mark.gpu

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
# bf16's rounding, and the matrix instruction's own sum of 128 products, whose
# error reaches 2^-12 of the sum of their magnitudes (measured on this chip)
BF16, MFMA = 2.0 ** -8, 2.0 ** -12


def data(rows, cols, t, seed):
    g = np.random.default_rng(seed)
    x = g.normal(size=(rows, cols)) * np.exp(g.normal(size=(1, cols)))
    return torch.from_numpy(x).to(TYPES[t]).to(dev())


def quantised(x, fmt):
    rows, cols = x.shape
    nb = -(-rows // 128)
    qt = torch.full((cols, nb * 128), 0x55, dtype=torch.uint8, device=dev())
    st = torch.full((nb, cols), 0x55, dtype=torch.uint8, device=dev())
    fp8g.fp8_quantize_transpose(x, fmt, qt, st)
    return qt, st


def same_codes(x, fmt):
    qt, st = quantised(x, fmt)
    q, s = train.quantize_transpose(x.float().cpu().numpy(), fmt)
    assert np.array_equal(st.cpu().numpy(), s)
    assert np.array_equal(qt.cpu().numpy(), q)


@pytest.mark.parametrize("t", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
@pytest.mark.parametrize("rows,cols", [(1, 16), (127, 112), (128, 128), (129, 144), (300, 400), (1024, 48)])
def test_quantiser_sizes(rows, cols, fmt, t):
    same_codes(data(rows, cols, t, rows + cols), fmt)


@pytest.mark.parametrize("t", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
def test_quantiser_special_values(fmt, t):
    info = torch.finfo(TYPES[t])
    x = data(256, 64, t, 9)
    x[3, 0] = float("nan")
    x[4, 0] = -float("nan")
    x[5, 1] = float("inf")
    x[6, 1] = -float("inf")
    x[:, 2] = float("inf")                       # no finite element
    x[:, 3] = 0.0
    x[::2, 3] = -0.0
    x[:, 4] = info.max
    x[:, 5] = info.smallest_normal * (torch.arange(256, device=dev()) % 3 - 1)
    x[:, 6] *= info.tiny
    x[:, 7] *= info.tiny * info.eps * 4          # subnormals
    x[0, 8] = info.max                           # everything else vanishes
    x[:, 9] = (torch.arange(256, device=dev()) - 128).to(x.dtype)
    x[:, 10] = torch.arange(256, device=dev()).to(x.dtype) / 16      # many exact ties
    x[:, 11] = 448.0
    x[7, 11] = 450.0
    same_codes(x, fmt)


def test_quantiser_strides_and_alignment():
    for t in ("f32", "bf16"):
        big = data(200, 80, t, 3)
        same_codes(big[:, 1:65], "e4m3")         # rows 80 apart, an odd start
        same_codes(big[:, 16:80], "e4m3")
        same_codes(big[5:6, :16], "e5m2")
    x = data(200, 32, "bf16", 4)
    wide = torch.full((32, 400), 9, dtype=torch.uint8, device=dev())
    st = torch.empty(2, 32, dtype=torch.uint8, device=dev())
    fp8g.fp8_quantize_transpose(x, "e4m3", wide[:, 16:272], st)
    assert torch.equal(wide[:, 16:272], quantised(x, "e4m3")[0])
    assert (wide[:, :16] == 9).all() and (wide[:, 272:] == 9).all()


def product(ops, M, N, offsets=None, G=1):
    qa, fa, sa, qb, fb, sb = ops
    d = torch.full((G, M, N), float("nan"), dtype=torch.bfloat16, device=dev())
    off = None if offsets is None else torch.tensor(offsets, dtype=torch.int32, device=dev())
    fp8g.grouped_gemm_fp8_wgrad(qa, fa, sa, qb, fb, sb, d, group_offsets=off)
    return d


def check_product(ops, d, offsets):
    qa, fa, sa, qb, fb, sb = ops
    ref, size = train.wgrad(qa.cpu().numpy(), fa, sa.cpu().numpy(), qb.cpu().numpy(), fb, sb.cpu().numpy(), offsets)
    got = bf16_bits_to_f64(d.view(torch.int16).cpu().numpy().view(np.uint16))
    tol = BF16 * (np.abs(ref) + MFMA * size) + MFMA * size
    off = np.abs(got - ref)
    assert (off <= tol).all(), float((off / np.maximum(tol, 1e-300)).max())


def operands(T, M, N, fa="e4m3", fb="e4m3", t="bf16", seed=0):
    qa, sa = quantised(data(T, M, t, seed) * 1e-3, fa)
    qb, sb = quantised(data(T, N, t, seed + 1), fb)
    return qa, fa, sa, qb, fb, sb


@pytest.mark.parametrize("T,M,N", [(1, 16, 16), (128, 256, 512), (200, 48, 272), (384, 528, 144), (1000, 1040, 2064),
                                   (640, 256, 256), (130, 16, 1024), (2048, 272, 528)])
def test_dense_sizes(T, M, N):
    banner(f"wgrad T={T} M={M} N={N}")
    ops = operands(T, M, N, seed=T)
    check_product(ops, product(ops, M, N), [0, -(-T // 128) * 128])


@pytest.mark.parametrize("fa", ["e4m3", "e5m2"])
@pytest.mark.parametrize("fb", ["e4m3", "e5m2"])
def test_formats(fa, fb):
    ops = operands(500, 144, 320, fa, fb, "f32", seed=5)
    check_product(ops, product(ops, 144, 320), [0, 512])


def test_a_sum_of_small_integers_is_exact():
    # (integers to 8 are e4m3 codes, sums of 128 products below 2^13: nothing rounds but the end)
    g = np.random.default_rng(1)
    a, b = g.integers(-8, 9, size=(256, 272)).astype(np.float32), g.integers(-8, 9, size=(256, 288)).astype(np.float32)
    a *= 2.0 ** g.integers(-30, 30, size=(1, 272))
    b *= 2.0 ** g.integers(-30, 30, size=(1, 288))
    qa, sa = quantised(to_dev(a), "e4m3")
    qb, sb = quantised(to_dev(b), "e4m3")
    d = product((qa, "e4m3", sa, qb, "e4m3", sb), 272, 288)
    want = torch.from_numpy((a.astype(np.float64).T @ b.astype(np.float64)).astype(np.float32)).to(torch.bfloat16)
    assert torch.equal(d[0].cpu(), want)


@pytest.mark.parametrize("counts,M,N", [([0, 130, 0, 1, 257, 128, 0], 272, 400), ([5], 64, 64), ([0, 0], 32, 48),
                                        ([1000, 3, 40, 700], 528, 784), ([1] * 40, 64, 80)])
def test_experts(counts, M, N):
    ends = np.concatenate([[0], np.cumsum([-(-c // 128) * 128 for c in counts])]).astype(int)
    T = int(ends[-1])
    if T == 0:
        e = torch.empty(0, dtype=torch.uint8, device=dev())
        d = product((e.view(M, 0), "e4m3", e.view(0, M), e.view(N, 0), "e4m3", e.view(0, N)), M, N, ends, len(counts))
        assert (d == 0).all()
        return
    ops = operands(T, M, N, seed=len(counts))
    d = product(ops, M, N, ends, len(counts))
    check_product(ops, d, ends)
    for g, c in enumerate(counts):
        if c == 0:
            assert (d[g].view(torch.int16) == 0).all()


def test_rows_past_the_last_expert_and_offsets_outside_their_contract():
    ops = operands(512, 48, 64, seed=2)
    check_product(ops, product(ops, 48, 64, [0, 128, 256], 2), [0, 128, 256])
    # clamped into [0, T] and rounded down to 128; a decreasing pair is an empty expert
    d = product(ops, 48, 64, [-500, 200, 100, 1 << 30], 3)
    ref = [(0, 128), (128, 0), (0, 512)]
    for g, (lo, hi) in enumerate(ref):
        if hi <= lo:
            assert (d[g] == 0).all()
        else:
            one = product(ops, 48, 64, [lo, hi], 1)
            assert torch.equal(one[0].view(torch.int16), d[g].view(torch.int16))


def test_nan_and_infinity_reach_their_rows_only():
    x = data(256, 64, "f32", 1)
    x[200, 7] = float("nan")
    y = data(256, 96, "f32", 2)
    y[3, 9] = float("inf")
    qa, sa = quantised(x, "e4m3")
    qb, sb = quantised(y, "e5m2")
    d = product((qa, "e4m3", sa, qb, "e5m2", sb), 64, 96)[0].float()
    bad = torch.zeros(64, 96, dtype=torch.bool, device=dev())
    bad[7, :] = True
    bad[:, 9] = True
    assert (torch.isfinite(d) == ~bad).all()
    assert torch.isnan(d[7]).all()


def test_strided_operands_and_the_same_bits_again():
    T, M, N = 300, 80, 96
    ops = operands(T, M, N, seed=8)
    d = product(ops, M, N)
    wa = torch.full((M, 1024), 0x7F, dtype=torch.uint8, device=dev())
    wb = torch.full((N, 640), 0x7F, dtype=torch.uint8, device=dev())
    wa[:, 128:512] = ops[0]
    wb[:, 16:400] = ops[3]
    e = product((wa[:, 128:512], "e4m3", ops[2], wb[:, 16:400], "e4m3", ops[5]), M, N)
    assert torch.equal(d.view(torch.int16), e.view(torch.int16))


def test_on_another_stream_and_in_a_graph():
    x, y = data(400, 144, "bf16", 1), data(400, 272, "bf16", 2)
    qa, sa = quantised(x, "e5m2")
    qb, sb = quantised(y, "e4m3")
    off = torch.tensor([0, 256, 256, 512], dtype=torch.int32, device=dev())
    d = torch.empty(3, 144, 272, dtype=torch.bfloat16, device=dev())

    def step():
        fp8g.fp8_quantize_transpose(x, "e5m2", qa, sa)
        fp8g.fp8_quantize_transpose(y, "e4m3", qb, sb)
        fp8g.grouped_gemm_fp8_wgrad(qa, "e5m2", sa, qb, "e4m3", sb, d, group_offsets=off)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(4):
        x.copy_(data(400, 144, "bf16", 30 + i))
        step()
        want = d.clone()
        check_product((qa, "e5m2", sa, qb, "e4m3", sb), d, [0, 256, 256, 512])
        d.fill_(7)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(want.view(torch.int16), d.view(torch.int16)), i


def test_gradient_of_a_product_against_differences():
    """With inputs that 8 bits hold exactly, D is the gradient of
    sum(dy * (x W^T)) with respect to W: differences of that sum say the same."""
    g = np.random.default_rng(0)
    x, dy = g.integers(-4, 5, size=(128, 32)).astype(np.float32), g.integers(-4, 5, size=(128, 16)).astype(np.float32)
    qa, sa = quantised(to_dev(dy), "e4m3")
    qb, sb = quantised(to_dev(x), "e4m3")
    d = product((qa, "e4m3", sa, qb, "e4m3", sb), 16, 32)[0].double().cpu().numpy()
    w = g.normal(size=(16, 32))
    f = lambda v: float((dy * (x @ v.T)).sum())  # noqa: E731
    for m in range(0, 16, 5):
        for n in range(0, 32, 7):
            up, dn = w.copy(), w.copy()
            up[m, n] += 0.5
            dn[m, n] -= 0.5
            # (the sum is linear; bf16's rounding of an integer up to 2048)
            assert abs((f(up) - f(dn)) - d[m, n]) <= BF16 * abs(d[m, n]) + 1e-9


@pytest.mark.parametrize("counts,M,N", [([300], 4096, 2304), ([130, 0, 500, 128, 0], 1040, 2064),
                                        ([128] * 5 + [0, 1000], 1296, 1808), ([1] * 33, 512, 784)])
def test_enough_tiles_for_the_large_kernel(counts, M, N):
    ends = np.concatenate([[0], np.cumsum([-(-c // 128) * 128 for c in counts])]).astype(int)
    banner(f"wgrad large counts={counts} M={M} N={N}")
    ops = operands(int(ends[-1]), M, N, "e5m2", "e4m3", seed=len(counts))
    d = product(ops, M, N, None if len(counts) == 1 else ends, len(counts))
    check_product(ops, d, ends)
