"""Products in 8-bit integers on the GPU, bit for bit against NumPy."""

import numpy as np
import pytest
import torch

import moe_grouped_gemm_quantizer_amd as fp8g
from tests import int8_ref as ref
from tests.gpu_util import dev, to_dev, to_host

pytestmark = pytest.mark.gpu

KINDS = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
STALE = 0x7A7B


def codes(rng, *shape):
    """Codes of all sizes, the largest and -128 among them."""
    c = rng.integers(-128, 128, shape, dtype=np.int64)
    return np.where(rng.random(shape) < 0.5, c // 8, c).astype(np.int8)


def scales(rng, *shape):
    return np.exp(rng.uniform(-9, -3, shape)).astype(np.float32)


def run_quantise(x, strided=False, shift=0):
    """x: a CPU tensor [rows][cols]. -> codes, scales of the GPU, and the exact fp32 values."""
    rows, cols = x.shape
    pad = 16 if strided else 0
    buf = torch.full((rows, cols + pad + shift), 7.0, dtype=x.dtype, device=dev())
    view = buf[:, shift:shift + cols]
    view.copy_(x)
    qbuf = torch.full((rows, cols + pad), 99, dtype=torch.int8, device=dev())
    s = torch.full((rows,), 5.0, device=dev())
    fp8g.int8_quantize(view, qbuf[:, :cols], s)
    q = to_host(qbuf)
    assert (q[:, cols:] == 99).all()
    return q[:, :cols], to_host(s), x.float().numpy()


@pytest.mark.parametrize("kind", list(KINDS))
@pytest.mark.parametrize("rows,cols", [(1, 16), (3, 32), (5, 512), (7, 528), (2, 1040), (9, 2048), (4, 2064),
                                       (3, 4096), (2, 8208), (2, 16384), (3, 16400), (2, 33024), (301, 208)])
@pytest.mark.parametrize("strided", [False, True])
def test_quantise(kind, rows, cols, strided):
    rng = np.random.default_rng(rows * 1000 + cols)
    x = rng.standard_normal((rows, cols)) * np.exp(rng.uniform(-8, 8, (rows, 1)))
    q, s, xf = run_quantise(torch.from_numpy(x).to(KINDS[kind]), strided, shift=3 if strided else 0)
    q0, s0 = ref.quantise(xf)
    assert np.array_equal(s.view(np.uint32), s0.view(np.uint32))
    assert np.array_equal(q, q0)


def test_quantise_halves_and_range():
    """Values that lie half way between codes (ties to even), the largest value itself,
    rows far up and down in fp32's range, zeros, and rows that count as zero."""
    rows = [np.arange(-127, 129, dtype=np.float64) * 0.5,      # amax 64: inv 127/64 exactly
            np.r_[np.full(128, 127.0), np.arange(-64, 64) + 0.5], np.zeros(256), np.full(256, -0.0),
            np.full(256, 3.4e38), np.linspace(-3.4e38, 3.4e38, 256), np.full(256, 2.0 ** -120),
            np.linspace(-(2.0 ** -119), 2.0 ** -119, 256), np.full(256, 2.0 ** -121), np.full(256, 2.0 ** -149)]
    x = torch.from_numpy(np.stack(rows)).float()
    q, s, xf = run_quantise(x)
    q0, s0 = ref.quantise(xf)
    assert np.array_equal(s.view(np.uint32), s0.view(np.uint32)) and np.array_equal(q, q0)
    assert (q[1, :128] == 127).all() and s[8] == 0 and s[9] == 0 and s[6] > 0


@pytest.mark.parametrize("kind", list(KINDS))
@pytest.mark.parametrize("cols", [64, 3008, 17008])
def test_quantise_nonfinite(kind, cols):
    x = torch.randn(6, cols, generator=torch.Generator().manual_seed(1)).to(KINDS[kind])
    x[1, 5], x[2, cols - 1], x[4, 0] = float("nan"), float("inf"), float("-inf")
    q, s, xf = run_quantise(x)
    assert np.isnan(s[[1, 2, 4]]).all() and (q[[1, 2, 4]] == 0).all()
    q0, s0 = ref.quantise(xf[[0, 3, 5]])
    assert np.array_equal(q[[0, 3, 5]], q0) and np.array_equal(s[[0, 3, 5]], s0)


def run_dense(rng, M, N, K):
    a, sa, b, sb = codes(rng, M, K), scales(rng, M), codes(rng, N, K), scales(rng, N)
    d = torch.full((M, N), STALE, dtype=torch.int16, device=dev())
    fp8g.gemm_int8(to_dev(a), to_dev(sa), to_dev(b), to_dev(sb), d)
    return to_host(d).view(np.uint16), ref.product(a, sa, b, sb)


@pytest.mark.parametrize("M", [1, 2, 15, 16, 17, 31, 32, 33, 64, 65, 127, 128, 129, 200, 256, 257, 300, 513])
@pytest.mark.parametrize("N,K", [(16, 16), (48, 1040), (272, 528)])
def test_dense_rows(M, N, K):
    got, want = run_dense(np.random.default_rng(M + N + K), M, N, K)
    assert np.array_equal(got, want)


@pytest.mark.parametrize("K", [16, 32, 48, 64, 80, 112, 128, 144, 240, 256, 272, 384, 400, 640, 2048, 2064, 7168])
@pytest.mark.parametrize("M,N", [(5, 64), (130, 144), (384, 272)])
def test_dense_depth(K, M, N):
    got, want = run_dense(np.random.default_rng(K * M), M, N, K)
    assert np.array_equal(got, want)


@pytest.mark.parametrize("N", [16, 32, 112, 128, 144, 240, 256, 272, 496, 512, 1040])
@pytest.mark.parametrize("M,K", [(3, 144), (100, 256), (260, 208)])
def test_dense_columns(N, M, K):
    got, want = run_dense(np.random.default_rng(N * M), M, N, K)
    assert np.array_equal(got, want)


@pytest.mark.parametrize("M,N,K", [
    # (the kernels from few rows to many, each with K a multiple of 128 and not)
    (9, 784, 640), (16, 4096, 528), (30, 2144, 384), (100, 2768, 240), (180, 960, 2480), (306, 2768, 384),
    (777, 2064, 1040), (1024, 2048, 256), (1128, 7184, 144), (2048, 4096, 128), (2048, 4096, 1024), (3001, 3600, 256),
    (4096, 4096, 256), (2305, 6672, 272), (2000, 4096, 272)])
def test_dense_kernels(M, N, K):
    got, want = run_dense(np.random.default_rng(M + K), M, N, K)
    assert np.array_equal(got, want)


@pytest.mark.parametrize("M,N,K", [(4, 16, 131056), (40, 32, 131056), (300, 272, 131056)])
def test_largest_sums(M, N, K):
    """Every code -128, as deep as the call allows: the sum is 2^31 - 2^18."""
    a = np.full((M, K), -128, np.int8)
    b = np.full((N, K), -128, np.int8)
    b[1] = 127
    one = np.ones
    d = torch.empty(M, N, dtype=torch.bfloat16, device=dev())
    fp8g.gemm_int8(to_dev(a), to_dev(one(M, np.float32)), to_dev(b), to_dev(one(N, np.float32)), d)
    got = to_host(d.float())
    want = torch.tensor([K * 16384.0, -K * 128 * 127.0]).bfloat16().float().numpy()
    assert (np.delete(got, 1, 1) == want[0]).all() and (got[:, 1] == want[1]).all()


def test_scales_that_are_not_finite():
    rng = np.random.default_rng(5)
    a, sa, b, sb = codes(rng, 40, 64), scales(rng, 40), codes(rng, 48, 64), scales(rng, 48)
    a[3] = 0
    sa[3], sa[7], sb[5] = np.nan, np.inf, 0.0
    d = torch.empty(40, 48, dtype=torch.bfloat16, device=dev())
    fp8g.gemm_int8(to_dev(a), to_dev(sa), to_dev(b), to_dev(sb), d)
    got = to_host(d.float())
    assert np.isnan(got[3]).all() and not np.isfinite(got[7]).any()
    rows = np.r_[0:3, 4:7, 8:40]
    want = torch.from_numpy((ref.product(a[rows], sa[rows], b, sb)).view(np.int16)).view(torch.bfloat16).float().numpy()
    assert np.array_equal(got[rows], want) and (got[rows, 5] == 0).all()


def run_contiguous(rng, counts, N, K, align=128, lead=0, tail=0):
    """Experts' rows padded to `align`, `lead` rows before the first and `tail` behind the last."""
    G = len(counts)
    offsets = [lead]
    for n in counts:
        offsets.append(offsets[-1] + -(-n // align) * align)
    M = offsets[-1] + tail
    a, sa, b, sb = codes(rng, M, K), scales(rng, M), codes(rng, G, N, K), scales(rng, G, N)
    d = torch.full((M, N), STALE, dtype=torch.int16, device=dev())
    off = torch.tensor(offsets, dtype=torch.int32, device=dev())
    fp8g.grouped_gemm_int8_contiguous(to_dev(a), to_dev(sa), to_dev(b), to_dev(sb), d, off)
    return to_host(d).view(np.uint16), ref.contiguous(a, sa, b, sb, offsets, np.full((M, N), STALE, np.uint16))


@pytest.mark.parametrize("counts,N,K", [
    ((1,), 16, 16), ((128, 128), 256, 128), ((0, 300, 1, 0, 129, 40), 272, 208), ((700, 5), 512, 256),
    ((0, 0, 3), 64, 64), ((256, 0, 512, 255, 257, 1), 528, 144)])
@pytest.mark.parametrize("align,lead,tail", [(128, 0, 0), (128, 128, 256), (1, 0, 0), (1, 5, 7), (16, 0, 3)])
def test_contiguous(counts, N, K, align, lead, tail):
    got, want = run_contiguous(np.random.default_rng(sum(counts) + K), counts, N, K, align, lead, tail)
    assert np.array_equal(got, want)


def test_contiguous_many_experts():
    rng = np.random.default_rng(3)
    counts = rng.integers(0, 4, 1024)
    counts[[0, 500, 1023]] = 0, 140, 2
    got, want = run_contiguous(rng, tuple(counts), 32, 48, align=1)
    assert np.array_equal(got, want)


def test_contiguous_without_rows():
    got, want = run_contiguous(np.random.default_rng(1), (0, 0), 64, 64, tail=9)
    assert np.array_equal(got, want) and (got == STALE).all()


@pytest.mark.parametrize("counts,max_m,N,K", [
    ((3, 0, 64), 64, 64, 64), ((0, 0), 16, 32, 32), ((1, 2, 3, 4, 5), 5, 272, 144), ((129, 256, 0, 7), 256, 528, 208),
    ((300, 17, 512, 260), 512, 256, 256), ((40, -5, 33, 1000), 40, 80, 400)])
@pytest.mark.parametrize("hint", [0, 8, 400])
def test_masked(counts, max_m, N, K, hint):
    rng = np.random.default_rng(max_m + K)
    G = len(counts)
    a, sa = codes(rng, G, max_m, K), scales(rng, G, max_m)
    b, sb = codes(rng, G, N, K), scales(rng, G, N)
    d = torch.full((G, max_m, N), STALE, dtype=torch.int16, device=dev())
    m = torch.tensor(counts, dtype=torch.int32, device=dev())
    fp8g.grouped_gemm_int8_masked(to_dev(a), to_dev(sa), to_dev(b), to_dev(sb), d, m, expected_m=hint)
    want = ref.masked(a, sa, b, sb, counts, np.full((G, max_m, N), STALE, np.uint16))
    assert np.array_equal(to_host(d).view(np.uint16), want)


def test_offsets_that_break_the_rules_stay_inside():
    """Offsets outside [0, M_total] and below earlier ones: clamped, to the earlier ones too."""
    rng = np.random.default_rng(8)
    M, G, N, K = 200, 4, 48, 64
    a, sa, b, sb = codes(rng, M, K), scales(rng, M), codes(rng, G, N, K), scales(rng, G, N)
    guard = torch.full((M + 64, N), STALE, dtype=torch.int16, device=dev())
    off = torch.tensor([-50, 30, 20, 2_000_000_000, 100], dtype=torch.int32, device=dev())
    fp8g.grouped_gemm_int8_contiguous(to_dev(a), to_dev(sa), to_dev(b), to_dev(sb), guard[32:32 + M], off)
    got = to_host(guard).view(np.uint16)
    want = ref.contiguous(a, sa, b, sb, [0, 30, 30, 200, 200], np.full((M, N), STALE, np.uint16))
    assert np.array_equal(got[32:32 + M], want) and (got[:32] == STALE).all() and (got[32 + M:] == STALE).all()


def test_layer_from_activations():
    """The quantiser and the product together: within the codes' half steps of the
    unquantised product."""
    rng = np.random.default_rng(11)
    M, N, K = 70, 96, 272
    x, w = rng.standard_normal((M, K)), rng.standard_normal((N, K))
    qx, sx, xf = run_quantise(torch.from_numpy(x).bfloat16())
    qw, sw, wf = run_quantise(torch.from_numpy(w).float())
    d = torch.empty(M, N, dtype=torch.bfloat16, device=dev())
    fp8g.gemm_int8(to_dev(qx), to_dev(sx), to_dev(qw), to_dev(sw), d)
    got = to_host(d.double())
    want = xf.astype(np.float64) @ wf.astype(np.float64).T
    # each code is off by at most half a step and 2^-16 (the product x inv), so a product of
    # values off by sx/2 and sw/2; then bf16's half step and fp32's three
    h = 0.5 + 2.0 ** -16
    ax, aw = np.abs(xf).astype(np.float64), np.abs(wf).astype(np.float64)
    off = h * sx[:, None] * aw.sum(1) + h * sw[None, :] * ax.sum(1)[:, None] + K * h * h * sx[:, None] * sw[None, :]
    assert (np.abs(got - want) <= off + (2.0 ** -8 + 4 * 2.0 ** -24) * (np.abs(want) + off)).all()


def test_captured_and_replayed():
    """A graph of quantiser and products, replayed with new inputs in the same buffers."""
    M, N, K = 300, 272, 400
    gen = torch.Generator(device=dev()).manual_seed(2)
    x = torch.randn(M, K, device=dev(), generator=gen)
    b = torch.randint(-127, 128, (2, N, K), dtype=torch.int8, device=dev(), generator=gen)
    sb = torch.rand(2, N, device=dev(), generator=gen)
    q, sa = torch.empty(M, K, dtype=torch.int8, device=dev()), torch.empty(M, device=dev())
    off = torch.tensor([0, 130, M], dtype=torch.int32, device=dev())
    d, e = (torch.empty(M, N, dtype=torch.bfloat16, device=dev()) for _ in range(2))

    def step(one, two):
        fp8g.int8_quantize(x, q, sa)
        fp8g.gemm_int8(q, sa, b[0], sb[0], one)
        fp8g.grouped_gemm_int8_contiguous(q, sa, b, sb, two, off)
    step(d, e)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(d, e)
    d2, e2 = torch.empty_like(d), torch.empty_like(e)
    for i in range(4):
        x.normal_(generator=gen)
        graph.replay()
        torch.cuda.synchronize()
        step(d2, e2)
        torch.cuda.synchronize()
        assert torch.equal(d, d2) and torch.equal(e, e2), i


def test_another_stream():
    gen = torch.Generator(device=dev()).manual_seed(4)
    a = torch.randint(-127, 128, (65, 256), dtype=torch.int8, device=dev(), generator=gen)
    b = torch.randint(-127, 128, (80, 256), dtype=torch.int8, device=dev(), generator=gen)
    sa, sb = torch.rand(65, device=dev(), generator=gen), torch.rand(80, device=dev(), generator=gen)
    d, e, f = (torch.zeros(65, 80, dtype=torch.bfloat16, device=dev()) for _ in range(3))
    fp8g.gemm_int8(a, sa, b, sb, d)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        fp8g.gemm_int8(a, sa, b, sb, e)
    fp8g.gemm_int8(a, sa, b, sb, f, stream=side)
    side.synchronize()
    assert torch.equal(d, e) and torch.equal(d, f)


def test_binding_refuses():
    i8 = dict(dtype=torch.int8, device=dev())
    a, b = torch.zeros(4, 32, **i8), torch.zeros(16, 32, **i8)
    sa, sb = torch.zeros(4, device=dev()), torch.zeros(16, device=dev())
    d = torch.zeros(4, 16, dtype=torch.bfloat16, device=dev())
    fp8g.gemm_int8(a, sa, b, sb, d)
    for bad in [(a.view(torch.uint8), sa, b, sb, d), (a, sa.double(), b, sb, d), (a, sa, b[:, :16], sb, d),
                (a, sa, b, sb[:8], d), (a, sa, b, sb, d.float()), (a.cpu(), sa, b, sb, d), (a, sa[:3], b, sb, d),
                (a.view(2, 2, 32), sa, b, sb, d)]:
        with pytest.raises(ValueError):
            fp8g.gemm_int8(*bad)
    x = torch.zeros(4, 32, device=dev())
    for bad in [(x.double(), a, sa), (x, a.view(torch.uint8), sa), (x[:, :16], a, sa), (x, a, sa[:2]),
                (x.t(), a, sa), (x, a, sa.int())]:
        with pytest.raises(ValueError):
            fp8g.int8_quantize(*bad)
    with pytest.raises(fp8g.Fp8GemmError):
        fp8g.int8_quantize(x[:, :24], torch.zeros(4, 24, **i8), sa)


@pytest.mark.parametrize("M,N,K", [(4200, 4368, 128), (8200, 3856, 128), (3200, 4096, 256), (12544, 2704, 128),
                                   (4096, 6160, 384), (6400, 5904, 128)])
def test_dense_last_round(M, N, K):
    """More tiles than CUs: last rounds that are empty, of a few tiles, of half of the CUs, of most."""
    got, want = run_dense(np.random.default_rng(M + N), M, N, K)
    assert np.array_equal(got, want)


@pytest.mark.parametrize("counts,N,K", [
    ((1500, 0, 900, 1, 700, 1300), 4368, 128), ((300, 290, 310, 257, 0, 512, 600, 256), 7184, 128),
    ((600, 700), 1040, 256), ((4096, 4096), 2048, 128)])
def test_contiguous_last_round(counts, N, K):
    got, want = run_contiguous(np.random.default_rng(N), counts, N, K, align=1, lead=3, tail=2)
    assert np.array_equal(got, want)


@pytest.mark.parametrize("counts,max_m,N,K", [
    ((200, 130, 256, 0, 180, 7, 255, 140, 256, 300), 256, 7184, 128), ((512, 300, 0, 512), 512, 4368, 256)])
def test_masked_last_round(counts, max_m, N, K):
    rng = np.random.default_rng(max_m + N)
    G = len(counts)
    a, sa = codes(rng, G, max_m, K), scales(rng, G, max_m)
    b, sb = codes(rng, G, N, K), scales(rng, G, N)
    d = torch.full((G, max_m, N), STALE, dtype=torch.int16, device=dev())
    m = torch.tensor(counts, dtype=torch.int32, device=dev())
    fp8g.grouped_gemm_int8_masked(to_dev(a), to_dev(sa), to_dev(b), to_dev(sb), d, m)
    want = ref.masked(a, sa, b, sb, counts, np.full((G, max_m, N), STALE, np.uint16))
    assert np.array_equal(to_host(d).view(np.uint16), want)


@pytest.mark.parametrize("K", [128, 144])
def test_offsets_in_any_order_stay_inside(K):
    """More experts than a wave has lanes, offsets at random: as their running maximum says."""
    rng = np.random.default_rng(K)
    M, G, N = 700, 150, 272
    a, sa, b, sb = codes(rng, M, K), scales(rng, M), codes(rng, G, N, K), scales(rng, G, N)
    off = rng.integers(-2 ** 31, 2 ** 31, G + 1)
    off[::3] = rng.integers(0, M + 1, len(off[::3]))
    off[:100] = np.minimum(off[:100], rng.integers(0, 300, 100))
    d = torch.full((M, N), STALE, dtype=torch.int16, device=dev())
    fp8g.grouped_gemm_int8_contiguous(to_dev(a), to_dev(sa), to_dev(b), to_dev(sb), d,
                                      torch.from_numpy(off.astype(np.int32)).to(dev()))
    starts = np.maximum.accumulate(np.clip(off, 0, M))
    want = ref.contiguous(a, sa, b, sb, starts, np.full((M, N), STALE, np.uint16))
    assert np.array_equal(to_host(d).view(np.uint16), want) and len(np.unique(starts)) > 4


@pytest.mark.parametrize("K", [65536, 65552])
def test_offsets_past_32_bits(K):
    """More than 2^32 elements of x, codes and operands: quantised and multiplied rows at both ends."""
    M, N = 66000, 144
    x = torch.zeros(M, K, dtype=torch.bfloat16, device=dev())
    rows = [0, 1, 32767, 32768, 65535, 65536, M - 2, M - 1]
    gen = torch.Generator(dev()).manual_seed(1)
    x[rows] = torch.randn(len(rows), K, device=dev(), generator=gen).to(torch.bfloat16)
    q = torch.full((M, K), 3, dtype=torch.int8, device=dev())
    s = torch.full((M,), -1.0, device=dev())
    fp8g.int8_quantize(x, q, s)
    qr, sr = ref.quantise(to_host(x[rows].float()))
    assert np.array_equal(to_host(q[rows]), qr) and np.array_equal(to_host(s[rows]), sr)
    assert int(s.count_nonzero()) == len(rows) and int(torch.count_nonzero(q[rows[3] + 1:rows[4]])) == 0
    del x
    rng = np.random.default_rng(K)
    b, sb = codes(rng, N, K), scales(rng, N)
    d = torch.full((M, N), STALE, dtype=torch.int16, device=dev())
    fp8g.gemm_int8(q, s, to_dev(b), to_dev(sb), d)
    want = ref.product(qr, sr, b, sb)
    assert np.array_equal(to_host(d[rows]).view(np.uint16), want)
    assert int((d[rows[3] + 1:rows[4]] & 0x7FFF).count_nonzero()) == 0
    off = torch.tensor([0, 32769, 65536, M], dtype=torch.int32, device=dev())
    three = np.stack([b[::-1], b, b[:, ::-1]])
    d2 = torch.full((M, N), STALE, dtype=torch.int16, device=dev())
    fp8g.grouped_gemm_int8_contiguous(q, s, to_dev(three.copy()), to_dev(np.stack([sb, sb, sb])), d2, off)
    for r, row in enumerate(rows):
        g = (row >= 32769) + (row >= 65536)
        assert np.array_equal(to_host(d2[row]).view(np.uint16), ref.product(qr[r:r + 1], sr[r:r + 1], three[g], sb)[0])


def test_captured_and_replayed_on_two_streams():
    """Quantiser and product captured twice, replayed at once on two streams with new inputs: no
    shared memory of the library's own."""
    M, N, K = 300, 528, 512
    gen = torch.Generator(dev()).manual_seed(3)
    w = torch.randn(N, K, device=dev(), generator=gen)
    qw, sw = torch.empty(N, K, dtype=torch.int8, device=dev()), torch.empty(N, device=dev())
    fp8g.int8_quantize(w, qw, sw)
    torch.cuda.synchronize()
    work = []
    for _ in range(2):
        x = torch.randn(M, K, device=dev(), generator=gen)
        q, s = torch.empty(M, K, dtype=torch.int8, device=dev()), torch.empty(M, device=dev())
        d = torch.empty(M, N, dtype=torch.bfloat16, device=dev())
        side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            fp8g.int8_quantize(x, q, s)
            fp8g.gemm_int8(q, s, qw, sw, d)
        work.append((x, q, s, d, side, graph))
    for t in range(4):
        for x, *_ in work:
            x.normal_(generator=gen)
        torch.cuda.synchronize()
        for *_, side, graph in work:
            with torch.cuda.stream(side):
                graph.replay()
        torch.cuda.synchronize()
        for x, q, s, d, *_ in work:
            q0, s0 = ref.quantise(to_host(x))
            assert np.array_equal(to_host(q), q0)
            want = ref.product(q0, s0, to_host(qw), to_host(sw))
            assert np.array_equal(to_host(d.view(torch.int16)).view(np.uint16), want)


@pytest.mark.parametrize("M,N,K", [(1013, 752, 256), (334, 2896, 896), (371, 2128, 2352), (612, 592, 4352), (145, 560, 3104),
                                   (45, 5712, 2704), (64, 16400, 144), (700, 4096, 400), (894, 6608, 768),
                                   (149, 19728, 640), (1500, 8208, 208)])
def test_dense_kernels_between(M, N, K):
    """Sizes where the choice among the kernels is close."""
    got, want = run_dense(np.random.default_rng(M + N), M, N, K)
    assert np.array_equal(got, want)
