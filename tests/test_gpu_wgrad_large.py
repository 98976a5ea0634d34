"""The weight gradient where 256x256 tiles serve it: chains of tiles in one
workgroup, every pair of formats, strides, offsets outside their contract, NaN."""

import numpy as np
import pytest
import torch

import moe_grouped_gemm_quantizer_amd as fp8g
from tests.gpu_util import dev, banner
from tests.test_gpu_wgrad import BF16, MFMA, check_product, operands, product, quantised

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("G,M,N", [(200, 16, 32), (3, 2064, 1552)])
def test_no_tokens_and_many_tiles(G, M, N):
    banner(f"wgrad T=0 G={G} M={M} N={N}")
    e = torch.empty(0, dtype=torch.uint8, device=dev())
    off = torch.zeros(G + 1, dtype=torch.int32, device=dev())
    d = torch.full((G, M, N), float("nan"), dtype=torch.bfloat16, device=dev())
    fp8g.grouped_gemm_fp8_wgrad(e.view(M, 0), "e4m3", e.view(0, M), e.view(N, 0), "e4m3", e.view(0, N), d,
                                group_offsets=off)
    assert (d.view(torch.int16) == 0).all()


def ends_of(counts):
    return np.concatenate([[0], np.cumsum([-(-c // 128) * 128 for c in counts])]).astype(int)


def integers(T, width, seed):
    """-4 .. 4 times a power of two for each column: codes of both formats, and
    sums of their products over some hundred tokens round only at the end."""
    g = torch.Generator(dev()).manual_seed(seed)
    x = torch.randint(-4, 5, (T, width), device=dev(), generator=g).float()
    return x * torch.exp2(torch.randint(-20, 21, (1, width), device=dev(), generator=g).float())


def exact(dy, x, ends):
    """D in float64 (exact here), rounded to bf16 once."""
    return torch.stack([(dy[i:j].double().t().contiguous() @ x[i:j].double()).to(torch.float32).to(torch.bfloat16)
                        for i, j in zip(ends, ends[1:])])


@pytest.mark.parametrize("fa", ["e4m3", "e5m2"])
@pytest.mark.parametrize("fb", ["e4m3", "e5m2"])
@pytest.mark.parametrize("counts,M,N", [([300], 3056, 2800), ([130, 0, 500, 128, 0, 77], 1040, 2064)])
def test_formats(counts, M, N, fa, fb):
    banner(f"wgrad formats {fa} x {fb} counts={counts} M={M} N={N}")
    ends = ends_of(counts)
    ops = operands(int(ends[-1]), M, N, fa, fb, seed=M)
    check_product(ops, product(ops, M, N, None if len(counts) == 1 else ends, len(counts)), ends)
    dy, x = integers(int(ends[-1]), M, 1), integers(int(ends[-1]), N, 2)
    d = product((*_q(dy, fa), *_q(x, fb)), M, N, None if len(counts) == 1 else ends, len(counts))
    assert torch.equal(d.view(torch.int16), exact(dy, x, ends).view(torch.int16))


# Tiles that a workgroup takes one after the other (256 of them on this chip, so
# from 257 tiles on): whole tiles of one step; of one and more steps; whole and
# ragged ones in turn (three, five or two of them an expert, so that the place in the expert
# shifts from one round to the next, or does not).
CHAINS = [([128] * 1000, 256, 256), ([128, 256, 1, 640, 128, 128] * 150, 256, 256), ([128] * 300, 528, 256),
          ([128, 300, 128, 0, 513, 1] * 60, 528, 256), ([128, 257] * 90, 272, 1040), ([128, 128, 384] * 120, 272, 512),
          ([2000], 4112, 4112), ([1300, 0, 700], 2576, 4096)]


@pytest.mark.parametrize("which", range(len(CHAINS)))
def test_tiles_one_after_the_other(which):
    counts, M, N = CHAINS[which]
    ends = ends_of(counts)
    T = int(ends[-1])
    banner(f"wgrad chain {which}: {len(counts)} experts T={T} M={M} N={N}")
    dy, x = integers(T, M, which), integers(T, N, 50 + which)
    ops = (*_q(dy, "e5m2"), *_q(x, "e4m3"))
    d = product(ops, M, N, ends, len(counts))
    if max(counts) <= 640:
        # (magnitudes to 16, sums to 640 of them: 14 bits)
        assert torch.equal(d.view(torch.int16), exact(dy, x, ends).view(torch.int16))
    else:
        for g, (i, j) in enumerate(zip(ends, ends[1:])):
            a, b = dy[i:j].double().t().contiguous(), x[i:j].double()
            ref, size = a @ b, a.abs() @ b.abs()
            tol = BF16 * (ref.abs() + MFMA * size) + MFMA * size
            assert ((d[g].double() - ref).abs() <= tol).all(), g
    assert torch.equal(product(ops, M, N, ends, len(counts)).view(torch.int16), d.view(torch.int16))


@pytest.mark.parametrize("counts,M,N", [([128] * 300, 128, 128), ([1, 200, 0, 513] * 60, 64, 112),
                                        ([128] * 700, 16, 48), ([300] * 150, 384, 128)])
def test_many_narrow_experts(counts, M, N):
    """More tiles than CUs, none of which 256x256 would fill: several rounds of
    the small kernel."""
    banner(f"wgrad narrow: {len(counts)} experts M={M} N={N}")
    ends = ends_of(counts)
    T = int(ends[-1])
    dy, x = integers(T, M, 5), integers(T, N, 6)
    d = product((*_q(dy, "e5m2"), *_q(x, "e4m3")), M, N, ends, len(counts))
    assert torch.equal(d.view(torch.int16), exact(dy, x, ends).view(torch.int16))


def _q(x, fmt):
    q, s = quantised(x, fmt)
    return q, fmt, s


def test_offsets_outside_their_contract_and_strided_operands():
    G, M, N, T = 3, 2064, 1552, 640
    dy, x = integers(T, M, 7), integers(T, N, 8)
    qa, fa, sa = _q(dy, "e5m2")
    qb, fb, sb = _q(x, "e4m3")
    # NaN codes around the operands: nothing outside them may be read into a sum
    wa = torch.full((M, 1024), 0x7F, dtype=torch.uint8, device=dev())
    wb = torch.full((N, 688), 0x7F, dtype=torch.uint8, device=dev())
    wa[:, 128:768], wb[:, 16:656] = qa, qb
    d = product((wa[:, 128:768], fa, sa, wb[:, 16:656], fb, sb), M, N, [-500, 200, 100, 1 << 30], G)
    want = exact(dy, x, [0, 128])[0], torch.zeros_like(d[1]), exact(dy, x, [0, 640])[0]
    for g in range(G):
        assert torch.equal(d[g].view(torch.int16), want[g].view(torch.int16)), g


def test_nan_and_infinity_reach_their_rows_only():
    counts, M, N = [200, 128, 300], 1296, 2064
    ends = ends_of(counts)
    T = int(ends[-1])
    dy, x = integers(T, M, 3), integers(T, N, 4)
    clean = exact(dy, x, ends)
    dy[130, 1290] = float("nan")               # expert 0, a ragged tile's row
    x[ends[1] + 5, 700] = float("inf")         # expert 1
    d = product((*_q(dy, "e5m2"), *_q(x, "e5m2")), M, N, ends, 3)
    bad = torch.zeros(3, M, N, dtype=torch.bool, device=dev())
    bad[0, 1290, :] = True
    bad[1, :, 700] = True
    assert torch.isnan(d[0, 1290]).all() and not torch.isfinite(d[1, :, 700]).any()
    assert torch.equal(d[~bad].view(torch.int16), clean[~bad].view(torch.int16))


def test_against_the_oracle_over_many_tokens():
    T, M, N = 8192, 272, 528
    ops = operands(T, M, N, "e5m2", "e4m3", seed=T)
    check_product(ops, product(ops, M, N), [0, T])
