"""Host side of the AdamW step's list: memory ranges that overlap."""

import random

import pytest

from moe_grouped_gemm_quantizer_amd._lib import _overlapping


def overlapping(written, read):
    return _overlapping([a for a, _ in written], [b for _, b in written], read)


@pytest.mark.parametrize("written,read,want", [
    ([], [], False), ([], [(0, 8)], False), ([(0, 8)], [], False),
    ([(0, 8), (8, 16)], [(16, 24)], False), ([(8, 16), (0, 8)], [(16, 24), (16, 20)], False),
    ([(0, 8), (0, 8)], [], True), ([(0, 8), (7, 9)], [], True), ([(0, 100), (40, 44)], [], True),
    ([(0, 8)], [(0, 8)], True), ([(0, 8)], [(7, 20)], True), ([(4, 8)], [(0, 5)], True), ([(4, 8)], [(0, 4)], False),
    ([(0, 100)], [(40, 44)], True), ([(40, 44)], [(0, 100)], True), ([(0, 4), (8, 12)], [(4, 8)], False),
    ([(0, 4), (8, 12)], [(4, 9)], True), ([(0, 4), (8, 12)], [(3, 8)], True),
    # (nothing lies in an empty range)
    ([(0, 0), (4, 8), (0, 0)], [(0, 0)], False), ([(0, 0)], [(4, 8)], False)])
def test_overlapping(written, read, want):
    assert overlapping(written, read) == want


def test_overlapping_as_every_pair_says():
    rng = random.Random(0)
    seen = set()
    for _ in range(3000):
        def some(most):
            size = [rng.randint(0, 6) for _ in range(rng.randint(0, most))]
            return [(a, a + k) if k else (0, 0) for a, k in zip((rng.randint(1, 60) for _ in size), size)]
        ranges, read = some(7), some(3)

        def meet(a, b):
            return max(a[0], b[0]) < min(a[1], b[1])
        want = any(meet(a, b) for i, a in enumerate(ranges) for b in ranges[:i] + read)
        seen.add(want)
        assert overlapping(ranges, read) == want
    assert seen == {False, True}
