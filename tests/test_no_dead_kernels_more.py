"""The library holds no kernel of scored routing, the 8-bit integer products or the AdamW step that no
call reaches."""

import os
import re
import shutil
import subprocess

import pytest

from moe_grouped_gemm_quantizer_amd._lib import LIB_PATH

pytestmark = pytest.mark.skipif(not os.path.exists(LIB_PATH) or shutil.which("nm") is None,
                                reason="library or nm missing")


@pytest.fixture(scope="module")
def names():
    return subprocess.run(["nm", "--defined-only", LIB_PATH], capture_output=True, text=True, check=True).stdout


TYPES = r"I(f|DF16b|DF16_)"


def test_scored_routing(names):
    have = set(re.findall(r"24route_scored_rows_kernel" + TYPES + r"Li(\d+)ELi(\d+)ELi(\d+)EEEvNS0_10ScoredArgsE", names))
    few = {(16, 1, 256), (16, 2, 256), (16, 4, 256), (64, 4, 256), (64, 8, 256), (64, 16, 256)}
    many = {(16, 1, 1024), (16, 2, 1024), (16, 4, 1024), (16, 8, 1024), (16, 12, 512), (16, 16, 512), (16, 12, 1024),
            (16, 16, 1024), (64, 8, 1024), (64, 16, 512)}
    assert {tuple(map(int, k[1:])) for k in have} == few | many and len(have) == 3 * len(few | many)
    back = set(re.findall(r"28route_scored_backward_kernel" + TYPES + r"Li(\d+)ELi(\d+)EEEv", names))
    assert {tuple(map(int, k[1:])) for k in back} == {k[:2] for k in few | many}


def test_integer_products(names):
    quant = set(re.findall(r"20int8_quantize_kernel" + TYPES + r"Li(\d+)ELi(\d+)EEEv", names))
    assert {tuple(map(int, k[1:])) for k in quant} == {(64, 1), (64, 4), (256, 4), (256, 8), (256, 0)} and len(quant) == 15
    tails = {"0", "1"}
    ring = set(re.findall(r"16int8_ring_kernelILi(\d+)ELi(\d+)ELi(\d+)ELb(\d)EEEv", names))
    assert ring == {(*k, t) for k in [("2", "2", "4"), ("4", "2", "3")] for t in tails}
    skinny = set(re.findall(r"18int8_skinny_kernelILi(\d+)ELi(\d+)ELi(\d+)ELb(\d)EEEv", names))
    assert skinny == {(*k, t) for k in [("1", "1", "3"), ("2", "2", "2"), ("4", "4", "1")] for t in tails}


def test_adamw(names):
    have = set(re.findall(r"12adamw_kernelILi(\d+)ENS0_(\w+?)EEEvT0_", names))
    assert have == {(b, a) for b in ("8", "32") for a in ("4Some", "3All")}
