"""The library holds no routing kernel that no call reaches."""

import os
import re
import shutil
import subprocess

import pytest

from moe_grouped_gemm_quantizer_amd._lib import LIB_PATH


@pytest.mark.skipif(not os.path.exists(LIB_PATH) or shutil.which("nm") is None, reason="library or nm missing")
def test_rows_kernels_are_the_ones_that_are_picked():
    names = subprocess.run(["nm", "--defined-only", LIB_PATH], capture_output=True, text=True, check=True).stdout
    # (the host's handle of each kernel; template arguments: type, lanes of a row, values of a lane, threads)
    have = set(re.findall(r"17route_rows_kernelI(f|DF16b|DF16_)Li(\d+)ELi(\d+)ELi(\d+)EEEvNS0_9RouteArgsE", names))
    few = {(lanes, per, 256) for lanes, per in ((16, 1), (16, 2), (16, 4), (64, 4), (64, 8), (64, 16))}
    many = {(16, 1, 1024), (16, 2, 1024), (16, 4, 1024), (16, 8, 1024), (16, 12, 512), (16, 16, 512),
            (64, 8, 1024), (64, 16, 1024)}
    assert {(int(a), int(b), int(c)) for _, a, b, c in have} == few | many
    assert len(have) == 3 * len(few | many)
