"""Static check of where the linear head's products wait for their loads (CPU).

The K loops fill their LDS stages by LDS-DMA and wait for a stage once, at the
barrier between its halves (see test_gemm_asm_waits.py, whose reading of the
compiled code this uses).  Every instantiation's loop must have that wait at
its barrier with no load in between, no other wait for loads, and no scratch
traffic, whose own loads and stores the wait would count.
"""
import os
import re
import shutil
import subprocess
import tempfile

import pytest

from precision_block_scaled_amd import build as B
from tests.test_gemm_asm_waits import _op, check_barrier_waits, functions, loop_blocks


@pytest.fixture(scope="module")
def kernels():
    if not (shutil.which("hipcc") or os.path.exists("/opt/rocm/bin/hipcc")):
        pytest.skip("hipcc not found")
    with tempfile.TemporaryDirectory() as d:
        out = os.path.join(d, "head.s")
        r = subprocess.run([B.hipcc(), *B.compile_flags(), "--cuda-device-only", "-S",
                            os.path.join(B.CSRC, "head.hip"), "-o", out], capture_output=True, text=True)
        assert r.returncode == 0, r.stderr[-2000:]
        with open(out) as f:
            return functions(f.read().split("\n"), "_ZN3pbs16head_gemm_kernel")


def test_k_loops_wait_at_their_barrier_alone(kernels):
    assert len(kernels) >= 4
    for name, body in kernels.items():
        loops = [b for _, blocks in loop_blocks(body) for b in blocks]
        bars = [b for b in loops if any(_op(l) == "s_barrier" for l in b)]
        assert bars, name
        for blk in loops:
            assert not check_barrier_waits(blk), (name, check_barrier_waits(blk))
            assert not any(_op(l).startswith("scratch_") for l in blk), name
            at = [i for i, l in enumerate(blk) if _op(l) == "s_barrier"]
            for i, l in enumerate(blk):
                if _op(l) == "s_waitcnt" and re.search(r"vmcnt\(", l):
                    assert any(0 < b - i < 12 for b in at), (name, l)
