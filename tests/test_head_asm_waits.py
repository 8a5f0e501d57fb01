"""Static check of where the linear head's products wait for their loads (CPU).

The K loops fill their LDS stages by LDS-DMA.  In the middle of K stage k a
wave waits for its loads of stage k + 1, all but those of B's stage k + 2 that
it has just issued, and for its LDS reads, then meets the others.  Loads
finish in order, so the counted wait is right if it leaves out exactly the
loads issued since the loop's start, and if nothing else in the loop waits for
loads (the compiler adds such waits where it cannot tell an LDS read from a
load in flight) or issues scratch traffic of its own.
"""
import os
import re
import shutil
import subprocess
import tempfile

import pytest

from precision_block_scaled_amd import build as B
from tests.test_gemm_asm_waits import _op, functions, loop_blocks


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
            return functions(f.read().split("\n"), r"_ZN3pbs\d+head_(?:logits|grads)_kernel")


def test_k_loops_wait_at_their_barrier_alone(kernels):
    assert len(kernels) >= 8
    for name, body in kernels.items():
        loops = [b for _, blocks in loop_blocks(body) for b in blocks if any(_op(l).startswith("v_mfma") for l in b)]
        assert len(loops) == (2 if "head_grads" in name else 1), name
        for loop in loops:
            ops = [(_op(l), l) for l in loop]
            assert not any(o.startswith(("scratch_", "global_", "flat_")) for o, _ in ops), name
            at = [i for i, (o, _) in enumerate(ops) if o == "s_barrier"]
            waits = [i for i, (o, l) in enumerate(ops) if o == "s_waitcnt" and "vmcnt" in l]
            assert len(at) == 1 and len(waits) == 1, name
            left = int(re.search(r"vmcnt\((\d+)\)", ops[waits[0]][1]).group(1))
            assert "lgkmcnt(0)" in ops[waits[0]][1] and waits[0] < at[0], name
            assert not any(o.startswith(("buffer_load", "ds_")) for o, _ in ops[waits[0]:at[0]]), name
            before = sum(o.startswith("buffer_load") for o, _ in ops[:waits[0]])
            after = sum(o.startswith("buffer_load") for o, _ in ops[at[0]:])
            assert left == before == after > 0, (name, left, before, after)
