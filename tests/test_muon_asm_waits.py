"""Static check of where the Newton-Schulz products wait for their loads (CPU), as for the linear head's.

In the middle of K stage k a wave waits for its loads of stage k + 1, all but
those of the stages after it up to the one D ahead, of which B's have been
issued, and for its LDS reads, then meets the others: the counted wait has to
leave out exactly D - 2 stages' loads and the loop's own so far, and nothing
else in the loop may wait for loads or move scratch memory.
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
        out = os.path.join(d, "muon.s")
        r = subprocess.run([B.hipcc(), *B.compile_flags(), "--cuda-device-only", "-S",
                            os.path.join(B.CSRC, "muon.hip"), "-o", out], capture_output=True, text=True)
        assert r.returncode == 0, r.stderr[-2000:]
        with open(out) as f:
            return functions(f.read().split("\n"), r"_ZN3pbs\d+ns_product_kernel")


def test_k_loops_wait_at_their_barrier_alone(kernels):
    assert len(kernels) == 4 * 6 + 5 + 2 * 5        # symmetric products, the next X, the last one in two types
    for name, body in kernels.items():
        loops = [b for _, blocks in loop_blocks(body) for b in blocks if any(_op(l).startswith("v_mfma") for l in b)]
        assert len(loops) == 1, name
        ops = [(_op(l), l) for l in loops[0]]
        assert not any(o.startswith(("scratch_", "global_", "flat_")) for o, _ in ops), name
        at = [i for i, (o, _) in enumerate(ops) if o == "s_barrier"]
        waits = [i for i, (o, l) in enumerate(ops) if o == "s_waitcnt" and "vmcnt" in l]
        assert len(at) == 1 and len(waits) == 1, name
        left = int(re.search(r"vmcnt\((\d+)\)", ops[waits[0]][1]).group(1))
        assert "lgkmcnt(0)" in ops[waits[0]][1] and waits[0] < at[0], name
        assert not any(o.startswith(("buffer_load", "ds_")) for o, _ in ops[waits[0]:at[0]]), name
        before = sum(o.startswith("buffer_load") for o, _ in ops[:waits[0]])
        after = sum(o.startswith("buffer_load") for o, _ in ops[at[0]:])
        ahead = int(re.search(r"ILi\d+ELi(\d+)E", name).group(1))
        assert left == (ahead - 2) * (before + after) + before and before == after > 0, (name, left, before, after)
