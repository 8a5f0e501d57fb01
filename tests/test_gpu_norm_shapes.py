"""The threads and chunks that layer norm gives a row of a width follow the tensors' types (from the dispatch log, in a
child process so that the environment variable is read at start-up)."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

SCRIPT = r"""
import sys, torch
sys.path.insert(0, sys.argv[1])
from precision_block_scaled_amd import pipeline as PL
BF, F32 = torch.bfloat16, torch.float32
for cols in (1032, 1200, 1536, 2056, 2560):
    for tx, ty in ((BF, BF), (BF, F32), (F32, BF), (F32, F32)):
        x, dy = torch.randn(64, cols, device="cuda").to(tx), torch.randn(64, cols, device="cuda").to(ty)
        print(f"[case] {cols} {str(tx)[6:]} {str(ty)[6:]}", file=sys.stderr, flush=True)
        _, mean, rstd = PL.layernorm(x, out_dtype=ty)
        PL.layernorm_grad(dy, x, None, mean, rstd)
torch.cuda.synchronize()
"""

# threads a row x chunks, (forward, gradient) for bf16 -> bf16, bf16 -> fp32, fp32 -> bf16, fp32 -> fp32: the shape with
# few empty threads, but for the wider types from where the next one measured faster
EXPECT = {1032: (("64 3", "64 3"), ("64 3", "64 3"), ("64 3", "64 3"), ("64 3", "256 1")),
          1200: (("64 3", "64 3"), ("64 3", "64 3"), ("64 3", "256 1"), ("64 3", "256 1")),
          1536: (("64 3", "256 1"), ("256 1", "256 1"), ("256 1", "256 1"), ("256 1", "256 1")),
          2056: (("192 2", "192 2"), ("192 2", "192 2"), ("256 2", "192 2"), ("256 2", "512 1")),
          2560: (("192 2", "192 2"), ("192 2", "192 2"), ("256 2", "512 1"), ("256 2", "512 1"))}


def test_shapes_follow_the_types():
    r = subprocess.run([sys.executable, "-c", SCRIPT, ROOT], capture_output=True, text=True,
                       env=dict(os.environ, PBS_LOG_LEVEL="1"), timeout=100, cwd=ROOT)
    assert r.returncode == 0, r.stderr[-2000:]
    got = {}
    for line in r.stderr.splitlines():
        if line.startswith("[case] "):
            case = line[7:]
        elif line.startswith("[pbs] layernorm"):
            f = dict(p.split("=") for p in line.split() if "=" in p)
            got.setdefault(case, []).append(f"{f['threads/row']} {f['chunks']}")
    names = ("bfloat16 bfloat16", "bfloat16 float32", "float32 bfloat16", "float32 float32")
    assert got == {f"{c} {n}": list(want) for c, row in EXPECT.items() for n, want in zip(names, row)}
