"""The operators with scales for blocks of 128 where a call meets its surroundings: a first call under
capture."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


FIRST = """
import sys
sys.path.insert(0, {root!r})
import torch
import fp8_block_scaled_06_gb300 as f
u = lambda *s: torch.randint(0, 0x70, s, dtype=torch.uint8, device="cuda")
one = lambda *s: torch.ones(s, device="cuda")
A, B = (u(12000, 272), one(94, 272)), (u(12000, 400), one(94, 400))
x, W, gu, dh = (u(3, 512), one(4, 3)), (u(512, 512), one(4, 4)), (u(3, 512), one(4, 3)), torch.randn((3, 256), device="cuda")
def step():
    return [f.gemm_block128(*A, *B, form="tn", out="f32"), f.gemm_block128(*x, *W), *f.gated_block128(*x, *W)[0],
            *f.gated_block128_backward(dh, *gu)[2]]
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    got = step()
g.replay()
torch.cuda.synchronize()
assert all(torch.equal(a, b) for a, b in zip(got, step()))
assert f.fp8_gemm_status()[0] == 0
print("right")
"""


def test_a_first_call_under_capture(fp8g):
    r = subprocess.run([sys.executable, "-c", FIRST.format(root=ROOT)], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip() == "right", r.stderr[-2000:]
