"""ace_moe_group asks the device once for the clusters it can place: a process whose
first call is captured gets a graph that replays like any other."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

CODE = """
import numpy as np, torch
from token_dynamic_expert_b200 import ace
import i8_oracle as ora
idx = torch.zeros(5000, 6, dtype=torch.int32, device="cuda")
off, so = torch.empty(33, dtype=torch.int32, device="cuda"), torch.empty_like(idx)
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    ace.ace_moe_group(idx, 32, off, so)
for seed in range(3):
    idx.copy_(torch.randint(0, 32, idx.shape, device="cuda", dtype=torch.int32))
    g.replay()
    torch.cuda.synchronize()
    roff, rso, _ = ora.group(idx.cpu().numpy(), None, 32)
    assert np.array_equal(off.cpu().numpy(), roff) and np.array_equal(so.cpu().numpy(), rso)
    ace.ace_moe_group(idx, 32, off, so)
    assert np.array_equal(so.cpu().numpy(), rso)
print("same")
"""


def test_first_call_of_a_process_is_captured():
    env = dict(os.environ, PYTHONPATH=os.pathsep.join([ROOT, os.path.join(ROOT, "tests")]))
    r = subprocess.run([sys.executable, "-c", CODE], capture_output=True, text=True, timeout=300, env=env, cwd=ROOT)
    assert r.returncode == 0 and r.stdout.strip() == "same", r.stdout + r.stderr
