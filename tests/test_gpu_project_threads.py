"""moe_project called for the first time by several threads at once, each on its stream: the table by which shares of K are
chosen is filled once and read complete."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

PROGRAM = """
import threading
import torch
from sparse_moe_router_gb300 import abi

gen = torch.Generator(device="cuda").manual_seed(1)
x, w = (torch.randn(n, 2048, device="cuda", generator=gen).to(torch.bfloat16) for n in (48, 1024))
cfg = abi.project_config(2048, 1024)
streams = [torch.cuda.Stream() for _ in range(8)]
outs = [torch.empty(48, 1024, dtype=torch.bfloat16, device="cuda") for _ in streams]
spaces = [abi.alloc_project_workspace(cfg, 48) for _ in streams]
abi.load()
gate, errors = threading.Barrier(len(streams)), []

def call(i):
    try:
        gate.wait(30)
        abi.moe_project(cfg, x, w, outs[i], spaces[i], stream=streams[i])
    except Exception as e:
        errors.append(e)

torch.cuda.synchronize()
threads = [threading.Thread(target=call, args=(i,)) for i in range(len(streams))]
for t in threads:
    t.start()
for t in threads:
    t.join()
torch.cuda.synchronize()
assert not errors, errors
want = torch.empty_like(outs[0])
abi.moe_project(cfg, x, w, want, spaces[0])
assert all(torch.equal(o, want) for o in outs)
assert all(abi.moe_check_status(s) == 0 for s in spaces)
"""


def test_first_calls_of_several_threads():
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    for _ in range(3):
        r = subprocess.run([sys.executable, "-c", PROGRAM], cwd=root, capture_output=True, text=True, timeout=300)
        assert r.returncode == 0, r.stderr[-2000:]
