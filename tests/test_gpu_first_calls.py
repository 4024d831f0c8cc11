"""The first calls of a process, made by several host threads at once: the same bits as calls
made one by one.  How a grouped product shares a contraction out is asked of the device by a
thread's first call, and decides the order of its sums."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

CHILD = """
import threading
import torch
from combine_warp_top_gb300 import moe

moe.load()
THREADS, K, N = 12, 8192, 40
gen = torch.Generator(device="cuda")
gen.manual_seed(0)


def normal(*size):
    return torch.randn(*size, generator=gen, device="cuda").bfloat16()


shape, norm = moe.Shape(N, 8, 1, 1, 1, 8), moe.NormShape(300, 4096, gate="channel")
rows, w = normal(N, K), normal(1, 264, K)
y, r, v = normal(300, 4096), normal(300, 4096), normal(4096).float()
lay = moe.Layout(shape)
lay["expert_counts"].fill_(N)
lay["expert_offsets"].copy_(torch.tensor([0, N]))
torch.cuda.synchronize()


def call(stream):
    with torch.cuda.stream(stream):
        out = torch.zeros(N, 264, device="cuda")
        s, x = torch.zeros_like(r), torch.zeros_like(r)
        moe.moe_grouped_gemm(rows, lay, shape, w, out, workspaces[stream])
        moe.moe_block_norm(y, r, v, v, v, norm, s, x)
        return out, s, x


streams = [torch.cuda.Stream() for _ in range(THREADS)]
workspaces = {s: moe.workspace(shape) for s in streams}
torch.cuda.synchronize()
gate, got = threading.Barrier(THREADS), [None] * THREADS


def work(i):
    gate.wait()
    got[i] = call(streams[i])


threads = [threading.Thread(target=work, args=(i,)) for i in range(THREADS)]
for t in threads:
    t.start()
for t in threads:
    t.join()
torch.cuda.synchronize()
want = call(streams[0])
torch.cuda.synchronize()
for g in got:
    assert all(torch.equal(a, b) for a, b in zip(g, want))
assert all(moe.moe_get_error(ws) == 0 for ws in workspaces.values())
print("same bits")
"""


@pytest.mark.parametrize("attempt", range(3))
def test_first_calls_of_several_threads(attempt):
    r = subprocess.run([sys.executable, "-c", CHILD], cwd=ROOT, capture_output=True, text=True,
                       timeout=300)
    assert r.returncode == 0 and "same bits" in r.stdout, r.stdout + r.stderr
