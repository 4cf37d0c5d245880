"""The first call of each paged-cache operator in a process, captured into a graph: what
is set up once (kernel attributes) is set up there."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

PROGRAM = """
import torch
import sink_sda_decode_gb300 as sda
i32 = dict(dtype=torch.int32, device="cuda")
q = torch.randn(2, 16, 512, device="cuda").to(torch.bfloat16)
pool = torch.randn(1024, 512, device="cuda").to(torch.bfloat16)
table = torch.arange(1024, **i32).view(2, 512)
ptr, n = torch.arange(3, **i32), torch.full((2,), 500, **i32)
sink, lse, scores = torch.zeros(16, device="cuda"), torch.zeros(2, 16, device="cuda"), torch.rand(2, 512, device="cuda")
call = {
    "attend": lambda: sda.chunk_attention(q, pool, table, ptr, n, sink, 0.04, k_per_block=1),
    "mass": lambda: [sda.attention_mass(q, pool, table, ptr, n, lse, 0.04, k_per_block=1)],
    "evict": lambda: sda.evict_slots(scores, table, n, 100, first=4, recent=10),
}[OP]
idx = torch.arange(1000, **i32)
sda.decode(q, pool, idx, torch.tensor([0, 500, 1000], **i32), sink, 0.04)
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    got = call()
g.replay()
torch.cuda.synchronize()
for a, b in zip(got, call()):
    assert torch.equal(a, b)
print("same")
"""


@pytest.mark.parametrize("op", ["attend", "mass", "evict"])
def test_first_call_captured(op):
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", f"OP = {op!r}\n" + PROGRAM], cwd=root, capture_output=True,
                       text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip() == "same", r.stderr[-2000:]
