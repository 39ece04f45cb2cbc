"""The packed and paged calls captured into a graph as the first calls of a process.

What a first call sets up (scratch pool, status word, kernels) may not depend on
a call outside a capture, so each case runs in a process of its own.
"""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

CODE = """
import sys
sys.path.insert(0, {root!r})
import torch
import head_dim_attention_gb300 as f
i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")
new = lambda *shape: torch.randn(*shape, device="cuda").half()
q, k, v, dout = new(1, 4, 300, 512), new(1, 2, 300, 512), new(1, 2, 300, 512), new(1, 4, 300, 512)
cu, lse, out = i32([0, 100, 300]), torch.zeros(1, 4, 300, device="cuda"), new(1, 4, 300, 512)
kc, vc, table, n = new(20, 2, 16, 512), new(20, 2, 16, 512), torch.arange(20, device="cuda").int()[None], i32([300])
q1, o1, l1 = new(1, 4, 1, 512), new(1, 4, 1, 512), torch.zeros(1, 4, 1, device="cuda")
slots, free, head, step = torch.arange(300, device="cuda"), i32([0]), i32([0]), i32([3])
calls = {{
    "varlen_fwd": lambda: f.attention_varlen_fwd(q, k, v, cu, causal=True, out=out, lse=lse),
    "varlen_bwd": lambda: f.attention_varlen_bwd(q, k, v, cu, out, lse, dout, causal=True),
    "tree": lambda: f.attention_tree_fwd(q1, kc, vc, table, n, out=o1, lse=l1),
    "plan": lambda: f.cache_plan(n, step, table.clone(), free, head, 16, 8),
    "append": lambda: f.cache_append(k, v, kc, vc, slots),
}}
f.load()
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    kept = calls[{which!r}]()
graph.replay()
torch.cuda.synchronize()
assert f.ffpa_check_status() == 0
captured = [x.clone() for x in (kept or (kc, vc))]
again = calls[{which!r}]() or (kc, vc)
torch.cuda.synchronize()
assert all(torch.equal(a, b) for a, b in zip(captured, again))
print("captured first")
"""


@pytest.mark.parametrize("which", ["varlen_fwd", "varlen_bwd", "tree", "plan", "append"])
def test_first_call_may_be_captured(which):
    r = subprocess.run([sys.executable, "-c", CODE.format(root=ROOT, which=which)], capture_output=True, text=True,
                       timeout=300, cwd=ROOT)
    assert r.returncode == 0 and "captured first" in r.stdout, r.stdout[-500:] + r.stderr[-2000:]
