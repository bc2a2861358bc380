"""The operators' first calls of a process may be inside a CUDA graph's capture: what
they prepare then is not captured.  Runs in a process of its own."""
import os
import subprocess
import sys

import pytest

from tests._gpu import needs_gpu

pytestmark = [pytest.mark.gpu, needs_gpu]
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

SCRIPT = '''
import torch
import int4_routed_expert_renorm_b200 as cm
T, E, k, K, N = 9, 16, 2, 256, 384
g = torch.Generator(device="cuda").manual_seed(0)
logits = torch.randn(T, E, device="cuda", generator=g)
ids, w = torch.empty(T, k, dtype=torch.int32, device="cuda"), torch.empty(T, k, device="cuda")
a = torch.randint(0, 100, (T, K), dtype=torch.uint8, device="cuda", generator=g)
b = torch.randint(0, 100, (N, K), dtype=torch.uint8, device="cuda", generator=g)
sa, sb = torch.rand(T, 2, device="cuda", generator=g), torch.rand(3, 2, device="cuda", generator=g)
new = lambda *s, dtype=torch.float32: torch.zeros(s, dtype=dtype, device="cuda")
counts, n, P, loss, grad, d = (new(E, dtype=torch.int32), new(1, dtype=torch.int32), new(E), new(1),
                               torch.ones(1, device="cuda"), new(T, E))
out = new(T, N)
ws = torch.empty(cm.coli_moe_balance_workspace_bytes(T, E), dtype=torch.uint8, device="cuda")

def calls():
    cm.coli_moe_balance(logits, None, ids, None, counts, n, P, loss, ws)
    cm.coli_moe_balance_backward(logits, None, None, counts, n, grad, ids, w, None, d, None, ws)
    cm.coli_fp8_matmul(a, sa, b, sb, out)

cm.coli_moe_route(logits, None, ids, w)      # another call has prepared the device
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    calls()
graph.replay()
torch.cuda.synchronize()
got = [t.clone() for t in (counts, P, loss, d, out)]
assert int(n) == T and int(counts.sum()) == T * k and bool(out.any()) and bool(d.any())
for t in (counts, P, loss, d, out):
    t.zero_()
calls()
assert all(torch.equal(x, y) for x, y in zip(got, (counts, P, loss, d, out)))
assert cm.coli_moe_get_status() == (0, 0)
print("captured first")
'''


def test_first_calls_inside_a_capture():
    r = subprocess.run([sys.executable, "-c", SCRIPT], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "captured first" in r.stdout, r.stdout + r.stderr
