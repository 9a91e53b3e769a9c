"""A process whose first calls are captured into a graph: nothing has been set up before,
and the graph's results are the eager calls'."""

import os
import subprocess
import sys

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CODE = """
import sys
import torch
import ggml_q2_quantized_gb300 as q2k

torch.cuda.set_device(0)
n_tokens, top_k, experts, n, k = int(sys.argv[1]), 2, 3, 256, 1024
w = torch.randint(0, 120, (experts * n * (k // 256) * 84,), dtype=torch.uint8, device="cuda:0")
x = torch.randn(n_tokens, k, device="cuda:0").bfloat16()
ids = torch.randint(-1, experts, (n_tokens, top_k), device="cuda:0", dtype=torch.int32)
weights = torch.rand(n_tokens, top_k, device="cuda:0")

def step():
    routes, _ = q2k.moe_route(ids, experts, check=False)
    xs = q2k.moe_sort(x, routes)
    y, z = q2k.linear(xs, w, n, act="silu", save=True, routes=routes)
    out = q2k.moe_combine(y, routes, weights=weights)
    dys, dw = q2k.moe_combine_backward(out, y, routes, weights)
    dx, _, db = q2k.linear_backward(dys, w, k, z=z, act="silu", bias=True, routes=routes)
    flat = q2k.linear(x, w[:w.numel() // experts], n)
    back = q2k.linear_backward(flat, w[:w.numel() // experts], k)[0]
    return out, dw, db, q2k.moe_sort_backward(dx, routes), flat, back

graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    held = step()
graph.replay()
torch.cuda.synchronize()
held = [t.clone() for t in held]
want = step()
torch.cuda.synchronize()
assert all(torch.equal(a, b) for a, b in zip(held, want)), [torch.equal(a, b) for a, b in zip(held, want)]
assert q2k.device_error() == 0
print("same")
"""


@pytest.mark.parametrize("n_tokens", [1, 200])
def test_first_calls_in_a_capture(n_tokens):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    res = subprocess.run([sys.executable, "-c", CODE, str(n_tokens)], cwd=ROOT, capture_output=True,
                         text=True, timeout=240)
    assert res.returncode == 0 and res.stdout.strip() == "same", res.stderr[-2000:]
