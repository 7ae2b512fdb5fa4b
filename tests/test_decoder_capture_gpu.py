"""The decoder calls captured into a CUDA graph as a process's first calls:
what a call sets up once (attributes, workspace pool, symbol addresses) must
not disturb the capture."""
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

CHILD = """
import sys
import torch
import vision_encoder_flash_gb300 as vef
dev = torch.device("cuda:0")
torch.manual_seed(1)
q, g = (torch.randn(2, 4, 300, 64, device=dev).to(torch.bfloat16) for _ in range(2))
k, v = (torch.randn(2, 2, 300, 64, device=dev).to(torch.bfloat16) for _ in range(2))
w = torch.randn(64, device=dev)
lens = torch.full((2,), 300, dtype=torch.int32, device=dev)
how = dict(window=70, n_sinks=3, scale=0.125)

def norm():
    return vef.qk_norm_rope(q, k, w, w)

def norm_gradient():
    return vef.qk_norm_rope_backward(g, k, q, k, w, w)

def window():
    return vef.forward_window(q, k, v, return_lse=True, **how)

def window_gradient():
    out = torch.zeros_like(q)
    lse = torch.zeros(2, 4, 300, device=dev)
    return vef.backward_window(g, q, k, v, out, lse, **how)

def cached():
    return (vef.forward_cached(q[:, :, :5], k, v, lens, **how),)

call = dict(norm=norm, norm_gradient=norm_gradient, window=window, window_gradient=window_gradient,
            cached=cached)[sys.argv[1]]
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    got = call()
for _ in range(2):
    graph.replay()
torch.cuda.synchronize()
assert all(torch.equal(a, b) for a, b in zip(got, call()))
assert vef.device_status() == 0
print("captured")
"""


@pytest.mark.parametrize("call", ["norm", "norm_gradient", "window", "window_gradient", "cached"])
def test_first_call_in_a_capture(call):
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    r = subprocess.run([sys.executable, "-c", CHILD, call], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "captured" in r.stdout, r.stderr[-2000:]
