"""How much device memory the gradients of windowed attention keep."""
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

CHILD = """
import torch
import vision_encoder_flash_gb300 as vef
dev = torch.device("cuda:0")
B, N, D = 5, 243 * 128, 128
x = [torch.randn(B, 1, N, D, device=dev).to(torch.bfloat16) for _ in range(4)]
grads = [torch.empty_like(x[0]) for _ in range(3)]
how = dict(window=1, n_sinks=N, scale=0.1)
out, lse = vef.forward_window(*x[:3], return_lse=True, **how)
small = [t[:, :, :100].contiguous() for t in x]
o, l = vef.forward_window(*small[:3], return_lse=True, scale=0.1)
vef.backward_window(small[3], *small[:3], o, l, scale=0.1)   # the pool and the kernels are there
torch.cuda.synchronize()
free = torch.cuda.mem_get_info(dev)[0]
vef.backward_window(x[3], *x[:3], out, lse, dq=grads[0], dk=grads[1], dv=grads[2], **how)
torch.cuda.synchronize()
print("took", free - torch.cuda.mem_get_info(dev)[0], torch.cuda.get_device_properties(dev).multi_processor_count)
assert vef.device_status() == 0
"""


def test_first_keys_in_eight_pieces_a_multiprocessor():
    """1215 tiles of first keys: as many pieces as the bound has room for, one
    each, not one more for every tile."""
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    r = subprocess.run([sys.executable, "-c", CHILD], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "took" in r.stdout, r.stderr[-2000:]
    took, sms = (int(x) for x in r.stdout.split("took")[1].split())
    # pieces of 128 KiB, 1 KiB of statistics for every 128 rows, and what the pool rounds up
    assert took <= 8 * sms * 2 ** 17 + 5 * 243 * 2 ** 10 + 2 ** 26, took
