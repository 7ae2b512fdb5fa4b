"""Windowed attention over the most keys that a call takes, 2^29 - 1: walks of
more than four million tiles, which take seconds each."""
import pytest

import vision_encoder_flash_gb300 as vef

pytestmark = pytest.mark.gpu

N, D = 2 ** 29 - 1, 8


@pytest.fixture(scope="module")
def kv():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    dev = torch.device("cuda", 0)
    if torch.cuda.mem_get_info(dev)[0] < 48 << 30:
        pytest.skip("needs 48 GB of free device memory")
    vef.load_library()
    k = torch.zeros(1, 1, N, D, dtype=torch.float16, device=dev)
    v = torch.full_like(k, 3.0)
    k[:, :, 0], v[:, :, 0] = 8.0, torch.arange(1, D + 1, device=dev)  # the key that takes all the weight
    yield torch, dev, k, v
    del k, v
    torch.cuda.empty_cache()


def test_forward_in_two_rounds(kv):
    """More items than blocks: a block's second item waits for the first's end."""
    torch, dev, k, v = kv
    heads = 2 * torch.cuda.get_device_properties(dev).multi_processor_count + 2
    q = torch.full((1, heads, 128, D), 8.0, dtype=k.dtype, device=dev)
    out, lse = vef.forward_window(q, k, v, scale=0.125, return_lse=True)
    torch.cuda.synchronize(dev)
    assert vef.device_status() == 0
    # scores 64 and 0: exp(-64) 2^29 is below 2^-63
    assert bool((out == v[:, :, :1]).all()) and bool((lse == 64).all())


def test_gradients(kv):
    torch, dev, k, v = kv
    q = torch.full((1, 1, 128, D), 8.0, dtype=k.dtype, device=dev)
    g = torch.ones_like(q)
    out, lse = vef.forward_window(q, k, v, scale=0.125, return_lse=True)
    dq, dk, dv = vef.backward_window(g, q, k, v, out, lse, scale=0.125)
    torch.cuda.synchronize(dev)
    assert vef.device_status() == 0
    # one key has all the weight: it gets the sum of dout, and nothing depends on the scores
    assert bool((dv[:, :, 0] == 128).all()) and not dv[:, :, 1:].any()
    assert not dq.any() and not dk.any()
