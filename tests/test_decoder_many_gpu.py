"""The decoder calls with more sequences, heads and callers than a grid
dimension, a warp or a stream holds: each part as the same part alone."""
import threading

import pytest

import vision_encoder_flash_gb300 as vef
from decoder_util import normal

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def td():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    vef.load_library()
    return torch, torch.device("cuda", 0)


def test_many_sequences(td):
    torch, dev = td
    B, M, D = 70001, 5, 16
    q, g = (normal(torch, (B, 2, M, D), "f16", 300 + i, dev) for i in range(2))
    k, v = (normal(torch, (B, 1, 9, D), "f16", 302 + i, dev) for i in range(2))
    lens = torch.arange(B, dtype=torch.int32, device=dev) % 11
    how = dict(window=4, n_sinks=1, scale=0.3)
    w = torch.linspace(0.5, 2.0, D, device=dev)
    positions = (torch.arange(B * M, dtype=torch.int32, device=dev) * 7919).view(B, M)
    kr = torch.zeros(B, 1, M, D, dtype=q.dtype, device=dev)

    def run(a, b):
        s = slice(a, b)
        how_s = dict(how, kv_len=lens[s])
        qn, _ = vef.qk_norm_rope(q[s], kr[s], w, w, positions=positions[s].contiguous())
        dn = vef.qk_norm_rope_backward(g[s], kr[s], q[s], kr[s], positions=positions[s].contiguous())
        out, lse = vef.forward_window(q[s], k[s], v[s], return_lse=True, **how_s)
        grads = vef.backward_window(g[s], q[s], k[s], v[s], out, lse, **how_s)
        return (qn, dn[0], out, lse, *grads, vef.forward_cached(q[s], k[s], v[s], **how_s))

    whole = run(0, B)
    for a in (0, 32767, 65534, 65535, 65536, B - 1):
        for x, y in zip(run(a, a + 1), whole):
            assert torch.equal(x, y[a:a + 1])
    assert vef.device_status() == 0


def test_many_heads(td):
    torch, dev = td
    H, D = 300001, 8
    q, k = (normal(torch, (1, h, 2, D), "bf16", 310 + i, dev) for i, h in enumerate((H, 3)))
    got = vef.qk_norm_rope(q, k, pos0=5)
    back = vef.qk_norm_rope_backward(q, k, q, k, pos0=5)
    for a in (0, 16383, 16384, 262144, H - 1):
        part = q[:, a:a + 1]
        want = vef.qk_norm_rope(part, k, pos0=5)
        assert torch.equal(got[0][:, a:a + 1], want[0]) and torch.equal(got[1], want[1])
        want = vef.qk_norm_rope_backward(part, k, part, k, pos0=5)
        assert torch.equal(back[0][:, a:a + 1], want[0]) and torch.equal(back[1], want[1])
    # one key head for 1030 query heads: 65920 rows of 64 new tokens
    q = normal(torch, (1, 1030, 64, 16), "f16", 312, dev)
    k, v = (normal(torch, (1, 1, 100, 16), "f16", 313 + i, dev) for i in range(2))
    lens = torch.tensor([90], dtype=torch.int32, device=dev)
    got = vef.forward_cached(q, k, v, lens, scale=0.2)
    for a in (0, 513, 1029):
        assert torch.equal(got[:, a:a + 1], vef.forward_cached(q[:, a:a + 1].contiguous(), k, v, lens, scale=0.2))


def test_threads(td):
    """Four host threads, each on its own stream, forty rounds of all calls."""
    torch, dev = td
    x = [normal(torch, (2, h, 400, 64), "bf16", 320 + i, dev) for i, h in enumerate((4, 2, 2, 4))]
    w = torch.linspace(0.5, 1.5, 64, device=dev)
    lens = torch.tensor([400, 250], dtype=torch.int32, device=dev)
    how = dict(window=90, n_sinks=2, scale=0.125, kv_len=lens)

    def run():
        qn, kn = vef.qk_norm_rope(x[0], x[1], w, w)
        out, lse = vef.forward_window(qn, kn, x[2], return_lse=True, **how)
        grads = vef.backward_window(x[3], qn, kn, x[2], out, lse, **how)
        back = vef.qk_norm_rope_backward(grads[0], grads[1], x[0], x[1], w, w)
        return (qn, kn, out, lse, *grads, *back, vef.forward_cached(qn[:, :, -3:], kn, x[2], **how))

    want = run()
    torch.cuda.synchronize(dev)
    errors = []

    def worker():
        try:
            torch.cuda.set_device(dev)
            stream = torch.cuda.Stream(dev)
            with torch.cuda.stream(stream):
                for _ in range(40):
                    got = run()
                stream.synchronize()
                if not all(torch.equal(a, b) for a, b in zip(got, want)):
                    errors.append("different results")
        except Exception as e:  # noqa: BLE001 - reported below
            errors.append(repr(e))

    threads = [threading.Thread(target=worker) for _ in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors and vef.device_status() == 0
