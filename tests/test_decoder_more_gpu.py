"""The decoder calls where the other tests take a shorter way: every round of
several threads, and caches of more shares than a join takes at once."""
import threading

import numpy as np
import pytest

from oracle import decoder as od
import vision_encoder_flash_gb300 as vef
from decoder_util import HALF_STEP, TINY, assert_within, f64, normal

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def td():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    vef.load_library()
    return torch, torch.device("cuda", 0)


@pytest.mark.parametrize("name", ["bf16", "f16"])
def test_every_round_of_threads(td, name):
    """Four host threads, each on its own stream, thirty rounds of all calls, each
    round compared on the device."""
    torch, dev = td
    x = [normal(torch, (2, h, 500, 72), name, 600 + i, dev) for i, h in enumerate((4, 2, 2, 4))]
    x[2][0, 0, 200, 7] = float("inf")  # hidden from the rows before it: the forward pass takes a second look
    w = torch.linspace(0.5, 1.5, 72, device=dev)
    lens = torch.tensor([500, 250], dtype=torch.int32, device=dev)
    how = dict(window=90, n_sinks=2, scale=0.125, kv_len=lens)
    v = torch.nan_to_num(x[2], posinf=1.0)

    def run():
        qn, kn = vef.qk_norm_rope(x[0], x[1], w, w)
        out, lse = vef.forward_window(qn, kn, x[2], return_lse=True, **how)
        fine, lse2 = vef.forward_window(qn, kn, v, return_lse=True, **how)
        grads = vef.backward_window(x[3], qn, kn, v, fine, lse2, **how)
        back = vef.qk_norm_rope_backward(grads[0], grads[1], x[0], x[1], w, w)
        return (qn, kn, out, lse, fine, *grads, *back, vef.forward_cached(qn[:, :, -3:], kn, v, **how))

    bits = {2: torch.int16, 4: torch.int32}
    want = [t.view(bits[t.element_size()]) for t in run()]
    torch.cuda.synchronize(dev)
    errors = []

    def worker():
        try:
            torch.cuda.set_device(dev)
            stream = torch.cuda.Stream(dev)
            with torch.cuda.stream(stream):
                wrong = torch.zeros(len(want), dtype=torch.int64, device=dev)
                for _ in range(30):
                    got = run()
                    wrong += torch.stack([(a.view(b.dtype) != b).any().long() for a, b in zip(got, want)])
                stream.synchronize()
                if bool(wrong.any()):
                    errors.append(wrong.tolist())
        except Exception as e:  # noqa: BLE001 - reported below
            errors.append(repr(e))

    threads = [threading.Thread(target=worker) for _ in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors and vef.device_status() == 0


@pytest.mark.parametrize("T,tree", [(1, False), (3, True), (11, False)])
@pytest.mark.parametrize("N", [33000, 40001, 140000])
def test_many_shares(td, N, T, tree):
    """One sequence in 129 to 512 shares of its keys."""
    torch, dev = td
    H, D = 2, 32
    q, k, v = (normal(torch, s, "f16", 620 + i, dev) for i, s in enumerate(((1, H, T, D), (1, 1, N, D), (1, 1, N, D))))
    lens = torch.tensor([N - 5], dtype=torch.int32, device=dev)
    words = [1, 3, 5] if tree else None
    mask = None if words is None else torch.tensor([words], dtype=torch.int64, device=dev)
    out = vef.forward_cached(q, k, v, lens, tree_mask=mask, scale=0.2)
    seen = od.cached_visible(T, N, None, 0, N - 5, words)[None]
    want, _, _, bound, _, _ = od.attention(f64(q), f64(k), f64(v), seen, float(np.float32(0.2)), HALF_STEP["f16"])
    assert_within(out, want, bound, "out", tiny=2 * TINY["f16"])
    assert torch.equal(out, vef.forward_cached(q, k, v, lens, tree_mask=mask, scale=0.2))
    # equal weights and values 0 or 1: all sums are exact, and a share that is left out shows
    k.zero_()
    v.copy_((v > 0.3).half())
    out = vef.forward_cached(q, k, v, lens, tree_mask=mask, scale=0.2)
    for t in range(T):
        count = f64(v[0, 0])[seen[0, t]].sum(0)
        want = np.broadcast_to(count / seen[0, t].sum(), (H, D))
        # one f32 reciprocal, one f32 product, one rounding to f16
        assert_within(out[0, :, t], want, 2.0 ** -22 * want, "share", u=HALF_STEP["f16"])


def test_scores_of_minus_infinity(td):
    """A row whose scores are all -infinity counts as one that sees nothing."""
    torch, dev = td
    for D in (64, 128):
        q, k, v = (normal(torch, (1, 2, 200, D), "bf16", 640 + i, dev) for i in range(3))
        q = q.abs() + 0.1
        k[:, :, :150] = float("-inf")
        out, lse = vef.forward_window(q, k, v, return_lse=True)
        assert not out[:, :, :150].any() and bool(torch.isneginf(lse[:, :, :150]).all())
        alone = vef.forward_window(q, torch.cat([torch.zeros_like(k[:, :, :150]), k[:, :, 150:]], 2), v, window=1)
        assert torch.equal(out[:, :, 150], alone[:, :, 150])  # its own key alone
        assert bool(torch.isfinite(out).all())
        lens = torch.tensor([150], dtype=torch.int32, device=dev)
        assert not vef.forward_cached(q[:, :, :3], k, v, lens).any()
