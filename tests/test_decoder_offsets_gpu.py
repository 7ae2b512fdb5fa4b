"""The decoder calls on tensors whose rows lie further apart than 32 bits of
bytes, and of elements, reach: the same results as on compact tensors, and
nothing else written."""
import pytest

import vision_encoder_flash_gb300 as vef
from decoder_util import normal

pytestmark = pytest.mark.gpu

ROWS, STRIDE, DIM = 300, 1 << 24, 64  # 299 rows on: 5.0e9 elements


@pytest.fixture(scope="module")
def far():
    """far(x): the values of x [1, heads, ROWS, DIM] in rows STRIDE elements
    apart, in 64-element columns of one 10 GB buffer; far(): such a view to
    write to."""
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    vef.load_library()
    dev = torch.device("cuda", 0)
    if torch.cuda.mem_get_info(dev)[0] < 24 << 30:
        pytest.skip("needs 24 GB of free device memory")
    buffer = torch.empty(ROWS * STRIDE, dtype=torch.bfloat16, device=dev)
    used = [0]

    def take(x=None, heads=None):
        heads = x.shape[1] if x is not None else heads
        view = buffer.as_strided((1, heads, ROWS, DIM), (0, 2 * DIM, STRIDE, 1), used[0])
        buffer.as_strided((ROWS, 2 * DIM * heads), (STRIDE, 1), used[0]).fill_(9.0)
        used[0] += 2 * DIM * heads
        if x is not None:
            view.copy_(x)
        return view

    def between(view):  # the columns between a view's heads
        return view.as_strided(view.shape, view.stride(), view.storage_offset() + DIM)

    yield torch, dev, take, between
    del buffer
    torch.cuda.empty_cache()


def test_rows_far_apart(far):
    torch, dev, take, between = far
    q, k, v, g = (normal(torch, (1, h, ROWS, DIM), "bf16", 200 + i, dev) for i, h in enumerate((4, 2, 2, 4)))
    w = torch.linspace(0.5, 1.5, DIM, device=dev)
    fq, fk, fv, fg = (take(t) for t in (q, k, v, g))
    outs = [take(heads=h) for h in (4, 2, 4, 2, 4, 4, 2, 2, 4)]
    how = dict(window=120, n_sinks=3, scale=0.125)
    # norm and rotation, forward and gradient
    want = vef.qk_norm_rope(q, k, w, w)
    got = vef.qk_norm_rope(fq, fk, w, w, q_out=outs[0], k_out=outs[1])
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    want = vef.qk_norm_rope_backward(g, v, q, k, w, w)
    got = vef.qk_norm_rope_backward(fg, fv, fq, fk, w, w, dq=outs[2], dk=outs[3])
    assert all(torch.equal(a, b) for a, b in zip(got[:2], want[:2]))
    for a, b in zip(got[2:], want[2:]):  # as many partial sums in the same order
        assert torch.equal(a, b)
    # attention, its gradients, and over a cache
    want, lse = vef.forward_window(q, k, v, return_lse=True, **how)
    got, flse = vef.forward_window(fq, fk, fv, out=outs[4], return_lse=True, **how)
    assert torch.equal(got, want) and torch.equal(flse, lse)
    grads = vef.backward_window(g, q, k, v, want, lse, **how)
    got = vef.backward_window(fg, fq, fk, fv, outs[4], lse, dq=outs[5], dk=outs[6], dv=outs[7], **how)
    assert all(torch.equal(a, b) for a, b in zip(got, grads))
    lens = torch.tensor([ROWS], dtype=torch.int32, device=dev)
    for T in (1, 40):
        want = vef.forward_cached(q[:, :, -T:], k, v, lens, **how)
        got = vef.forward_cached(fq[:, :, -T:], fk, fv, lens, out=outs[8][:, :, -T:], **how)
        assert torch.equal(got, want)
    assert all(bool((between(t) == 9).all()) for t in outs)
    assert vef.device_status() == 0
