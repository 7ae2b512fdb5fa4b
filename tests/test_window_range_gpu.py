"""Gradients of windowed attention whose terms lie at the ends of the type's
range: small and large gradients, weights of long rows."""
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


# dout's size, k's size (q's is its inverse, so that the scores stay), v's size
SIZES = [(1e-3, 32.0, 1.0), (1e-5, 32.0, 1.0), (1e-7, 512.0, 1.0), (1e-3, 1 / 32.0, 1.0), (1e-5, 1 / 256.0, 1.0),
         (1e3, 1 / 64.0, 1.0), (1.2e4, 1 / 256.0, 0.5), (100.0, 1 / 512.0, 1000.0), (1e-5, 16.0, 100.0), (1.0, 1.0, 1.0)]


@pytest.mark.parametrize("shape,window,sinks", [((1, 2, 1, 700, 64), None, 0), ((1, 4, 2, 1200, 96), 300, 3)])
@pytest.mark.parametrize("size", SIZES)
@pytest.mark.parametrize("name", ["f16", "bf16"])
def test_sizes_of_gradients(td, name, size, shape, window, sinks):
    """Bounds relative to the terms: nothing is allowed for terms below the
    type's normal numbers but what the largest of them gives (below)."""
    torch, dev = td
    B, H, K, N, D = shape
    g_size, k_size, v_size = size
    u, tiny = HALF_STEP[name], TINY[name]
    q, k, v, g = (normal(torch, (B, h, N, D), name, 500 + i, dev, s)
                  for i, (h, s) in enumerate(((H, 1 / k_size), (K, k_size), (K, v_size), (H, g_size))))
    how = dict(window=window, n_sinks=sinks, scale=0.7 / D ** 0.5)
    out, lse = vef.forward_window(q, k, v, return_lse=True, **how)
    grads = vef.backward_window(g, q, k, v, out, lse, **how)
    seen = od.window_visible(N, N, window, sinks, None, None)[None]
    scale = float(np.float32(how["scale"]))
    a = [f64(t) for t in (q, k, v, g)]
    want, _, weights, bound, score, _ = od.attention(*a[:3], seen, scale, u)
    # out is rounded to the type, which has no digits below its normal numbers
    bound = bound + 2 * tiny
    wants, bounds = od.attention_backward(a[3], *a[:3], want, weights, seen, scale, u, bound, score)
    # f16: weights and score gradients are held with 2^-40 of the largest that they can be, 1 and
    # 2 |dout| |v|, as their smallest step, however many a sum has
    step = 2.0 ** -40 if name == "f16" else 0.0
    most = 2 * max(np.linalg.norm(a[3], axis=-1).max() * np.linalg.norm(a[2], axis=-1).max(), 1e-300)
    rows = H // K * N
    floors = (step * most * scale * np.abs(a[1]).max() * N, step * most * scale * np.abs(a[0]).max() * rows,
              step * np.abs(a[3]).max() * rows)
    for got, w, b, f, what in zip(grads, wants, bounds, floors, ("dq", "dk", "dv")):
        if np.abs(w).max() > 6e4 and name == "f16":
            continue  # not representable
        assert_within(got, w, b, what, tiny=2 * tiny + f)
    assert all(torch.equal(x, y) for x, y in zip(grads, vef.backward_window(g, q, k, v, out, lse, **how)))


def test_weights_of_long_rows(td):
    """16 rows at the end of 300000 keys: weights of 2^-18, below f16's normal
    numbers; dv, a sum of few of them, keeps its digits."""
    torch, dev = td
    N, M, D = 300000, 16, 16
    q, g = (normal(torch, (1, 2, M, D), "f16", 520 + i, dev, s) for i, s in enumerate((0.1, 600.0)))
    k, v = (normal(torch, (1, 1, N, D), "f16", 522 + i, dev) for i in range(2))
    how = dict(scale=0.5)
    out, lse = vef.forward_window(q, k, v, return_lse=True, **how)
    _, _, dv = vef.backward_window(g, q, k, v, out, lse, **how)
    s = (q.double() @ k.double().transpose(2, 3)) * 0.5
    mask = torch.arange(N, device=dev)[None] <= (N - M + torch.arange(M, device=dev))[:, None]
    w = torch.softmax(s.masked_fill(~mask, float("-inf")), -1)
    want = (w.transpose(2, 3) @ g.double()).sum(1, keepdim=True)
    # each weight: its rounding, and the f32 scores' (D products of up to 1, an exponential)
    size = (w.transpose(2, 3) @ g.double().abs()).sum(1, keepdim=True)
    u = HALF_STEP["f16"]
    bound = u * want.abs() + (u + 2.0 ** -17) * size * (1 + u) + 2 * TINY["f16"]
    over = (dv.double() - want).abs() - bound
    assert float(over.max()) <= 0, float(over.max())


def test_a_part_of_the_batch_is_small(td):
    """Sequences whose gradients differ by 2^20 in size: each keeps its own digits."""
    torch, dev = td
    q, k, v, g = (normal(torch, (3, 2, 300, 64), "f16", 530 + i, dev) for i in range(4))
    g = g * torch.tensor([1.0, 2.0 ** -10, 2.0 ** 10], device=dev, dtype=g.dtype).view(3, 1, 1, 1)
    how = dict(window=100, n_sinks=2, scale=0.125)
    out, lse = vef.forward_window(q, k, v, return_lse=True, **how)
    whole = vef.backward_window(g, q, k, v, out, lse, **how)
    for b in range(3):
        x = [t[b:b + 1] for t in (g, q, k, v, out)]
        alone = vef.backward_window(*x, lse[b:b + 1].contiguous(), **how)
        assert all(torch.equal(y[b:b + 1], z) for y, z in zip(whole, alone))
    # a power of two on dout is one on the gradients, as far as f16 has it
    big = vef.backward_window(g[:1] * 16, *(t[:1] for t in (q, k, v, out)), lse[:1].contiguous(), **how)
    for y, z in zip(whole, big):
        far = y[:1].abs() >= 2.0 ** -13
        assert torch.equal(y[:1][far] * 16, z[far])


def test_no_number_among_the_rows(td):
    """A NaN in a row of dout reaches its own tiles alone; the others' power does
    not come from it."""
    torch, dev = td
    q, k, v, g = (normal(torch, (1, 1, 1024, 64), "f16", 540 + i, dev, s) for i, s in enumerate((1.0, 1.0, 1.0, 1e-3)))
    how = dict(window=64, scale=0.125)
    out, lse = vef.forward_window(q, k, v, return_lse=True, **how)
    want = vef.backward_window(g, q, k, v, out, lse, **how)
    g[0, 0, 500] = float("inf")
    got = vef.backward_window(g, q, k, v, out, lse, **how)
    for x, y in zip(got, want):
        assert torch.equal(x[:, :, :256], y[:, :, :256]) and torch.equal(x[:, :, 768:], y[:, :, 768:])


@pytest.mark.parametrize("call", ["window", "cached"])
@pytest.mark.parametrize("name", ["f16", "bf16"])
def test_many_small_weights_beside_a_large_one(td, name, call):
    """One key of weight 1 and 2^19 of 2^-23.4, which f16 does not have: together
    they are a twentieth of the result."""
    torch, dev = td
    N, D, score = 2 ** 19, 8, 16.22
    k = torch.zeros(1, 1, N, D, device=dev)
    k[:, :, 0] = 1.0
    v = 1.0 + 0.5 * torch.rand(1, 1, N, D, generator=torch.Generator(device=dev).manual_seed(5), device=dev)
    v[:, :, 0] = 0.25
    k, v = (t.to(torch.float16 if name == "f16" else torch.bfloat16) for t in (k, v))
    q = torch.ones(1, 1, 1, D, dtype=k.dtype, device=dev)
    scale = float(np.float32(score / D))
    if call == "window":
        out, lse = vef.forward_window(q, k, v, scale=scale, return_lse=True)
    else:  # so many sequences that none's keys are shared out
        B = 700
        lens = torch.full((B,), N, dtype=torch.int32, device=dev)
        out = vef.forward_cached(q.expand(B, 1, 1, D), k.expand(B, 1, N, D), v.expand(B, 1, N, D), lens, scale=scale)
        assert bool((out == out[:1]).all())
        out = out[:1]
    w = torch.full((N,), np.exp(-scale * D), dtype=torch.float64, device=dev)
    w[0] = 1.0
    want = (w[:, None] * v[0, 0].double()).sum(0) / w.sum()
    # each weight is rounded (u, and in f16 2^-32 of the largest), so is the result.  How many products
    # of a matrix instruction are added before a cut to f32 is not specified: each of the N additions
    # may be cut by 2^-23 of the sum (to 24 digits, downwards); those of the weights go 128 at a time
    u = HALF_STEP[name]
    bound = (2 * u + N * 2.0 ** -23 + N / 128 * 2.0 ** -24 + 2.0 ** -16) * want
    if name == "f16":
        bound = bound + 2.0 ** -32 * 1.5 * N
    assert bool(((out[0, 0, 0].double() - want).abs() <= bound).all()), (out[0, 0, 0], want, bound)
    if call == "window":
        assert abs(float(lse) - (scale * D + float(torch.log(w.sum())))) <= 2.0 ** -10


@pytest.mark.parametrize("call", ["window", "cached"])
def test_small_weights_add_up(td, call):
    """The same with sums that are exact: 2^16 keys, the large weight on a V of 0,
    the others on ones.  Held times 2^7 a weight is a multiple of 2^-24, and the
    sum of them, below 1, has 24 digits."""
    torch, dev = td
    N, D, score = 2 ** 16, 8, 16.22
    k = torch.zeros(1, 1, N, D, dtype=torch.float16, device=dev)
    v = torch.ones_like(k)
    k[:, :, 0], v[:, :, 0] = 1.0, 0.0
    q = torch.ones(1, 1, 1, D, dtype=k.dtype, device=dev)
    scale = float(np.float32(score / D))
    if call == "window":
        out = vef.forward_window(q, k, v, scale=scale)
    else:
        B = 700
        lens = torch.full((B,), N, dtype=torch.int32, device=dev)
        out = vef.forward_cached(q.expand(B, 1, 1, D), k.expand(B, 1, N, D), v.expand(B, 1, N, D), lens, scale=scale)
    w = (N - 1) * np.exp(-scale * D)
    want = w / (1 + w)
    # a weight is off by 2^-32, the result by u, the f32 score and exponential by 2^-16 (16 is held to
    # 2^-20, 2 D + 8 roundings), the sum of the weights, 128 at a time, by N / 128 2^-24
    bound = (HALF_STEP["f16"] + 2.0 ** -16 + N / 128 * 2.0 ** -24) * want + 2.0 ** -32 * N
    assert float((out.double() - want).abs().max()) <= bound, (out.flatten()[:2], want, bound)
