"""GPU tests of the q/k norm with rotation and its gradient against the f64
oracle (oracle/decoder.py), within bounds counted from the roundings."""
import numpy as np
import pytest

from oracle import decoder as od
import vision_encoder_flash_gb300 as vef
from decoder_util import HALF_STEP, TINY, assert_within, dtype, f64, laid_out, normal

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def td():
    import torch
    if not torch.cuda.is_available():
        raise RuntimeError("GPU tests need a CUDA device")
    from vision_encoder_flash_gb300 import build
    build.build()
    vef.load_library()
    return torch, torch.device("cuda", 0)


CASES = [
    # type, (B, Hq, Hk, N, D), rope_dims, layout, weights, positions
    ("bf16", (1, 2, 1, 1, 64), 64, "plain", "f32", None),
    ("bf16", (2, 5, 1, 37, 128), 128, "packed", "f32", "random"),
    ("f16", (2, 4, 2, 19, 72), 72, "plain", "same", "random"),     # 8-byte vectors
    ("f16", (1, 3, 3, 33, 80), 48, "padded", "f32", None),         # part of the head turns
    ("f32", (2, 3, 1, 21, 64), 64, "packed", "f32", "far"),
    ("f32", (1, 4, 4, 9, 72), 40, "padded", None, "random"),
    ("bf16", (1, 2, 2, 7, 8), 8, "plain", None, None),
    ("bf16", (3, 2, 1, 5, 127), 127, "plain", "same", "far"),      # odd: one element at a time
    ("f32", (1, 1, 1, 6, 1), 1, "plain", "f32", None),             # nothing to turn
    ("f16", (1, 2, 1, 6, 7), 5, "plain", "f32", "negative"),
    ("f32", (1, 2, 1, 6, 128), 0, "plain", "f32", None),
    ("bf16", (1, 33, 9, 3, 32), 32, "packed", "f32", None),        # heads over several slices
    ("bf16", (2, 16, 4, 1500, 64), 64, "packed", "same", "random"),  # many blocks
]


def build(td, case, seed):
    torch, dev = td
    name, (B, H, K, N, D), rope, layout, wtype, where = case
    q = laid_out(torch, normal(torch, (B, H, N, D), name, seed, dev, 3.0), layout)
    k = laid_out(torch, normal(torch, (B, K, N, D), name, seed + 1, dev, 0.2), layout)
    w = [None, None]
    if wtype:
        wt = "f32" if wtype == "f32" else name
        w = [normal(torch, (D,), wt, seed + 2 + i, dev) for i in range(2)]
    rng = np.random.default_rng(seed + 9)
    how, pos = {}, np.arange(N)[None].repeat(B, 0)
    if where is None:
        how["pos0"] = 11
        pos = pos + 11
    else:
        low, high = {"random": (0, 4000), "far": (2 ** 31 - 5000, 2 ** 31 - 1), "negative": (-300, 0)}[where]
        pos = rng.integers(low, high, (B, N))
        how["positions"] = torch.from_numpy(pos.astype(np.int32)).to(dev)
    factors = rng.uniform(0.5, 4.0, max(1, rope // 2)).astype(np.float32) if seed % 2 else None
    if factors is not None:
        how["factors"] = torch.from_numpy(factors).to(dev)
    how.update(rope_dims=rope, base=10000.0 if seed % 3 else 500.0, eps=1e-5)
    return q, k, w, pos, factors, how


@pytest.mark.parametrize("i", range(len(CASES)))
def test_forward(td, i):
    torch, dev = td
    name, (_, _, _, _, D), rope, *_ = CASES[i]
    q, k, w, pos, factors, how = build(td, CASES[i], 100 + i)
    got = vef.qk_norm_rope(q, k, w[0], w[1], **how)
    for x, weight, y, what in ((q, w[0], got[0], "q"), (k, w[1], got[1], "k")):
        want, bound = od.qk_norm_rope(f64(x), None if weight is None else f64(weight), pos, rope, how["base"], factors,
                                      float(np.float32(how["eps"])))
        assert y.is_contiguous() and y.dtype == x.dtype
        assert_within(y, want, bound, what, HALF_STEP[name], TINY[name])


@pytest.mark.parametrize("name,D", [("f16", 24), ("bf16", 48), ("f32", 24), ("f32", 40), ("f16", 80), ("f32", 48),
                                    ("bf16", 96), ("f32", 72), ("f16", 72), ("f32", 80), ("f32", 56)])
def test_lanes_without_a_power_of_two(td, name, D):
    """Rows of 3, 5, 6, 9, 10 and (no gain, padded to 8) 7 vectors, several in
    a warp: against the oracle, and in place."""
    case = (name, (2, 5, 3, 70, D), D, "packed", "f32", "random")
    q, k, w, pos, factors, how = build(td, case, 500 + D)
    got = vef.qk_norm_rope(q, k, w[0], w[1], **how)
    for x, weight, y, what in ((q, w[0], got[0], "q"), (k, w[1], got[1], "k")):
        want, bound = od.qk_norm_rope(f64(x), f64(weight), pos, D, how["base"], factors, float(np.float32(how["eps"])))
        assert_within(y, want, bound, what, HALF_STEP[name], TINY[name])
    vef.qk_norm_rope(q, k, w[0], w[1], q_out=q, k_out=k, **how)
    assert td[0].equal(q, got[0]) and td[0].equal(k, got[1])


@pytest.mark.parametrize("i", range(len(CASES)))
def test_backward(td, i):
    torch, dev = td
    name, shape, rope, layout, *_ = CASES[i]
    q, k, w, pos, factors, how = build(td, CASES[i], 200 + i)
    gq = laid_out(torch, normal(torch, q.shape, name, 300 + i, dev), layout)
    gk = laid_out(torch, normal(torch, k.shape, name, 400 + i, dev), "plain")
    got = vef.qk_norm_rope_backward(gq, gk, q, k, w[0], w[1], **how)
    again = vef.qk_norm_rope_backward(gq, gk, q, k, w[0], w[1], **how)
    for n, (x, g, weight, what) in enumerate(((q, gq, w[0], "q"), (k, gk, w[1], "k"))):
        dx, dw, bx, bw = od.qk_norm_rope_backward(f64(g), f64(x), None if weight is None else f64(weight), pos, rope,
                                                  how["base"], factors, float(np.float32(how["eps"])))
        assert_within(got[n], dx, bx, "d" + what, HALF_STEP[name], TINY[name])
        if weight is None:
            assert got[2 + n] is None
        else:
            assert got[2 + n].dtype == torch.float32
            assert_within(got[2 + n], dw, bw, "dw of " + what, HALF_STEP["f32"])
            assert torch.equal(got[2 + n], again[2 + n])


def test_backward_against_differences(td):
    """The f32 gradient's directional derivative, from forward calls."""
    torch, dev = td
    q, k, w, pos, factors, how = build(td, ("f32", (1, 2, 1, 4, 24), 16, "plain", "f32", "random"), 501)
    gq, gk = normal(torch, q.shape, "f32", 1, dev), normal(torch, k.shape, "f32", 2, dev)
    dq, dk, dwq, dwk = vef.qk_norm_rope_backward(gq, gk, q, k, w[0], w[1], **how)
    along = [normal(torch, x.shape, "f32", 7 + i, dev) for i, x in enumerate((q, k, *w))]

    def loss(step):
        a = [x + step * d for x, d in zip((q, k, *w), along)]
        oq, ok = vef.qk_norm_rope(*a, **how)
        return float((oq.double() * gq.double()).sum() + (ok.double() * gk.double()).sum())

    h = 2.0 ** -6
    slope = (8 * (loss(h) - loss(-h)) - (loss(2 * h) - loss(-2 * h))) / (12 * h)  # error of order h^4
    want = sum(float((d.double() * g.double()).sum()) for d, g in zip(along, (dq, dk, dwq, dwk)))
    # 288 terms of size < 50, each an f32 result good to 2^-18: 0.06 in the
    # sums, over h; the fourth-order term is below that
    assert abs(slope - want) <= 2e-3 * max(1.0, abs(want)) + 288 * 2.0 ** -22 / h


@pytest.mark.parametrize("name", ["bf16", "f32"])
def test_in_place_and_into_a_cache(td, name):
    """Results over the inputs, over a packed buffer, and as rows of a cache;
    what lies around them stays."""
    torch, dev = td
    B, H, K, N, D = 2, 4, 2, 9, 64
    packed = normal(torch, (B, N, H + 2 * K, D), name, 5, dev)
    q, k = packed[:, :, :H].transpose(1, 2), packed[:, :, H:H + K].transpose(1, 2)
    oq, ok = vef.qk_norm_rope(q, k, pos0=3)
    cache = torch.full((B, K, 32, D), 7.0, dtype=packed.dtype, device=dev)
    _, same = vef.qk_norm_rope(q, k, pos0=3, k_out=cache[:, :, 10:10 + N])
    assert torch.equal(cache[:, :, 10:10 + N], ok) and same.data_ptr() == cache[:, :, 10:].data_ptr()
    assert bool((cache[:, :, :10] == 7).all()) and bool((cache[:, :, 10 + N:] == 7).all())
    values = packed[:, :, H + K:].clone()
    g = normal(torch, packed.shape, name, 6, dev)
    gq, gk = g[:, :, :H].transpose(1, 2), g[:, :, H:H + K].transpose(1, 2)
    dq, dk, *_ = vef.qk_norm_rope_backward(gq, gk, q, k, pos0=3)
    keep = g[:, :, H + K:].clone()
    vef.qk_norm_rope_backward(gq, gk, q, k, pos0=3, dq=gq, dk=gk)
    assert torch.equal(gq, dq) and torch.equal(gk, dk) and torch.equal(g[:, :, H + K:], keep)
    vef.qk_norm_rope(q, k, pos0=3, q_out=q, k_out=k)
    assert torch.equal(q, oq) and torch.equal(k, ok) and torch.equal(packed[:, :, H + K:], values)
    with pytest.raises(vef.VattnError):
        vef.qk_norm_rope(q, k, q_out=packed[:, :, 1:H + 1].transpose(1, 2))
    with pytest.raises(vef.VattnError):
        vef.qk_norm_rope(oq, ok, q_out=oq[:, :1].expand(B, H, N, D))


def test_broadcast_rows_and_special_values(td):
    torch, dev = td
    one = normal(torch, (1, 1, 4, 32), "bf16", 8, dev)
    q = one.expand(3, 6, 4, 32)
    oq, ok = vef.qk_norm_rope(q, one.expand(3, 1, 4, 32))
    assert torch.equal(oq, oq[:1, :1].expand(3, 6, 4, 32)) and torch.equal(ok, oq[:, :1])
    x = torch.zeros(1, 1, 3, 32, device=dev)
    x[0, 0, 1, 5] = float("nan")
    x[0, 0, 2] = 1e18  # squares stay in range
    y, _ = vef.qk_norm_rope(x, x)
    assert bool((y[0, 0, 0] == 0).all()) and bool(torch.isnan(y[0, 0, 1]).all())
    assert bool(torch.isfinite(y[0, 0, 2]).all())


def test_empty_and_streams(td):
    torch, dev = td
    z = torch.zeros(2, 0, 5, 16, device=dev)
    k = normal(torch, (2, 3, 5, 16), "f32", 1, dev)
    oq, ok = vef.qk_norm_rope(z, k)
    assert oq.shape == z.shape and torch.equal(ok, vef.qk_norm_rope(k, k)[0])
    w = torch.ones(16, device=dev)
    none = torch.zeros(0, 3, 5, 16, device=dev)
    dq, dk, dwq, dwk = vef.qk_norm_rope_backward(none, none, none, none, w, w)
    assert bool((dwq == 0).all()) and bool((dwk == 0).all()) and dq.shape == none.shape
    s = torch.cuda.Stream(dev)
    s.wait_stream(torch.cuda.current_stream(dev))
    a = vef.qk_norm_rope(k, k, w, w, stream=s)[0]
    b = vef.qk_norm_rope_backward(k, k, k, k, w, w, stream=s)
    s.synchronize()
    assert torch.equal(a, vef.qk_norm_rope(k, k, w, w)[0])
    assert all(torch.equal(x, y) for x, y in zip(b, vef.qk_norm_rope_backward(k, k, k, k, w, w)))


def test_graph_replay(td):
    """Two captured graphs with weight gradients, replayed with new values."""
    torch, dev = td
    x = [normal(torch, (2, 4, 65, 64), "bf16", 20 + i, dev) for i in range(4)]
    w = normal(torch, (64,), "f32", 30, dev)
    run = lambda: vef.qk_norm_rope(x[0], x[1], w, w) + vef.qk_norm_rope_backward(*x, w, w)
    run()
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = run()
        graphs.append((g, out))
    for i, t in enumerate(x):
        t.copy_(normal(torch, t.shape, "bf16", 40 + i, dev))
    for g, _ in graphs:
        g.replay()
    want = run()
    torch.cuda.synchronize(dev)
    for _, out in graphs:
        assert all(torch.equal(a, b) for a, b in zip(out, want))
