"""GPU tests of causal attention under a window with visible first keys, and
of its gradients, against the f64 oracle within counted bounds."""
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
    # type, (B, Hq, Hk, M, N, D), window, sinks, kv_len, q_start, layout
    ("f16", (1, 1, 1, 1, 1, 8), None, 0, None, None, "plain"),
    ("bf16", (1, 2, 2, 64, 64, 32), 32, 2, None, None, "plain"),
    ("f16", (2, 4, 2, 128, 128, 64), None, 0, None, None, "packed"),
    ("bf16", (1, 4, 1, 129, 129, 128), 1, 0, None, None, "plain"),       # a row sees itself alone
    ("f16", (1, 6, 2, 257, 257, 72), 100, 5, None, None, "padded"),
    ("bf16", (1, 3, 1, 300, 300, 96), 128, 130, None, None, "packed"),   # first keys past one tile
    ("f16", (2, 2, 1, 70, 300, 64), 90, 3, None, None, "plain"),         # queries end a longer sequence
    ("bf16", (2, 2, 2, 300, 70, 40), None, 0, None, None, "plain"),      # more queries than keys: first rows empty
    ("f16", (4, 4, 2, 200, 200, 64), 64, 1, [200, 131, 1, 0], [0, 0, 0, 0], "plain"),  # padded batch
    ("bf16", (3, 2, 1, 50, 400, 104), 70, 2, [400, 333, 20], None, "packed"),
    ("f16", (3, 5, 5, 190, 260, 56), None, 0, [260, 255, 129], [70, 100, -30], "padded"),
    ("bf16", (1, 8, 1, 640, 640, 64), 200, 4, None, None, "plain"),
    ("f16", (1, 2, 1, 1030, 1030, 128), 256, 1, None, None, "packed"),
    ("bf16", (1, 1, 1, 1500, 1500, 80), None, 0, None, None, "plain"),
    ("bf16", (1, 2, 2, 384, 384, 16), 128, 128, None, None, "plain"),    # every border on a tile's
    ("f16", (1, 2, 2, 140, 140, 24), 10 ** 12, 10 ** 12, None, None, "plain"),
    ("f16", (1, 7, 7, 150, 150, 120), 40, 0, None, None, "packed"),
    ("bf16", (2, 3, 3, 33, 500, 64), 16, 3, [500, 17], [480, -20], "plain"),
    ("f16", (1, 1, 1, 5, 0, 16), None, 0, None, None, "plain"),          # no keys at all
    ("f16", (2, 5, 1, 1111, 1111, 96), None, 0, [1111, 737], [0, 0], "plain"),  # key tiles cut into many chunks
    ("bf16", (1, 6, 2, 1300, 1300, 128), 300, 140, None, None, "packed"),       # chunks of the first keys' tiles
]


def build(td, case, seed):
    torch, dev = td
    name, (B, H, K, M, N, D), window, sinks, kv_len, q_start, layout = case
    x = [normal(torch, s, name, seed + i, dev) for i, s in enumerate(((B, H, M, D), (B, K, N, D), (B, K, N, D), (B, H, M, D)))]
    seen = np.stack([od.window_visible(M, N, window, sinks, None if kv_len is None else kv_len[b],
                                       None if q_start is None else q_start[b]) for b in range(B)])
    # what no row sees and what rows that see nothing hold does not matter
    gone_k, gone_q = ~seen.any(1), ~seen.any(2)
    if kv_len is not None:
        for b in range(B):
            gone = torch.from_numpy(np.flatnonzero(gone_k[b] & (np.arange(N) >= kv_len[b]))).to(dev)
            x[1][b][:, gone] = float("nan")
            x[2][b][:, gone] = float("inf")
            rows = torch.from_numpy(np.flatnonzero(gone_q[b])).to(dev)
            x[0][b][:, rows] = float("nan")
            x[3][b][:, rows] = float("-inf")
    x = [laid_out(torch, t, layout) if t.numel() else t for t in x]
    ints = lambda v: None if v is None else torch.tensor(v, dtype=torch.int32, device=dev)
    how = dict(window=window, n_sinks=sinks, scale=0.7 / D ** 0.5, kv_len=ints(kv_len), q_start=ints(q_start))
    return x, seen, how


@pytest.mark.parametrize("i", range(len(CASES)))
def test_forward_and_gradients(td, i):
    torch, dev = td
    name = CASES[i][0]
    u, tiny = HALF_STEP[name], TINY[name]
    (q, k, v, g), seen, how = build(td, CASES[i], 1000 + 10 * i)
    out, lse = vef.forward_window(q, k, v, return_lse=True, **how)
    want, wlse, weights, bound, score, lse_bound = od.attention(f64(q), f64(k), f64(v), seen, float(np.float32(how["scale"])), u)
    assert_within(out, want, bound, "out", tiny=2 * tiny)
    empty = np.isinf(wlse)
    got_lse = f64(lse)
    assert np.array_equal(np.isneginf(got_lse), empty)
    assert_within(np.where(empty, 0, got_lse), np.where(empty, 0, wlse), lse_bound, "lse")
    assert not f64(out)[empty].any()
    assert torch.equal(out, vef.forward_window(q, k, v, **how))

    grads = vef.backward_window(g, q, k, v, out, lse, **how)
    torch.cuda.synchronize(dev)
    assert vef.device_status() == 0
    wants, bounds = od.attention_backward(f64(g), f64(q), f64(k), f64(v), want, weights, seen,
                                          float(np.float32(how["scale"])), u, bound, score)
    # f16 weights below 2^-14 round by up to 2^-25: as many of them as rows or keys
    small = 0.0 if name != "f16" else 2.0 ** -24 * (max(seen.shape[1:]) + 1) * 8
    for got, w, b, what in zip(grads, wants, bounds, ("dq", "dk", "dv")):
        assert_within(got, w, b, what, tiny=2 * tiny + small)
    again = vef.backward_window(g, q, k, v, out, lse, **how)
    assert all(torch.equal(a, b) for a, b in zip(grads, again))


def test_gradients_against_differences(td):
    """Directional derivative in f16 of a small case, by forward calls."""
    torch, dev = td
    x = [normal(torch, s, "f16", 60 + i, dev) for i, s in enumerate(((1, 2, 40, 32), (1, 1, 40, 32), (1, 1, 40, 32), (1, 2, 40, 32)))]
    how = dict(window=9, n_sinks=2, scale=0.25)
    out, lse = vef.forward_window(*x[:3], return_lse=True, **how)
    grads = vef.backward_window(x[3], *x[:3], out, lse, **how)
    along = [torch.sign(t) for t in grads]  # every term adds up: the slope is the gradients' 1-norm
    step = 2.0 ** -4

    def loss(s):
        a = [(t.float() + s * d.float()).half() for t, d in zip(x[:3], along)]
        return float((vef.forward_window(*a, **how).double() * x[3].double()).sum())

    slope = (8 * (loss(step) - loss(-step)) - (loss(2 * step) - loss(-2 * step))) / (12 * step)
    want = sum(float(g.double().abs().sum()) for g in grads)
    # inputs and results are f16: each of the 2560 results is off by 2^-11 of
    # up to 4 times |g| ~ 0.8, and the moved inputs by 2^-11 of up to 4 each
    # against gradients whose 1-norm is `want`
    assert abs(slope - want) <= (2560 * 2.0 ** -11 * 2 + want * 2.0 ** -9) / step + 0.02 * want


def test_masked_infinities_do_not_reach_other_rows(td):
    """NaN and infinity in keys and values that a row does not see, inside a
    tile that it reads."""
    torch, dev = td
    for name in ("f16", "bf16"):
        for D in (64, 128):
            q, k, v = (normal(torch, (1, 2, 300, D), name, 70 + i, dev) for i in range(3))
            how = dict(window=50, n_sinks=2, scale=0.1)
            clean = vef.forward_window(q, k, v, **how)
            k[0, :, 140], v[0, :, 140] = float("nan"), float("inf")
            v[0, 1, 200, 3] = float("nan")
            out = vef.forward_window(q, k, v, **how)
            hit = torch.zeros(300, dtype=torch.bool, device=dev)
            hit[140:190] = True
            hit2 = hit.clone()
            hit2[200:250] = True
            for h, rows in ((0, hit), (1, hit2)):
                got, ref = f64(out[0, h, ~rows]), f64(clean[0, h, ~rows])
                assert np.all(np.isfinite(got))
                # the same sums, weights rounded to the type or not
                assert np.abs(got - ref).max() <= 4 * HALF_STEP[name] * 4
            assert bool(torch.isnan(out[0, 0, hit]).all())
            assert bool(torch.isnan(out[0, 1, 200:250, 3]).all())


def test_views_written_and_left_alone(td):
    """Results into parts of larger buffers; what lies around stays."""
    torch, dev = td
    q, k, v = (normal(torch, (2, 4, 90, 64), "bf16", 80 + i, dev) for i in range(3))
    how = dict(window=33, n_sinks=1, scale=0.1)
    want, lse = vef.forward_window(q, k, v, return_lse=True, **how)
    big = torch.full((2, 100, 6, 64), 5.0, dtype=q.dtype, device=dev)
    out = big[:, 4:94, 1:5].transpose(1, 2)
    assert vef.forward_window(q, k, v, out=out, **how) is out
    assert torch.equal(out, want)
    g = normal(torch, q.shape, "bf16", 90, dev)
    grads = vef.backward_window(g, q, k, v, want, lse, **how)
    packed = torch.full((2, 90, 14, 64), 5.0, dtype=q.dtype, device=dev)
    parts = [packed[:, :, a:a + 4].transpose(1, 2) for a in (0, 5, 10)]
    got = vef.backward_window(g, q, k, v, want, lse, dq=parts[0], dk=parts[1], dv=parts[2], **how)
    assert all(a is b for a, b in zip(got, parts)) and all(torch.equal(a, b) for a, b in zip(grads, got))
    rest = torch.ones(100, 6, dtype=torch.bool, device=dev)
    rest[4:94, 1:5] = False
    assert bool((big[:, rest] == 5).all()) and bool((packed[:, :, [4, 9]] == 5).all())


def test_shared_keys_of_a_broadcast(td):
    """Keys broadcast over the batch and the heads (strides of zero)."""
    torch, dev = td
    q = normal(torch, (3, 4, 150, 64), "f16", 100, dev)
    one = [normal(torch, (1, 1, 150, 64), "f16", 101 + i, dev) for i in range(2)]
    how = dict(window=60, n_sinks=1, scale=0.1)
    wide = [t.expand(3, 2, 150, 64) for t in one]
    full = [t.contiguous() for t in wide]
    out, lse = vef.forward_window(q, *wide, return_lse=True, **how)
    want, wlse = vef.forward_window(q, *full, return_lse=True, **how)
    assert torch.equal(out, want) and torch.equal(lse, wlse)
    a, b = (vef.backward_window(q, q, *kv, out, lse, **how) for kv in (wide, full))
    assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_first_keys_without_end(td):
    """Every key is a first key, and the window one key wide: as without a
    window, in a workspace of the size of the call's tensors, not of its
    tiles' product."""
    torch, dev = td
    x = [normal(torch, (1, 1, 24577, 128), "bf16", 105 + i, dev) for i in range(4)]
    out, lse = vef.forward_window(*x[:3], window=1, n_sinks=24577, scale=0.1, return_lse=True)
    wout, wlse = vef.forward_window(*x[:3], scale=0.1, return_lse=True)
    assert torch.equal(out, wout) and torch.equal(lse, wlse)
    torch.cuda.synchronize(dev)
    free = torch.cuda.mem_get_info(dev)[0]
    got = vef.backward_window(x[3], *x[:3], out, lse, window=1, n_sinks=24577, scale=0.1)
    torch.cuda.synchronize(dev)
    # 192 key tiles in up to seven pieces of 128 KiB, and the results
    assert free - torch.cuda.mem_get_info(dev)[0] < 2 ** 28
    want = vef.backward_window(x[3], *x[:3], out, lse, scale=0.1)
    for a, b in zip(got, want):  # the same products, cut into other chunks: rounded once from sums in f32
        assert torch.allclose(a.float(), b.float(), rtol=2 ** -7, atol=2 ** -7 * float(b.float().abs().max()))


def test_streams_and_graphs(td):
    torch, dev = td
    x = [normal(torch, (2, 4, 260, 64), "bf16", 110 + i, dev) for i in range(4)]
    lens = torch.tensor([260, 200], dtype=torch.int32, device=dev)
    start = torch.zeros(2, dtype=torch.int32, device=dev)
    how = dict(window=100, n_sinks=2, scale=0.125, kv_len=lens, q_start=start)

    def run(stream=None):
        out, lse = vef.forward_window(*x[:3], return_lse=True, stream=stream, **how)
        return (out, lse) + vef.backward_window(x[3], *x[:3], out, lse, stream=stream, **how)

    want = run()
    streams = [torch.cuda.Stream(dev) for _ in range(3)]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream(dev))
    got = [run(s) for s in streams]  # at once: no workspace is shared
    torch.cuda.synchronize(dev)
    for r in got:
        assert all(torch.equal(a, b) for a, b in zip(r, want))
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = run()
        graphs.append((g, out))
    for i, t in enumerate(x):
        t.copy_(normal(torch, t.shape, "bf16", 120 + i, dev))
    lens.copy_(torch.tensor([111, 260], dtype=torch.int32))
    for (g, _), s in zip(graphs, streams):  # both graphs at once, on two streams
        s.wait_stream(torch.cuda.current_stream(dev))
        with torch.cuda.stream(s):
            g.replay()
    torch.cuda.synchronize(dev)
    want = run()
    torch.cuda.synchronize(dev)
    for _, out in graphs:
        assert all(torch.equal(a, b) for a, b in zip(out, want))
    assert vef.device_status() == 0


@pytest.mark.parametrize("dim", [64, 80, 96, 128])
def test_short_walks_do_not_race(td, dim):
    """Key tiles cut down to single items, then query tiles, by the same
    blocks: twelve calls, all alike."""
    torch, dev = td
    x = [normal(torch, s, "f16", 140 + i, dev) for i, s in enumerate(((2, 5, 1111, dim), (2, 1, 1111, dim), (2, 1, 1111, dim), (2, 5, 1111, dim)))]
    out, lse = vef.forward_window(*x[:3], return_lse=True, scale=dim ** -0.5)
    first = vef.backward_window(x[3], *x[:3], out, lse, scale=dim ** -0.5)
    for _ in range(11):
        again = vef.backward_window(x[3], *x[:3], out, lse, scale=dim ** -0.5)
        assert all(torch.equal(a, b) for a, b in zip(first, again))
    # against the formula in f32: P and D are rounded by 2^-11 (dq, dk, dv are
    # sums of about 500 of them, of random sign), the results once more
    s = [t.float() for t in x]
    k, v = (t.expand(2, 5, 1111, dim) for t in s[1:3])
    mask = torch.ones(1111, 1111, dtype=torch.bool, device=dev).tril()
    w = torch.softmax((s[0] @ k.transpose(2, 3) * dim ** -0.5).masked_fill(~mask, float("-inf")), -1)
    ds = w * (s[3] @ v.transpose(2, 3) - (s[3] * (w @ v)).sum(-1, keepdim=True)) * dim ** -0.5
    wants = (ds @ k, (ds.transpose(2, 3) @ s[0]).sum(1, keepdim=True), (w.transpose(2, 3) @ s[3]).sum(1, keepdim=True))
    for got, want in zip(first, wants):
        assert float((got.float() - want).norm() / want.norm()) <= 2.0 ** -9


def test_lengths_outside_the_buffer_are_held(td):
    torch, dev = td
    q, k, v = (normal(torch, (3, 2, 40, 32), "f16", 130 + i, dev) for i in range(3))
    ints = lambda *a: torch.tensor(a, dtype=torch.int32, device=dev)
    got = vef.forward_window(q, k, v, kv_len=ints(2 ** 31 - 1, -5, 40), q_start=ints(0, 0, 2 ** 31 - 1))
    want = vef.forward_window(q, k, v, kv_len=ints(40, 0, 0), q_start=ints(0, 0, 0))
    assert torch.equal(got, want) and not f64(got[1:]).any()


def test_no_query_heads_and_no_keys(td):
    """Key heads without query heads (their gradients are zeros; there is no
    row of out and lse to read), and query rows without keys."""
    torch, dev = td
    k = normal(torch, (2, 2, 300, 64), "bf16", 160, dev)
    q = k.new_empty(2, 0, 200, 64)
    out, lse = vef.forward_window(q, k, k, return_lse=True)
    dq, dk, dv = vef.backward_window(q, q, k, k, out, lse, dk=torch.full_like(k, 7.0), dv=torch.full_like(k, 7.0))
    assert out.shape == dq.shape == q.shape and lse.shape == (2, 0, 200)
    assert not dk.any() and not dv.any()
    none = k[:, :, :0]
    out, lse = vef.forward_window(k, none, none, return_lse=True)
    assert not out.any() and bool(torch.isneginf(lse).all())
    dq, dk, dv = vef.backward_window(k, k, none, none, out, lse)
    assert not dq.any() and dk.shape == dv.shape == none.shape
    assert vef.device_status() == 0


@pytest.mark.parametrize("bad", [dict(window=0), dict(scale=0.0), dict(n_sinks=-1)])
def test_refusals(td, bad):
    torch, dev = td
    q = normal(torch, (1, 2, 8, 16), "f16", 1, dev)
    with pytest.raises((ValueError, vef.VattnError)):
        vef.forward_window(q, q, q, **bad)


def test_refused_tensors(td):
    torch, dev = td
    q = normal(torch, (1, 2, 8, 16), "f16", 1, dev)
    with pytest.raises(vef.VattnError):
        vef.forward_window(q, q, q, out=q)
    with pytest.raises(vef.VattnError):
        vef.forward_window(q[..., :12], q[..., :12], q[..., :12])
    with pytest.raises(ValueError):
        vef.forward_window(q.transpose(2, 3), q, q)
    with pytest.raises(ValueError):
        vef.forward_window(q, q, q[:, :1])
    with pytest.raises(TypeError):
        vef.forward_window(q, q.bfloat16(), q)
    with pytest.raises(TypeError):
        vef.forward_window(q, q, q, kv_len=torch.ones(1, dtype=torch.int64, device=dev))
    with pytest.raises(ValueError):
        vef.forward_window(q, q, q, kv_len=torch.ones(2, dtype=torch.int32, device=dev))
