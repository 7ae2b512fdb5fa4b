"""GPU tests of the attention of new tokens over a cache against the f64
oracle within counted bounds."""
import numpy as np
import pytest

from oracle import decoder as od
import vision_encoder_flash_gb300 as vef
from decoder_util import HALF_STEP, TINY, assert_within, f64, laid_out, normal

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


def tree_words(T, rng):
    bits = [1]
    for t in range(1, T):
        bits.append(bits[int(rng.integers(0, t))] | 1 << t)
    return bits


CASES = [
    # type, (B, Hq, Hk, T, N, D), kv_len, window, sinks, tree, layout
    ("bf16", (1, 1, 1, 1, 1, 8), [1], None, 0, False, "plain"),
    ("f16", (3, 4, 2, 1, 200, 64), [200, 77, 1], None, 0, False, "plain"),
    ("bf16", (2, 8, 1, 1, 1500, 128), [1500, 640], None, 0, False, "packed"),
    ("f16", (2, 32, 8, 1, 700, 64), [700, 65], 128, 4, False, "plain"),
    ("bf16", (2, 6, 2, 2, 300, 72), [300, 64], None, 0, False, "padded"),
    ("f16", (2, 4, 4, 5, 400, 40), [390, 5], 30, 70, False, "plain"),
    ("bf16", (3, 4, 1, 7, 300, 96), [300, 3, 0], None, 0, False, "plain"),        # fewer rows in use than new tokens
    ("f16", (2, 4, 2, 31, 500, 64), [500, 131], None, 0, True, "plain"),
    ("bf16", (2, 8, 2, 64, 300, 128), [300, 64], 40, 3, True, "packed"),
    ("f16", (2, 3, 1, 64, 200, 32), [200, 30], 7, 2, True, "plain"),              # a window inside the tree
    ("bf16", (1, 5, 1, 13, 4000, 64), [3777], 1000, 4, True, "plain"),
    ("f16", (1, 16, 1, 17, 260, 104), [260], None, 0, True, "padded"),
    ("bf16", (40, 4, 4, 1, 130, 64), [130 - 3 * b for b in range(40)], None, 0, False, "plain"),
    ("f16", (1, 2, 2, 1, 9000, 64), [9000], None, 0, False, "plain"),             # one long sequence
    ("bf16", (1, 128, 2, 3, 90, 16), [90], 20, 0, True, "plain"),                 # 192 rows a key head
    ("f16", (2, 2, 1, 3, 0, 16), [0, 0], None, 0, False, "plain"),                # no cache at all
]


def build(td, case, seed):
    torch, dev = td
    name, (B, H, K, T, N, D), lens, window, sinks, tree, layout = case
    rng = np.random.default_rng(seed)
    q, k, v = (normal(torch, s, name, seed + i, dev) for i, s in enumerate(((B, H, T, D), (B, K, N, D), (B, K, N, D))))
    words = [tree_words(T, rng) for _ in range(B)] if tree else None
    seen = np.stack([od.cached_visible(T, N, window, sinks, lens[b], words[b] if tree else None) for b in range(B)])
    for b in range(B):  # rows that are seen by none: unused, or before the window
        gone = torch.from_numpy(np.flatnonzero(~seen[b].any(0))).to(dev)
        k[b][:, gone], v[b][:, gone] = float("nan"), float("inf")
    q, k, v = (laid_out(torch, t, layout) if t.numel() else t for t in (q, k, v))
    mask = None
    if tree:
        mask = torch.tensor([[w - (1 << 64) if w >> 63 else w for w in ws] for ws in words], dtype=torch.int64, device=dev)
    return (q, k, v, torch.tensor(lens, dtype=torch.int32, device=dev)), seen, dict(
        tree_mask=mask, window=window, n_sinks=sinks, scale=1.3 / D ** 0.5)


@pytest.mark.parametrize("i", range(len(CASES)))
def test_against_the_oracle(td, i):
    torch, dev = td
    name = CASES[i][0]
    x, seen, how = build(td, CASES[i], 2000 + 10 * i)
    out = vef.forward_cached(*x, **how)
    want, _, _, bound, _, _ = od.attention(*(f64(t) for t in x[:3]), seen, float(np.float32(how["scale"])), HALF_STEP[name])
    assert_within(out, want, bound, "out", tiny=2 * TINY[name])
    assert torch.equal(out, vef.forward_cached(*x, **how))


@pytest.mark.parametrize("D", [8, 24, 32, 40, 64, 72, 120, 128])
@pytest.mark.parametrize("H,T", [(1, 1), (4, 4), (5, 5), (8, 4), (11, 3), (7, 11)])
def test_rows_and_widths(td, H, T, D):
    """Rows for one, two and four groups of warps, of every width of a shared
    row, in two layouts, one a tree under a window."""
    for i, (window, tree, layout) in enumerate(((None, False, "packed"), (50, True, "padded"))):
        case = ("f16" if i else "bf16", (2, 2 * H, 2, T, 333, D), [333, 70], window, 2 * i, tree, layout)
        x, seen, how = build(td, case, 700 + D + H)
        out = vef.forward_cached(*x, **how)
        want, _, _, bound, _, _ = od.attention(*(f64(t) for t in x[:3]), seen, float(np.float32(how["scale"])),
                                               HALF_STEP[case[0]])
        assert_within(out, want, bound, "out", tiny=2 * TINY[case[0]])


@pytest.mark.parametrize("N", [150, 260, 390, 510])
def test_few_shares(td, N):
    """Two to four shares of the keys, some of them without a key in short
    sequences: against the oracle, on three streams at once, and replayed with
    other lengths."""
    torch, dev = td
    case = ("f16", (5, 8, 2, 3, N, 72), [N, 129, 40, 3, 0], None, 2, True, "plain")
    x, seen, how = build(td, case, 900 + N)
    out = vef.forward_cached(*x, **how)
    want, _, _, bound, _, _ = od.attention(*(f64(t) for t in x[:3]), seen, float(np.float32(how["scale"])), HALF_STEP["f16"])
    assert_within(out, want, bound, "out", tiny=2 * TINY["f16"])
    streams = [torch.cuda.Stream(dev) for _ in range(3)]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream(dev))
    got = [vef.forward_cached(*x, stream=s, **how) for s in streams]
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize(dev)
    assert all(torch.equal(t, out) for t in got)
    with torch.cuda.graph(graph):
        again = vef.forward_cached(*x, **how)
    for t in x[1:3]:
        t.copy_(normal(torch, t.shape, "f16", 950, dev))
    x[3].copy_(torch.tensor([0, N, 3, 131, 64], dtype=torch.int32))
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize(dev)
    assert torch.equal(again, vef.forward_cached(*x, **how))


def test_words_without_bits_and_stray_bits(td):
    torch, dev = td
    q, k, v = (normal(torch, s, "bf16", 5 + i, dev) for i, s in enumerate(((1, 2, 4, 32), (1, 1, 50, 32), (1, 1, 50, 32))))
    lens = torch.tensor([40], dtype=torch.int32, device=dev)
    words = [1, 0, 0b101, 0b1000]  # the second token sees nothing, the last only itself and the cache
    mask = torch.tensor([words], dtype=torch.int64, device=dev)
    out = vef.forward_cached(q, k, v, lens, tree_mask=mask)
    seen = od.cached_visible(4, 50, None, 0, 40, words)[None]
    want, _, _, bound, _, _ = od.attention(f64(q), f64(k), f64(v), seen, 1.0, HALF_STEP["bf16"])
    assert_within(out, want, bound, "out", tiny=2 * TINY["bf16"])
    assert not f64(out[0, :, 1]).any()
    stray = mask | (1 << 40) | -(1 << 63)
    stray[0, 1] = 0
    assert torch.equal(out, vef.forward_cached(q, k, v, lens, tree_mask=stray))


def test_special_values_in_branches(td):
    """A drafted token's NaN stays on its branch."""
    torch, dev = td
    q, k, v = (normal(torch, s, "f16", 15 + i, dev) for i, s in enumerate(((1, 4, 3, 64), (1, 2, 100, 64), (1, 2, 100, 64))))
    lens = torch.tensor([90], dtype=torch.int32, device=dev)
    mask = torch.tensor([[0b001, 0b011, 0b101]], dtype=torch.int64, device=dev)
    clean = vef.forward_cached(q, k, v, lens, tree_mask=mask)
    most = float(v.abs().max())
    k[0, :, 88], v[0, :, 88] = float("nan"), float("nan")  # new token 1
    out = vef.forward_cached(q, k, v, lens, tree_mask=mask)
    # a tile with a NaN takes its weights unrounded, others round them by up
    # to u = 2^-11 each, and both round the result by u: each is within u |out|
    # + (u + 2^-13 for the f32 sums) sum(p |v|) <= (2 u + 2^-13) max |v| of the
    # formula, so they are within twice that of each other
    diff = np.abs(f64(out[:, :, [0, 2]]) - f64(clean[:, :, [0, 2]]))
    assert diff.max() <= 2 * (2 * HALF_STEP["f16"] + 2.0 ** -13) * most
    assert bool(torch.isnan(out[:, :, 1]).all())


def test_a_chain_is_the_window_call(td):
    torch, dev = td
    for T in (1, 6, 64):
        q, k, v = (normal(torch, s, "bf16", 25 + i, dev) for i, s in enumerate(((2, 4, T, 64), (2, 2, 333, 64), (2, 2, 333, 64))))
        lens = torch.tensor([333, 200], dtype=torch.int32, device=dev)
        how = dict(window=70, n_sinks=2, scale=0.125)
        a = f64(vef.forward_cached(q, k, v, lens, **how))
        b = f64(vef.forward_window(q, k, v, kv_len=lens, **how))
        # two roundings of the weights and of the result each, |v| <= 5
        assert np.abs(a - b).max() <= 4 * HALF_STEP["bf16"] * 5


def test_streams_graphs_and_views(td):
    torch, dev = td
    q, k, v = (normal(torch, s, "bf16", 35 + i, dev) for i, s in enumerate(((2, 8, 1, 128), (2, 2, 3000, 128), (2, 2, 3000, 128))))
    lens = torch.tensor([2500, 900], dtype=torch.int32, device=dev)
    run = lambda **kw: vef.forward_cached(q, k, v, lens, scale=0.1, **kw)
    want = run()
    streams = [torch.cuda.Stream(dev) for _ in range(3)]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream(dev))
    got = [run(stream=s) for s in streams]
    torch.cuda.synchronize(dev)
    assert all(torch.equal(t, want) for t in got)
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = run()
        graphs.append((g, out))
    lens.copy_(torch.tensor([2999, 1], dtype=torch.int32))
    for (g, _), s in zip(graphs, streams):
        s.wait_stream(torch.cuda.current_stream(dev))
        with torch.cuda.stream(s):
            g.replay()
    torch.cuda.synchronize(dev)
    want = run()
    assert all(torch.equal(out, want) for _, out in graphs)
    big = torch.full((2, 1, 10, 128), 3.0, dtype=q.dtype, device=dev)
    run(out=big[:, :, 1:9].transpose(1, 2))
    assert torch.equal(big[:, :, 1:9].transpose(1, 2), want) and bool((big[:, :, [0, 9]] == 3).all())


def test_broadcast_rows(td):
    """A cache whose rows, heads or sequences are one (strides of zero)."""
    torch, dev = td
    q = normal(torch, (2, 4, 3, 64), "f16", 150, dev)
    lens = torch.tensor([70, 12], dtype=torch.int32, device=dev)
    for shape in ((2, 2, 1, 64), (1, 1, 70, 64), (1, 1, 1, 64)):
        wide = [normal(torch, shape, "f16", 151 + i, dev).expand(2, 2, 70, 64) for i in range(2)]
        got = vef.forward_cached(q, *wide, lens, scale=0.125)
        assert torch.equal(got, vef.forward_cached(q, *[t.contiguous() for t in wide], lens, scale=0.125))


def test_refusals(td):
    torch, dev = td
    q, k = (normal(torch, s, "f16", 1, dev) for s in ((1, 2, 65, 16), (1, 2, 100, 16)))
    lens = torch.tensor([100], dtype=torch.int32, device=dev)
    with pytest.raises(vef.VattnError):
        vef.forward_cached(q, k, k, lens)  # 65 new tokens
    q = q[:, :, :4]
    with pytest.raises(TypeError):
        vef.forward_cached(q, k, k, None)
    with pytest.raises(TypeError):
        vef.forward_cached(q, k, k, lens, tree_mask=torch.ones(1, 4, dtype=torch.int32, device=dev))
    with pytest.raises(ValueError):
        vef.forward_cached(q, k, k, lens, tree_mask=torch.ones(1, 5, dtype=torch.int64, device=dev))
    with pytest.raises(vef.VattnError):
        vef.forward_cached(q, k, k, lens, out=k[:, :, :4])
