"""GPU tests of causal attention over packed prompts: against the f64 oracle
within counted bounds, and bit for bit against the same prompts alone."""
import numpy as np
import pytest

from oracle import decoder as od
import vision_encoder_flash_gb300 as vef
from decoder_util import HALF_STEP, TINY, assert_within, f64, laid_out, normal
from serving_util import ints

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


def rows(td, name, heads, total, D, seed, layout="plain"):
    torch, dev = td
    H, K = heads
    return [laid_out(torch, normal(torch, (1, h, total, D), name, seed + i, dev), layout) for i, h in enumerate((H, K, K))]


def starts(torch, lens, dev, first=0):
    return ints(torch, (first + np.concatenate([[0], np.cumsum(lens)])).tolist(), dev)


CASES = [
    # type, (Hq, Hk), D, lengths, window, sinks, layout
    ("bf16", (1, 1), 8, [1], None, 0, "plain"),
    ("f16", (2, 2), 32, [14, 1, 40, 0, 128, 127], None, 0, "packed"),
    ("bf16", (4, 2), 64, [129, 300, 2, 256, 31], None, 0, "packed"),
    ("f16", (6, 2), 72, [500, 33, 131], None, 0, "padded"),              # three heads a key head
    ("bf16", (5, 1), 128, [257, 64, 385], 100, 3, "packed"),
    ("f16", (3, 3), 96, [700, 90], 130, 200, "plain"),                    # first keys beyond a tile
    ("bf16", (16, 4), 40, [1] * 60 + [200], None, 0, "packed"),
    ("f16", (8, 1), 128, [1100], 1, 0, "plain"),                          # each row itself
    ("bf16", (2, 1), 104, [0, 0, 640, 0], 64, 1, "padded"),
]


@pytest.mark.parametrize("i", range(len(CASES)))
def test_against_the_oracle(td, i):
    torch, dev = td
    name, heads, D, lens, window, sinks, layout = CASES[i]
    total = sum(lens)
    q, k, v = rows(td, name, heads, total, D, 4000 + 10 * i, layout)
    cu = starts(torch, lens, dev)
    scale = 1.2 / D ** 0.5
    out, lse = vef.forward_packed(q, k, v, cu, window=window, n_sinks=sinks, scale=scale, return_lse=True)
    at = 0
    for b, n in enumerate(lens):
        part = [f64(x)[:, :, at:at + n] for x in (q, k, v)]
        seen = od.window_visible(n, n, window, sinks, n, 0)[None]
        want, want_lse, _, bound, _, lse_bound = od.attention(*part, seen, float(np.float32(scale)), HALF_STEP[name])
        assert_within(out[:, :, at:at + n], want, bound, f"out {b}", tiny=2 * TINY[name])
        assert np.all(np.abs(f64(lse)[:, :, at:at + n] - want_lse) <= lse_bound + 1e-30), f"lse {b}"
        at += n
    assert torch.equal(out, vef.forward_packed(q, k, v, cu, window=window, n_sinks=sinks, scale=scale))
    assert vef.device_status() == 0


@pytest.mark.parametrize("D", [8, 24, 64, 72, 120, 128])
@pytest.mark.parametrize("heads", [(1, 1), (2, 1), (3, 1), (4, 4), (12, 4)])
def test_each_prompt_as_if_alone(td, heads, D):
    """Many lengths around tiles: the same bits as forward_window on each prompt."""
    torch, dev = td
    lens = [1, 31, 32, 33, 127, 128, 129, 255, 257, 384, 0, 511, 5, 650]
    name = "f16" if D % 16 else "bf16"
    for window, sinks in ((None, 0), (90, 2)):
        q, k, v = rows(td, name, heads, sum(lens) + 9, D, D, "packed")
        out = torch.full_like(q, 7.0)
        cu = starts(torch, lens, dev, first=4)
        got, lse = vef.forward_packed(q, k, v, cu, window=window, n_sinks=sinks, scale=0.2, out=out, return_lse=True)
        assert got is out
        at = 4
        for n in lens:
            part = [x[:, :, at:at + n].contiguous() for x in (q, k, v)]
            want, want_lse = vef.forward_window(*part, window=window, n_sinks=sinks, scale=0.2, return_lse=True)
            assert torch.equal(out[:, :, at:at + n], want) and torch.equal(lse[:, :, at:at + n], want_lse), n
            at += n
        assert bool((out[:, :, :4] == 7).all()) and bool((out[:, :, at:] == 7).all())  # rows of nobody


def test_many_prompts(td):
    """More prompts than warps, more row blocks than threads, one long prompt among them."""
    torch, dev = td
    rng = np.random.default_rng(7)
    lens = rng.integers(0, 40, size=3000).tolist() + [9000] + rng.integers(0, 300, size=200).tolist()
    q, k, v = rows(td, "bf16", (4, 2), sum(lens), 64, 4300, "packed")
    cu = starts(torch, lens, dev)
    out = vef.forward_packed(q, k, v, cu, scale=0.125)
    ends = np.cumsum(lens)
    for b in (0, 17, 2999, 3000, 3001, len(lens) - 1) + tuple(rng.integers(0, len(lens), 20)):
        n, at = lens[b], int(ends[b]) - lens[b]
        if n:
            want = vef.forward_window(*(x[:, :, at:at + n].contiguous() for x in (q, k, v)), scale=0.125)
            assert torch.equal(out[:, :, at:at + n], want)
    assert vef.device_status() == 0


@pytest.mark.parametrize("n_seqs", [1, 2, 31, 32, 33, 64, 97, 127, 128, 129, 200])
@pytest.mark.parametrize("heads", [(1, 1), (3, 1), (4, 2), (7, 1)])
def test_blocks_find_what_the_list_has(td, heads, n_seqs):
    """Around the most prompts for which blocks find their pairs themselves, several rounds of
    them, odd and even groups: against each prompt alone."""
    torch, dev = td
    rng = np.random.default_rng(n_seqs)
    lens = rng.integers(0, 700, size=n_seqs)
    lens[rng.integers(0, n_seqs)] = 3000
    lens = lens.tolist()
    q, k, v = rows(td, "bf16", heads, sum(lens), 64, 4800 + n_seqs, "packed")
    out = torch.full_like(q, 7.0)
    vef.forward_packed(q, k, v, starts(torch, lens, dev), scale=0.125, out=out)
    ends = np.cumsum(lens)
    for b in {0, n_seqs - 1, int(np.argmax(lens)), *rng.integers(0, n_seqs, 8).tolist()}:
        n, at = lens[b], int(ends[b]) - lens[b]
        if n:
            want = vef.forward_window(*(x[:, :, at:at + n].contiguous() for x in (q, k, v)), scale=0.125)
            assert torch.equal(out[:, :, at:at + n], want), b
    assert not bool((out == 7).all(-1).any())  # every row was computed
    assert vef.device_status() == 0


def test_a_buffer_longer_than_the_list_in_shared_memory(td):
    """Over 2^20 rows: the list is counted in the workspace."""
    torch, dev = td
    total = (1 << 20) + 777
    q, k, v = (torch.randn(1, 1, total, 8, device=dev).half() for _ in range(3))
    lens = [1000, total - 1500, 500]
    cu = starts(torch, lens, dev)
    out = vef.forward_packed(q, k, v, cu, window=200, scale=0.3)
    at = 0
    for n in lens:
        want = vef.forward_window(*(x[:, :, at:at + n] for x in (q, k, v)), window=200, scale=0.3)
        assert torch.equal(out[:, :, at:at + n], want)
        at += n


def test_other_prompts_do_not_get_through(td):
    """NaN and infinities in one prompt (keys, values, queries) leave the others' bits alone."""
    torch, dev = td
    for D in (64, 128):
        lens = [100, 200, 70, 300]
        q, k, v = rows(td, "f16", (4, 2), sum(lens), D, 4400, "packed")
        cu = starts(torch, lens, dev)
        clean = vef.forward_packed(q, k, v, cu, scale=0.1)
        for lo, hi in ((100, 300), (370, 670)):
            dirty = [x.clone() for x in (q, k, v)]
            for x in dirty:
                x[:, :, lo:hi:7] = float("nan")
                x[:, :, lo + 1:hi:9] = float("inf")
            out = vef.forward_packed(*dirty, cu, scale=0.1)
            assert torch.equal(out[:, :, :lo], clean[:, :, :lo]) and torch.equal(out[:, :, hi:], clean[:, :, hi:])
        # a value that later rows of its own prompt see, and earlier ones do not
        dirty = v.clone()
        dirty[:, :, 150, 3] = float("nan")
        out = vef.forward_packed(q, k, dirty, cu, scale=0.1)
        bad = torch.isnan(out)
        assert bool(bad[:, :, 150:300, 3].all()) and int(bad.sum()) == 4 * 150
        part = [x[:, :, 100:300].contiguous() for x in (q, k, dirty)]
        want = vef.forward_window(*part, scale=0.1)
        assert torch.equal(torch.nan_to_num(out[:, :, 100:300]), torch.nan_to_num(want))
        assert torch.equal(out[:, :, :100], clean[:, :, :100]) and torch.equal(out[:, :, 300:], clean[:, :, 300:])


def test_starts_out_of_range(td):
    """Values outside the buffer are held to it; a prompt that ends before it begins is empty."""
    torch, dev = td
    q, k, v = rows(td, "bf16", (2, 1), 300, 64, 4500)
    out = torch.full_like(q, 7.0)
    vef.forward_packed(q, k, v, ints(torch, [-50, 100, 2 ** 31 - 1], dev), scale=0.1, out=out)
    want = vef.forward_packed(q, k, v, ints(torch, [0, 100, 300], dev), scale=0.1)
    assert torch.equal(out, want)
    out.fill_(7.0)
    vef.forward_packed(q, k, v, ints(torch, [0, 100, 60, 60], dev), scale=0.1, out=out)
    assert torch.equal(out[:, :, :100], want[:, :, :100]) and bool((out[:, :, 100:] == 7).all())
    # prompts with more rows than there are: none is computed
    for bad in ([0, 300, 0, 300, 0, 300, 0, 300, 0, 300, 0, 300], [0, 200, 0, 200], [2 ** 31 - 1, -2 ** 31] * 2000 + [300], [5] * 9):
        out.fill_(7.0)
        vef.forward_packed(q, k, v, ints(torch, bad, dev), scale=0.1, out=out)
        assert bool((out == 7).all())
    assert vef.device_status() == 0
    for empty in (ints(torch, [0], dev), ints(torch, [0, 0], dev)):
        out.fill_(7.0)
        vef.forward_packed(q, k, v, empty, out=out)
        assert bool((out == 7).all())
    none = [x[:, :, :0] for x in (q, k, v)]
    assert vef.forward_packed(*none, ints(torch, [0, 0], dev)).shape == (1, 2, 0, 64)


def test_streams_graphs_and_threads(td):
    torch, dev = td
    lens = [400, 3, 900, 260]
    q, k, v = rows(td, "bf16", (8, 2), sum(lens), 128, 4600, "packed")
    cu = starts(torch, lens, dev)
    how = dict(window=300, n_sinks=4, scale=0.09)
    want = vef.forward_packed(q, k, v, cu, **how)
    streams = [torch.cuda.Stream(dev) for _ in range(3)]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream(dev))
    got = [vef.forward_packed(q, k, v, cu, stream=s, **how) for s in streams]
    torch.cuda.synchronize(dev)
    assert all(torch.equal(t, want) for t in got)
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = vef.forward_packed(q, k, v, cu, **how)
        graphs.append((g, out))
    cu.copy_(starts(torch, [10, 1000, 0, 553], dev))
    for (g, _), s in zip(graphs, streams):
        s.wait_stream(torch.cuda.current_stream(dev))
        with torch.cuda.stream(s):
            g.replay()
    torch.cuda.synchronize(dev)
    want = vef.forward_packed(q, k, v, cu, **how)
    assert all(torch.equal(out, want) for _, out in graphs)


def test_refusals(td):
    torch, dev = td
    q, k, v = rows(td, "f16", (2, 1), 50, 16, 4700)
    cu = ints(torch, [0, 50], dev)
    with pytest.raises(TypeError):
        vef.forward_packed(q, k, v, None)
    with pytest.raises(TypeError):
        vef.forward_packed(q, k, v, cu.long())
    with pytest.raises(ValueError):
        vef.forward_packed(q, k, v, cu.cpu())
    with pytest.raises(ValueError):
        vef.forward_packed(q, k, v, cu[:0])
    with pytest.raises(ValueError):
        vef.forward_packed(q, k, v[:, :, :40], cu)
    with pytest.raises(vef.VattnError):
        vef.forward_packed(q, k[:, :, :40], v[:, :, :40], cu)
    with pytest.raises(vef.VattnError):
        vef.forward_packed(q.expand(2, 2, 50, 16), k.expand(2, 1, 50, 16), v.expand(2, 1, 50, 16), cu)
    with pytest.raises(vef.VattnError):
        vef.forward_packed(q, k, v, cu, out=q)
