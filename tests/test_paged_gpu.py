"""GPU tests of the attention of new tokens over the paged 8-bit cache against
the f64 oracle within counted bounds."""
import numpy as np
import pytest

from oracle import decoder as od
from oracle import serving as osv
import vision_encoder_flash_gb300 as vef
from decoder_util import HALF_STEP, TINY, assert_within, f64, laid_out, normal
from serving_util import filled, ints, values

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


def signed(words):
    return [w - (1 << 64) if w >> 63 else w for w in words]


def against_the_oracle(out, q, cache, window, sinks, words, scale, name, what="out"):
    """out of forward_paged on a cache (k, v, scales, table, lens), words per sequence or None."""
    k, v, ks, vs = values(cache[0]), values(cache[1]), f64(cache[2]), f64(cache[3])
    table, lens = cache[4].tolist(), cache[5].tolist()
    page = k.shape[2]
    B, H, T, D = q.shape
    N = max(1, table and len(table[0]) * page)
    ones = np.ones_like(k)
    rows = [[osv.gathered(x, s, table[b], min(max(lens[b], 0), N)) for x, s in ((k, ks), (v, vs), (ones, vs))] for b in range(B)]
    K = k.shape[1]
    kk, vv, sv = np.zeros((B, K, N, D)), np.zeros((B, K, N, D)), np.ones((B, K, N))
    seen = np.zeros((B, T, N), bool)
    for b in range(B):
        n = min(max(lens[b], 0), N)
        kk[b, :, :n], vv[b, :, :n], sv[b, :, :n] = rows[b][0][0], rows[b][1][0], rows[b][2][0][..., 0]
        seen[b] = od.cached_visible(T, N, window, sinks, lens[b], words[b] if words else None)
        seen[b, :, :n] &= rows[b][0][1]
    want, bound = osv.paged_attention(f64(q), kk, vv, sv, seen, float(np.float32(scale)), HALF_STEP[name])
    assert_within(out, want, bound, what, tiny=2 * TINY[name])


CASES = [
    # type, (B, Hq, Hk, T, D), page, kv_len, window, sinks, tree, layout of the pool, of q
    ("bf16", (1, 1, 1, 1, 16), 16, [1], None, 0, False, "heads", "plain"),
    ("f16", (3, 4, 2, 1, 64), 16, [200, 77, 1], None, 0, False, "heads", "plain"),
    ("bf16", (2, 8, 1, 1, 128), 64, [1500, 640], None, 0, False, "tokens", "packed"),
    ("f16", (2, 32, 8, 1, 64), 32, [700, 65], 128, 4, False, "both", "plain"),
    ("bf16", (2, 6, 2, 2, 80), 48, [300, 64], None, 0, False, "tokens", "padded"),
    ("f16", (2, 4, 4, 5, 48), 112, [390, 5], 30, 70, False, "heads", "plain"),
    ("bf16", (3, 4, 1, 7, 96), 16, [300, 3, 0], None, 0, False, "heads", "plain"),   # fewer rows in use than new tokens
    ("f16", (2, 4, 2, 31, 64), 32, [500, 131], None, 0, True, "tokens", "plain"),
    ("bf16", (2, 8, 2, 64, 128), 64, [300, 64], 40, 3, True, "heads", "packed"),
    ("f16", (2, 3, 1, 64, 32), 1024, [200, 30], 7, 2, True, "heads", "plain"),        # a window inside the tree
    ("bf16", (1, 5, 1, 13, 64), 64, [3777], 1000, 4, True, "tokens", "plain"),
    ("f16", (1, 16, 1, 17, 112), 80, [260], None, 0, True, "both", "padded"),
    ("bf16", (40, 4, 4, 1, 64), 16, [130 - 3 * b for b in range(40)], None, 0, False, "heads", "plain"),
    ("f16", (1, 2, 2, 1, 64), 128, [9000], None, 0, False, "heads", "plain"),         # one long sequence
    ("bf16", (1, 128, 2, 3, 16), 32, [90], 20, 0, True, "heads", "plain"),            # 192 rows a key head
    ("bf16", (2, 4, 2, 1, 32), 16, [-3, 10 ** 6], None, 0, False, "heads", "plain"),  # lengths outside the table
]


def build(td, case, seed):
    torch, dev = td
    name, (B, H, K, T, D), page, lens, window, sinks, tree, layout, q_layout = case
    rng = np.random.default_rng(seed)
    q = laid_out(torch, normal(torch, (B, H, T, D), name, seed, dev), q_layout)
    held = [min(max(n, 0), 5000) if n > 10 ** 5 or n < 0 else n for n in lens]
    held = [64 if n > 10 ** 5 else h for n, h in zip(lens, held)]
    cache = list(filled(torch, (K, D), held, page, seed, dev, layout))
    if held != lens:
        cache[5] = ints(torch, lens, dev)
    words = [tree_words(T, rng) for _ in range(B)] if tree else None
    mask = torch.tensor([signed(w) for w in words], dtype=torch.int64, device=dev) if tree else None
    return q, cache, words, dict(tree_mask=mask, window=window, n_sinks=sinks, scale=1.3 / D ** 0.5)


@pytest.mark.parametrize("i", range(len(CASES)))
def test_against_the_oracle(td, i):
    torch, dev = td
    case = CASES[i]
    q, cache, words, how = build(td, case, 3000 + 10 * i)
    out = vef.forward_paged(q, *cache, **how)
    against_the_oracle(out, q, cache, case[4], case[5], words, how["scale"], case[0])
    assert torch.equal(out, vef.forward_paged(q, *cache, **how))
    assert vef.device_status() == 0


@pytest.mark.parametrize("D", [16, 32, 48, 64, 80, 96, 112, 128])
@pytest.mark.parametrize("H,T", [(1, 1), (4, 4), (4, 6), (5, 5), (8, 4), (11, 3), (8, 7), (7, 11), (4, 31), (5, 50)])
def test_rows_and_widths(td, H, T, D):
    """Rows for one, two and four groups of warps, of every width, boxes of 16, 32 and 64 rows."""
    torch, dev = td
    for i, (page, window, tree, layout) in enumerate(((64, None, False, "tokens"), (96, 50, True, "both"), (16, 33, False, "heads"))):
        case = ("f16" if i else "bf16", (2, 2 * H, 2, T, D), page, [333, 70], window, 2 * i, tree, layout, "packed")
        q, cache, words, how = build(td, case, 800 + D + H)
        out = vef.forward_paged(q, *cache, **how)
        against_the_oracle(out, q, cache, window, 2 * i, words, how["scale"], case[0])


@pytest.mark.parametrize("N", [64, 65, 128, 130, 250, 390, 510, 900, 2049])
def test_shares(td, N):
    """One share of the keys to many, some without a key in short sequences: on three streams at
    once, and replayed with other lengths, pages and values."""
    torch, dev = td
    case = ("f16", (5, 8, 2, 3, 80), 16, [N, 129, 40, 3, 0], None, 2, True, "heads", "plain")
    case = case[:3] + ([min(n, N) for n in case[3]],) + case[4:]
    q, cache, words, how = build(td, case, 900 + N)
    out = vef.forward_paged(q, *cache, **how)
    against_the_oracle(out, q, cache, None, 2, words, how["scale"], "f16")
    streams = [torch.cuda.Stream(dev) for _ in range(3)]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream(dev))
    got = [vef.forward_paged(q, *cache, stream=s, **how) for s in streams]
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize(dev)
    assert all(torch.equal(t, out) for t in got)
    with torch.cuda.graph(graph):
        again = vef.forward_paged(q, *cache, **how)
    for t in cache[:2]:
        t.view(torch.uint8).copy_(torch.randint(0, 0x7f, t.shape, dtype=torch.uint8, device=dev))
    cache[4].copy_(cache[4].flip(0))
    cache[5].copy_(torch.tensor([0, N, 3, min(N, 131), 64], dtype=torch.int32))
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize(dev)
    assert torch.equal(again, vef.forward_paged(q, *cache, **how))
    against_the_oracle(again, q, cache, None, 2, words, how["scale"], "f16")


@pytest.mark.parametrize("name", ["f16", "bf16"])
def test_window_edges_and_first_keys(td, name):
    """Windows and first keys that end inside boxes, tiles and pages."""
    torch, dev = td
    for i, (page, window, sinks, T) in enumerate(((64, 1, 0, 1), (64, 100, 5, 1), (16, 17, 16, 2), (32, 33, 40, 1),
                                                  (128, 200, 130, 3), (48, 290, 1, 1), (64, 64, 300, 1), (16, 2000, 3, 4))):
        case = (name, (2, 4, 2, T, 64), page, [301, 130], window, sinks, False, "heads", "plain")
        q, cache, words, how = build(td, case, 1200 + i)
        out = vef.forward_paged(q, *cache, **how)
        against_the_oracle(out, q, cache, window, sinks, None, how["scale"], name, f"case {i}")


def test_pages_that_are_not_there(td):
    """Rows of a missing page are seen by none: given back behind a window, or a row left empty."""
    torch, dev = td
    case = ("bf16", (3, 4, 2, 1, 64), 32, [500, 100, 20], None, 0, False, "heads", "plain")
    q, cache, _, how = build(td, case, 1300)
    for gone in ([[0, 3, 3], [1, 2, 2]], [[0, 0, 16], [1, 0, 4], [2, 0, 1]]):
        table = cache[4].clone()
        for b, lo, hi in gone:
            table[b, lo:hi] = torch.tensor([-1, 2 ** 31 - 1, -2 ** 31, cache[0].shape[0]] * 4, dtype=torch.int32, device=dev)[:hi - lo]
        with_gaps = cache[:4] + [table, cache[5]]
        out = vef.forward_paged(q, *with_gaps, **how)
        against_the_oracle(out, q, with_gaps, None, 0, None, how["scale"], "bf16")
    assert not f64(out).any()
    # what lies before the window may go
    how["window"] = 70
    want = vef.forward_paged(q, *cache, **how)
    table = cache[4].clone()
    table[0, :(500 - 70) // 32] = -1
    assert torch.equal(want, vef.forward_paged(q, *cache[:4], table, cache[5], **how))
    # no pages at all
    none = [t[:0] for t in cache[:4]]
    assert not f64(vef.forward_paged(q, *none, cache[4], cache[5], **how)).any()
    assert not f64(vef.forward_paged(q, *cache[:4], cache[4][:, :0].contiguous(), cache[5], **how)).any()


@pytest.mark.parametrize("D", [48, 80, 112])
@pytest.mark.parametrize("H,T", [(1, 1), (4, 3), (4, 6), (4, 8), (4, 11), (4, 16), (8, 40)])
def test_rows_behind_each_other_and_apart(td, H, T, D):
    """Rows of an odd number of 16 bytes, contiguous in their page or not: the same bits, with
    pages that are not there, and a NaN among the new tokens."""
    torch, dev = td
    for page, window, N in ((16, None, 700), (48, 90, 260), (256, None, 2900)):
        case = ("bf16", (2, 2 * H, 2, T, D), page, [N, N - 77], window, 3, T > 2, "heads", "plain")
        q, cache, words, how = build(td, case, 1360 + D + T)
        gone = [x.clone() for x in cache]
        gone[4][0, 0], gone[4][1, 1] = -1, 2 ** 31 - 1
        row = N - 77 - 1  # the newest token of sequence 1
        bad = [cache[0], cache[1].view(torch.uint8).clone().view(cache[1].dtype)] + list(cache[2:])
        bad[1].view(torch.uint8)[cache[4][1, row // page].item(), 1, row % page, D - 1] = 0xff
        for which in (cache, gone, bad):
            apart = [x.transpose(1, 2).contiguous().transpose(1, 2) for x in which[:2]] + list(which[2:])
            assert which[0].stride(2) == D and apart[0].stride(2) == 2 * D
            out = vef.forward_paged(q, *which, **how)
            other = vef.forward_paged(q, *apart, **how)
            assert torch.equal(torch.isnan(out), torch.isnan(other))
            assert torch.equal(out.nan_to_num(nan=3.0), other.nan_to_num(nan=3.0))
            if which is bad:
                assert bool(torch.isnan(out[1, H:, T - 1, D - 1]).all())
                assert int(torch.isnan(out).sum()) == H
            else:
                against_the_oracle(out, q, which, window, 3, words, how["scale"], "bf16")
    assert vef.device_status() == 0


def test_pages_shared_by_sequences(td):
    torch, dev = td
    case = ("f16", (2, 4, 1, 1, 64), 16, [64, 64], None, 0, False, "heads", "plain")
    q, cache, _, how = build(td, case, 1350)
    cache[4][1, :3] = cache[4][0, :3]
    cache[4][0, 1] = cache[4][0, 0]  # and one page twice in one sequence
    out = vef.forward_paged(q, *cache, **how)
    against_the_oracle(out, q, cache, None, 0, None, how["scale"], "f16")


def test_scales_far_apart(td):
    """Pages whose scales differ by many powers of two, and by none of two: rows led by either."""
    torch, dev = td
    for name in ("f16", "bf16"):
        case = (name, (2, 8, 2, 2, 64), 16, [200, 90], None, 0, False, "heads", "plain")
        q, cache, _, how = build(td, case, 1400)
        n_pages = cache[0].shape[0]
        rng = np.random.default_rng(5)
        for lo, hi in ((-32, -20), (-30, 2), (-20, 6)):
            v_scale = torch.from_numpy(2.0 ** rng.uniform(lo, hi, size=(n_pages, 2))).float().to(dev)
            with_scale = cache[:3] + [v_scale] + cache[4:]
            out = vef.forward_paged(q, *with_scale, **how)
            against_the_oracle(out, q, with_scale, None, 0, None, how["scale"], name, f"2^{lo} .. 2^{hi}")
        # a scale of 0: zeros
        v_scale = cache[3].clone()
        v_scale[cache[4][0, 2:5].long()] = 0
        with_scale = cache[:3] + [v_scale] + cache[4:]
        out = vef.forward_paged(q, *with_scale, **how)
        against_the_oracle(out, q, with_scale, None, 0, None, how["scale"], name, "a scale of 0")
    # a page of zeros with the smallest scale, which takes nearly all of the weight
    case = ("bf16", (1, 1, 1, 1, 16), 16, [32], None, 0, False, "heads", "plain")
    q, cache, _, how = build(td, case, 1401)
    first, second = cache[4][0].tolist()
    cache[0].view(torch.uint8)[first] = 0x38                    # keys of ones
    cache[0].view(torch.uint8)[second] = 0xb8                   # and of minus ones
    cache[1].view(torch.uint8)[first] = 0
    cache[2].fill_(1.0)
    cache[3][first], cache[3][second] = 2.0 ** -32, 2.0 ** 10
    q.fill_(0.5)
    out = vef.forward_paged(q, *cache, scale=1.0)
    against_the_oracle(out, q, cache, None, 0, None, 1.0, "bf16")


def test_large_and_small_queries(td):
    """bf16 rows near both ends of the range, zeros, and elements far apart in one row."""
    torch, dev = td
    case = ("bf16", (1, 6, 1, 1, 64), 16, [100], None, 0, False, "heads", "plain")
    q, cache, _, how = build(td, case, 1450)
    q[0, 0] *= 2.0 ** 100
    q[0, 1] *= 2.0 ** -100
    q[0, 2] = 0
    q[0, 3, 0, ::2] *= 2.0 ** -40
    q[0, 4] *= 2.0 ** -133
    for h, scale in ((0, 2.0 ** -103), (1, 2.0 ** 97), (2, 1.0), (3, 0.1), (4, 2.0 ** 120), (5, 2.0 ** -120)):
        out = vef.forward_paged(q[:, h:h + 1], *cache, scale=scale)
        against_the_oracle(out, q[:, h:h + 1], cache, None, 0, None, scale, "bf16", f"head {h}")


def test_words_without_bits_and_stray_bits(td):
    torch, dev = td
    case = ("bf16", (1, 2, 1, 4, 32), 16, [40], None, 0, False, "heads", "plain")
    q, cache, _, how = build(td, case, 1500)
    words = [1, 0, 0b101, 0b1000]  # the second token sees nothing, the last only itself and the cache
    mask = torch.tensor([words], dtype=torch.int64, device=dev)
    how["tree_mask"] = mask
    out = vef.forward_paged(q, *cache, **how)
    against_the_oracle(out, q, cache, None, 0, [words], how["scale"], "bf16")
    assert not f64(out[0, :, 1]).any()
    stray = mask | (1 << 40) | -(1 << 63)
    stray[0, 1] = 0
    how["tree_mask"] = stray
    assert torch.equal(out, vef.forward_paged(q, *cache, **how))


def test_values_that_are_not_finite(td):
    """NaN keys and values reach the rows that see them and no others; q's as forward_window has it."""
    torch, dev = td
    case = ("f16", (1, 4, 2, 3, 64), 16, [90], None, 0, True, "heads", "plain")
    q, cache, _, how = build(td, case, 1550)
    words = [0b001, 0b011, 0b101]
    how["tree_mask"] = torch.tensor([words], dtype=torch.int64, device=dev)
    clean = vef.forward_paged(q, *cache, **how)
    P = int(cache[4][0, 88 // 16])
    dirty = [cache[0].clone(), cache[1].clone()]
    for t in dirty:
        t.view(torch.uint8)[P, 0, 88 % 16, 5] = 0xff  # new token 1, first key head
    out = vef.forward_paged(q, *dirty, *cache[2:], **how)
    others = [0, 2]
    # the loops over visible pairs take the weights unrounded: within the bound of the formula
    zeroed = [t.clone() for t in dirty]
    for t in zeroed:
        t.view(torch.uint8)[P, 0, 88 % 16, 5] = 0
    keep = torch.zeros_like(out)
    keep[:, :, others] = out[:, :, others]
    ref = vef.forward_paged(q, *zeroed, *cache[2:], **how)
    keep[:, :, 1] = ref[:, :, 1]
    against_the_oracle(keep, q, zeroed + cache[2:], None, 0, [words], how["scale"], "f16")
    assert bool(torch.isnan(out[:, :2, 1]).all()) and torch.equal(out[:, 2:], clean[:, 2:])
    # only v, in a key of the cache that all see: that column is NaN, the others are not
    dirty = cache[1].clone()
    dirty.view(torch.uint8)[int(cache[4][0, 0]), 1, 3, 7] = 0x7f
    out = vef.forward_paged(q, cache[0], dirty, *cache[2:], **how)
    bad = torch.isnan(out)
    assert bool(bad[:, 2:, :, 7].all()) and int(bad.sum()) == 2 * 3
    assert torch.equal(out[~bad], clean[~bad])
    # infinities of q: scores of either sign are NaN; a row of NaN stays in its row
    q2 = q.clone()
    q2[0, 0, 0, 0], q2[0, 3, 2, 1] = float("inf"), float("nan")
    out = vef.forward_paged(q2, *cache, **how)
    assert bool(torch.isnan(out[0, 3, 2]).all()) and bool(torch.isnan(out[0, 0, 0]).any())
    same = torch.ones(out.shape[:3], dtype=torch.bool, device=dev)
    same[0, 0, 0] = same[0, 3, 2] = False
    assert torch.equal(out[same], clean[same])


def test_scales_of_pages_that_no_row_sees(td):
    """A page of new tokens that see nothing and that nothing sees, its bytes and scales NaN."""
    torch, dev = td
    for T in (20, 40):
        case = ("bf16", (1, 4, 1, T, 64), 16, [96], None, 0, False, "heads", "plain")
        q, cache, _, how = build(td, case, 1570 + T)
        words = [(1 << t) if t < T - 16 else 0 for t in range(T)]  # the last 16 fill the last page
        how["tree_mask"] = torch.tensor([words], dtype=torch.int64, device=dev)
        clean = vef.forward_paged(q, *cache, **how)
        against_the_oracle(clean, q, cache, None, 0, [words], how["scale"], "bf16")
        last = cache[4][0, 5].item()
        for x in cache[:2]:
            x.view(torch.uint8)[last] = 0x7f
        for s in cache[2:4]:
            s[last] = float("nan")
        out = vef.forward_paged(q, *cache, **how)
        assert torch.equal(out, clean)
        assert not f64(out)[0, :, T - 16:].any()


@pytest.mark.parametrize("D", [32, 64, 128])
@pytest.mark.parametrize("H,T", [(4, 6), (4, 12), (4, 15), (4, 31)])
def test_a_nan_in_wide_blocks(td, H, T, D):
    """A NaN value among the new tokens of a tree: all of the rows that see it, and no others."""
    torch, dev = td
    case = ("f16", (2, H, 1, T, D), 32, [300, 77], 150, 5, True, "heads", "plain")
    q, cache, words, how = build(td, case, 1580 + T + D)
    clean = vef.forward_paged(q, *cache, **how)
    against_the_oracle(clean, q, cache, 150, 5, words, how["scale"], "f16")
    bad = list(cache)
    bad[1] = cache[1].view(torch.uint8).clone()
    at = [1, T - 2]  # of each sequence's new tokens
    for b, n in enumerate(case[3]):
        row = n - T + at[b]
        bad[1][cache[4][b, row // 32].item(), 0, row % 32] = 0x7f
    bad[1] = bad[1].view(cache[1].dtype)
    out = vef.forward_paged(q, *bad, **how)
    seen = torch.tensor([[bool(words[b][t] >> at[b] & 1) for t in range(T)] for b in range(2)], device=dev)
    seen = seen[:, None, :, None].expand_as(out)
    assert bool(seen.any()) and not bool(seen.all())
    assert bool(torch.isnan(out[seen]).all())
    against_the_oracle(torch.where(seen, clean, out), q, cache, 150, 5, words, how["scale"], "f16")


def test_agrees_with_the_16_bit_cache(td):
    """The same values in a contiguous 16-bit cache: both within their bounds of each other."""
    torch, dev = td
    case = ("f16", (2, 8, 2, 5, 64), 16, [300, 130], 90, 3, False, "heads", "plain")
    q, cache, _, how = build(td, case, 1600)
    table = cache[4].long()
    rows = [(x.float() * s[..., None, None])[table].transpose(1, 2).flatten(2, 3).half() for x, s in zip(cache[:2], cache[2:4])]
    a, b = f64(vef.forward_paged(q, *cache, **how)), f64(vef.forward_cached(q, *rows, cache[5], **how))
    top = float(torch.nan_to_num(rows[1]).abs().max())
    # two roundings of the weights and of the result each, and 2^-13 for the f32 sums
    assert np.abs(a - b).max() <= 2 * (2 * HALF_STEP["f16"] + 2.0 ** -13) * top


def test_streams_graphs_and_views(td):
    torch, dev = td
    case = ("bf16", (2, 8, 2, 1, 128), 64, [2500, 900], None, 0, False, "tokens", "plain")
    q, cache, _, _ = build(td, case, 1700)
    run = lambda **kw: vef.forward_paged(q, *cache, scale=0.1, **kw)
    want = run()
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = run()
        graphs.append((g, out))
    streams = [torch.cuda.Stream(dev) for _ in range(2)]
    cache[5].copy_(torch.tensor([2431, 1], dtype=torch.int32))
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


def test_many_sequences_and_heads(td):
    torch, dev = td
    B = 70001
    q = normal(torch, (B, 2, 1, 16), "f16", 1800, dev)
    k, v = (torch.randint(0, 0x7f, (B, 1, 16, 16), dtype=torch.uint8, device=dev) for _ in range(2))
    ks, vs = (torch.rand(B, 1, device=dev) * 0.01 + 0.001 for _ in range(2))
    table = torch.arange(B, dtype=torch.int32, device=dev).flip(0).view(B, 1).contiguous()
    lens = torch.arange(B, dtype=torch.int32, device=dev) % 18
    whole = vef.forward_paged(q, k, v, ks, vs, table, lens)
    for a in (0, 32767, 65535, 65536, B - 1):
        s = slice(a, a + 1)
        assert torch.equal(whole[s], vef.forward_paged(q[s], k, v, ks, vs, table[s], lens[s]))
    # one key head for 1030 query heads: 65920 rows of 64 new tokens
    q = normal(torch, (1, 1030, 64, 16), "f16", 1801, dev)
    cache = filled(torch, (1, 16), [90], 16, 1802, dev)
    got = vef.forward_paged(q, *cache, scale=0.2)
    for a in (0, 513, 1029):
        against_the_oracle(got[:, a:a + 1], q[:, a:a + 1], cache, None, 0, None, 0.2, "f16")
    assert vef.device_status() == 0


def test_refusals(td):
    torch, dev = td
    case = ("f16", (1, 4, 2, 4, 64), 16, [40], None, 0, False, "heads", "plain")
    q, cache, _, _ = build(td, case, 1900)
    with pytest.raises(vef.VattnError):
        vef.forward_paged(normal(torch, (1, 4, 65, 64), "f16", 1, dev), *cache)  # 65 new tokens
    with pytest.raises(TypeError):
        vef.forward_paged(q.float(), *cache)
    with pytest.raises(TypeError):
        vef.forward_paged(q, *cache, tree_mask=torch.ones(1, 4, dtype=torch.int32, device=dev))
    with pytest.raises(ValueError):
        vef.forward_paged(q, *cache, window=0)
    with pytest.raises(ValueError):
        vef.forward_paged(q[..., :48], *cache)
    with pytest.raises(vef.VattnError):
        vef.forward_paged(q[:, :3], *cache)  # heads that do not divide
    with pytest.raises(vef.VattnError):
        vef.forward_paged(q, *cache, out=q)
    with pytest.raises(vef.VattnError):
        vef.forward_paged(q, *cache, scale=0.0)
