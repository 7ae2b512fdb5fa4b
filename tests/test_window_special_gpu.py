"""NaN and infinity in the values of windowed attention: they reach the rows
that see them and no other, at the cost of a few tiles."""
import numpy as np
import pytest

from oracle import decoder as od
import vision_encoder_flash_gb300 as vef
from decoder_util import f64, normal

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def td():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    vef.load_library()
    return torch, torch.device("cuda", 0)


def kinds(v, seen, group):
    """[B, H, M, D]: the sum over the seen keys of what is not finite in v
    [B, K, N, D] (0 where nothing is), every weight being positive."""
    odd = np.where(np.isfinite(v), 0.0, v)
    some = ~np.isfinite(v)
    out = np.zeros((v.shape[0], v.shape[1] * group, seen.shape[1], v.shape[3]))
    for b in range(v.shape[0]):
        for k in range(v.shape[1]):
            for j, d in zip(*np.nonzero(some[b, k])):
                with np.errstate(invalid="ignore"):
                    out[b, k * group:(k + 1) * group, seen[b, :, j], d] += odd[b, k, j, d]
    return out


CASES = [
    # type, (B, Hq, Hk, M, N, D), window, sinks, kv_len, q_start
    ("f16", (1, 2, 2, 300, 300, 64), 50, 2, None, None),
    ("bf16", (1, 3, 1, 700, 700, 128), 129, 130, None, None),             # first keys past one tile, an odd group
    ("f16", (1, 4, 1, 513, 513, 72), None, 0, None, None),
    ("bf16", (2, 2, 1, 200, 640, 40), 300, 3, [640, 333], None),           # queries end a longer sequence
    ("f16", (2, 2, 2, 400, 400, 96), 128, 0, [400, 131], [0, 0]),
    ("bf16", (1, 2, 2, 384, 384, 32), 128, 128, None, None),               # every border on a tile's
    ("f16", (1, 1, 1, 90, 260, 8), 70, 1, None, [-20]),
    ("bf16", (1, 40, 4, 900, 900, 64), 200, 0, None, None),                # more units than blocks
    ("bf16", (2, 16, 4, 3000, 3000, 128), 500, 5, None, None),             # several rounds of items, some taken again
    ("f16", (2, 18, 6, 2500, 2500, 64), None, 0, [2500, 1700], [0, 0]),
]


@pytest.mark.parametrize("many", [False, True])
@pytest.mark.parametrize("i", range(len(CASES)))
def test_reaches_the_rows_that_see_it(td, i, many):
    torch, dev = td
    name, (B, H, K, M, N, D), window, sinks, kv_len, q_start = CASES[i]
    rng = np.random.default_rng(40 + i)
    q, k, v = (normal(torch, s, name, 400 + 3 * i + j, dev) for j, s in enumerate(((B, H, M, D), (B, K, N, D), (B, K, N, D))))
    ints = lambda x: None if x is None else torch.tensor(x, dtype=torch.int32, device=dev)
    # scores of a few units: no weight is so small that it rounds to 0
    how = dict(window=window, n_sinks=sinks, scale=0.25 / D ** 0.5, kv_len=ints(kv_len), q_start=ints(q_start))
    want, wlse = vef.forward_window(q, k, v, return_lse=True, **how)
    bad = rng.choice([np.nan, np.inf, -np.inf, np.inf], size=(B, K, N, D))
    place = rng.random((B, K, N, D)) < (0.02 if many else 3.0 / (N * D))
    place[:, :, [0, N // 2, N - 1], D - 1] = True
    if many:
        place[:, :, N // 3] = True
    bad, place = torch.from_numpy(bad).to(dev).to(v.dtype), torch.from_numpy(place).to(dev)
    v = torch.where(place, bad, v)
    out, lse = vef.forward_window(q, k, v, return_lse=True, **how)
    assert torch.equal(lse, wlse)
    seen = np.stack([od.window_visible(M, N, window, sinks, None if kv_len is None else kv_len[b],
                                       None if q_start is None else q_start[b]) for b in range(B)])
    expect = kinds(f64(v), seen, H // K)
    got, clean = f64(out), f64(want)
    hit = expect != 0  # (NaN too)
    assert hit.any()
    assert np.array_equal(got[~hit], clean[~hit])
    assert np.array_equal(np.isnan(got[hit]), np.isnan(expect[hit]))
    inf = hit & ~np.isnan(expect)
    assert np.array_equal(got[inf], expect[inf])
    assert torch.equal(out.view(torch.int16), vef.forward_window(q, k, v, **how).view(torch.int16))
    assert vef.device_status() == 0


@pytest.mark.parametrize("window", [None, 1024])
@pytest.mark.parametrize("dim", [64, 128])
def test_costs_a_few_tiles(td, dim, window):
    """One NaN at a first key of a long prompt: seen by all rows, hidden from
    none but the first block's; and values that are NaN throughout."""
    torch, dev = td
    N = 8192
    q, k, v = (normal(torch, (1, h, N, dim), "bf16", 430 + i, dev) for i, h in enumerate((16, 4, 4)))
    how = dict(window=window, n_sinks=4, scale=0.25 / dim ** 0.5)

    def time(values):
        best = float("inf")
        for _ in range(6):
            a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
            a.record()
            for _ in range(4):
                out = vef.forward_window(q, k, values, **how)
            b.record()
            torch.cuda.synchronize(dev)
            best = min(best, a.elapsed_time(b))
        return best, out

    clean, want = time(v)
    one = v.clone()
    one[0, 1, 1, 5] = float("nan")
    t_one, out = time(one)
    full = torch.full_like(v, float("nan"))
    t_full, none = time(full)
    print(f"dim {dim} window {window}: clean {clean / 4 * 1e3:.1f} us, one {t_one / 4 * 1e3:.1f}, all {t_full / 4 * 1e3:.1f}")
    rest = torch.ones_like(out, dtype=torch.bool)
    rest[0, 4:8, 1:, 5] = False
    assert torch.equal(out[rest], want[rest]) and bool(torch.isnan(out[~rest]).all())
    assert bool(torch.isnan(none).all())
    assert vef.device_status() == 0
    # what is looked at once more is two to five tiles of a walk of 9 to 64
    assert t_one < 2 * clean and t_full < 12 * clean
