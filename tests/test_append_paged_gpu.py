"""GPU tests of appending to the paged cache: every byte and scale against the
f64 oracle, exact but for values within f32's error of a rounding's border."""
import numpy as np
import pytest

from oracle import serving as osv
import vision_encoder_flash_gb300 as vef
from decoder_util import f64, laid_out, normal
from serving_util import ints, pool, values

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


def check(got, scale, want, what):
    """A pool and its scales against the oracle's; NaN where the oracle has it."""
    got, scale = values(got), f64(scale)
    off = np.argwhere((scale != want.scale) & ~want.loose)
    assert off.size == 0, f"{what}: {len(off)} scales, first {off[0]}: {scale[tuple(off[0])]} not {want.scale[tuple(off[0])]}"
    tight = (scale == want.scale)[:, :, None, None]
    ok = ((got >= want.lo) & (got <= want.hi)) | (np.isnan(got) & np.isnan(want.lo)) | ~tight
    off = np.argwhere(~ok)
    assert off.size == 0, (f"{what}: {len(off)} values, first {off[0]}: {got[tuple(off[0])]}, not "
                           f"{want.lo[tuple(off[0])]} .. {want.hi[tuple(off[0])]}")


class Server:
    """A cache and its oracle, to which both append the same rows."""

    def __init__(self, td, heads, page, dim, tables, n_pages, layout="heads", seed=0):
        self.torch, self.dev = td
        torch = self.torch
        self.k, self.v, self.big = pool(torch, n_pages, heads, page, dim, layout, self.dev)
        self.ks, self.vs = (torch.full((n_pages, heads), 2.0, device=self.dev) for _ in range(2))
        self.tables, self.table = tables, ints(torch, tables, self.dev)
        self.want = [osv.Cache(values(x), f64(s)) for x, s in ((self.k, self.ks), (self.v, self.vs))]
        self.lens = [0] * len(tables)

    def cache(self):
        return self.k, self.v, self.ks, self.vs, self.table, ints(self.torch, self.lens, self.dev)

    def append(self, k, v, new, rope, packed, positions=None, factors=None, base=10000.0, **kw):
        """k, v [1, H, total, D] (packed) or [B, H, T, D]; new: tokens of each sequence."""
        torch, dev = self.torch, self.dev
        self.lens = [a + b for a, b in zip(self.lens, new)]
        starts = np.concatenate([[0], np.cumsum(new)])
        cu = ints(torch, starts.tolist(), dev) if packed else None
        pos = None if positions is None else ints(torch, positions, dev)
        fac = None if factors is None else torch.tensor(factors, dtype=torch.float32, device=dev)
        vef.append_paged(k, v, *self.cache(), cu_seqlens=cu, rope_dims=rope, positions=pos, base=base, factors=fac, **kw)
        kn, vn = f64(k), f64(v)
        for b, n in enumerate(new):
            xk, xv = (x[0, :, starts[b]:starts[b] + n] if packed else x[b] for x in (kn, vn))
            at = np.arange(self.lens[b] - n, self.lens[b])
            if positions is not None:
                at = np.asarray(positions[0][starts[b]:starts[b] + n] if packed else positions[b])
            with np.errstate(invalid="ignore"):
                xk, err = osv.rotated(xk, at, rope, base, None if fac is None else f64(fac))
                self.want[0].append(self.tables[b], self.lens[b], xk, err)
                self.want[1].append(self.tables[b], self.lens[b], xv, np.zeros_like(xv))

    def check(self):
        check(self.k, self.ks, self.want[0], "k")
        check(self.v, self.vs, self.want[1], "v")
        assert vef.device_status() == 0


def tables_for(B, most, n_pages, seed):
    return np.random.default_rng(seed).permutation(n_pages)[:B * most].reshape(B, most).tolist()


CASES = [
    # type, H, D, page, rope, layout of the pool, of k and v
    ("bf16", 2, 64, 16, 64, "heads", "packed"),
    ("f16", 1, 128, 64, 128, "tokens", "plain"),
    ("bf16", 3, 80, 48, 48, "both", "padded"),
    ("f16", 4, 16, 32, 16, "heads", "packed"),
    ("bf16", 2, 96, 16, 20, "tokens", "plain"),     # halves that 16 bytes do not cut
    ("f16", 2, 48, 112, 7, "heads", "packed"),      # an odd number of rotated dims
    ("f16", 1, 32, 1024, 32, "heads", "plain"),     # more of a page than the threads hold
    ("bf16", 1, 112, 256, 0, "both", "packed"),     # no rotation
    ("bf16", 3, 80, 48, 40, "tokens", "packed"),    # halves that 8 bytes cut, and 16 do not
    ("f16", 2, 48, 1024, 24, "heads", "plain"),     # such, and more of a page than the threads hold
]


@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("i", range(len(CASES)))
def test_appends_in_turn(td, i, packed):
    """Prompts, parts and tokens after each other: scales that grow, pages begun anew."""
    torch, dev = td
    name, H, D, page, rope, layout, rows = CASES[i]
    B = 3
    most = 400 // page + 3
    s = Server(td, H, page, D, tables_for(B, most, B * most + 2, i), B * most + 2, layout)
    rng = np.random.default_rng(50 + i)
    steps = [[37, 1, page], [1, 1, 1], [5, 0, 150], [1, 1, 1], [page, 2, 3], [1, 1, 1]] if packed else \
        [[41] * 3, [1] * 3, [2] * 3, [page + 1] * 3, [1] * 3, [64] * 3]
    for n, new in enumerate(steps):
        scale = float(2.0 ** rng.integers(-3, 4))
        shape = (1, H, sum(new), D) if packed else (B, H, new[0], D)
        k, v = (laid_out(torch, normal(torch, shape, name, 100 * i + 10 * n + j, dev, scale), rows) for j in range(2))
        s.append(k, v, new, rope, packed)
        s.check()


@pytest.mark.parametrize("D", [16, 32, 48, 64, 80, 96, 112, 128])
@pytest.mark.parametrize("page", [16, 80, 1008])
def test_widths_and_pages(td, page, D):
    torch, dev = td
    B, H, T = 2, 2, 130
    most = -(-2 * T // page) + 1
    s = Server(td, H, page, D, tables_for(B, most, B * most, page), B * most, "tokens")
    for n, name in enumerate(("bf16", "f16")):
        k, v = (normal(torch, (B, H, T, D), name, D + n + j, dev) for j in range(2))
        s.append(k, v, [T] * B, D // 2 if n else D, False)
    s.check()


def test_positions_factors_and_base(td):
    """Rows at positions of their own: a tree's depths, far ones, in both forms."""
    torch, dev = td
    rng = np.random.default_rng(3)
    for packed in (False, True):
        s = Server(td, 2, 32, 64, tables_for(2, 4, 8, 7), 8)
        shape = (1, 2, 20, 64) if packed else (2, 2, 10, 64)
        k, v = (normal(torch, shape, "f16", 4 + j, dev) for j in range(2))
        positions = rng.integers(0, 2 ** 31 - 1, size=(1, 20) if packed else (2, 10)).tolist()
        s.append(k, v, [10, 10], 64, packed, positions=positions, factors=rng.uniform(1, 8, 32).tolist(), base=500000.0)
        s.check()


def test_borders_of_scales(td):
    """Largest values on, just below and just above 448 powers of two; zeros; the smallest scale."""
    torch, dev = td
    tops = [448.0, 450.0, 446.0, 1.75, 1.7578125, 0.0, 2.0 ** -40, 3.0e38, 2.0 ** -133, 896.0]
    s = Server(td, 1, 16, 16, [[i] for i in range(len(tops))], len(tops))
    k = torch.zeros(len(tops), 1, 2, 16, dtype=torch.bfloat16, device=dev)
    for i, t in enumerate(tops):
        k[i, 0, 0, 3], k[i, 0, 1, 5], k[i, 0, 1, 7] = t, -t, t / 300
    s.append(k, k.clone(), [2] * len(tops), 0, False)
    s.check()
    assert f64(s.ks)[:, 0].tolist() == [osv.scale_for(float(x)) for x in f64(k).reshape(len(tops), -1).max(1)]


def test_every_rounding(td):
    """All f16 values between 0 and 448, each rounded to nearest even."""
    torch, dev = td
    x = torch.arange(0, 0x5f00 + 1, dtype=torch.int16).view(torch.float16)  # 0 .. 448
    x = torch.cat([x, -x]).to(dev)
    x = torch.nn.functional.pad(x, (0, -x.numel() % 128))
    n = x.numel() // 128
    page = 128
    s = Server(td, 1, page, 128, [list(range(-(-n // page)))], -(-n // page))
    rows = x.view(1, 1, n, 128).clone()
    rows[0, 0, ::page, 0] = 448.0  # each page's scale is 1
    s.append(rows, rows.clone(), [n], 0, False)
    s.check()
    assert bool((s.ks == 1).all())


def test_values_that_are_not_finite(td):
    torch, dev = td
    s = Server(td, 2, 16, 32, [[0], [1]], 2)
    k, v = (normal(torch, (2, 2, 5, 32), "bf16", 21 + j, dev) for j in range(2))
    k[0, 0, 2, 4], k[1, 1, 0, 31], v[0, 1, 1, 0], v[1, 0, 4, 7] = float("nan"), float("inf"), -float("inf"), float("nan")
    s.append(k, v, [5, 5], 32, False)
    s.check()
    assert np.isnan(values(s.k)[0, 0, 2, [4, 20]]).all()  # with its partner of the rotation
    assert int(np.isnan(values(s.v)[:, :, :5]).sum()) == 2


@pytest.mark.parametrize("rope", [128, 40])
@pytest.mark.parametrize("page", [48, 128, 256, 1024])
def test_not_finite_in_larger_pages(td, page, rope):
    """Rows that a block holds, in 256 or 512 threads, and more of them; several pages a block."""
    torch, dev = td
    H, D, n = 5, 128, [2100, 900, 7]
    most = 2200 // page + 2
    s = Server(td, H, page, D, tables_for(3, most, 3 * most, 77 + page), 3 * most, "tokens")
    for part, new in enumerate((n, [1, 30, 70])):
        k, v = (normal(torch, (1, H, sum(new), D), "bf16", 61 + 2 * part + j, dev, 4.0 ** part) for j in range(2))
        k[0, 1, 0, 3], k[0, 4, sum(new) - 1, 100] = float("inf"), float("nan")
        v[0, 0, sum(new) // 2, 127], v[0, 3, 0, 0] = -float("inf"), float("inf")
        s.append(k, v, new, rope, True)
        s.check()


def test_rows_that_have_no_place(td):
    """Missing pages, rows before 0 and behind the table are dropped; all other bytes stay."""
    torch, dev = td
    tables = [[3, -1, 5], [7, 1, 2 ** 31 - 1], [0, 8, 4]]
    for packed in (False, True):
        s = Server(td, 2, 16, 64, tables, 8)
        before = s.big.clone()
        s.lens = [40 - 33, 40 - 33, 60 - 33]  # ends: 40 rows, 40, and 60 of 48
        shape = (1, 2, 99, 64) if packed else (3, 2, 33, 64)
        k, v = (normal(torch, shape, "f16", 31 + j, dev) for j in range(2))
        s.append(k, v, [33] * 3, 64, packed)
        s.check()
        for P in (6, 8):
            if P < 8:
                assert torch.equal(s.big[:, P], before[:, P])
        s = Server(td, 2, 16, 64, tables, 8)
        s.lens = [-20, -40, -33]  # 13 rows of 33, none, none
        s.append(k, v, [33] * 3, 64, packed)
        s.check()


def test_sequences_without_rows_and_rows_without_sequence(td):
    torch, dev = td
    s = Server(td, 1, 16, 16, tables_for(4, 3, 12, 9), 12)
    k, v = (normal(torch, (1, 1, 50, 16), "f16", 41 + j, dev) for j in range(2))
    lens = [0, 20, 0, 5]
    s.lens = lens
    cu = ints(torch, [7, 7, 27, 27, 32], dev)  # rows 0 .. 6 and 32 .. 49 belong to nobody
    vef.append_paged(k, v, *s.cache(), cu_seqlens=cu, rope_dims=16)
    for b, (a, n) in enumerate(((7, 0), (7, 20), (27, 0), (27, 5))):
        y, err = osv.rotated(f64(k)[0, :, a:a + n], np.arange(n), 16)
        s.want[0].append(s.tables[b], n, y, err)
        s.want[1].append(s.tables[b], n, f64(v)[0, :, a:a + n], np.zeros((1, n, 16)))
    s.check()
    # values outside the rows are held to them, and what is out of order reads nothing it must not
    for bad in ([-5, 7, 27, 27, 2 ** 31 - 1], [40, 30, 20, 10, 0], [0, 50, 0, 50, 0]):
        vef.append_paged(k, v, *s.cache(), cu_seqlens=ints(torch, bad, dev), rope_dims=16)
    torch.cuda.synchronize(dev)
    assert vef.device_status() == 0


def test_repeated_calls_streams_and_graphs(td):
    """The same call leaves the same bytes; captured and replayed with new lengths and rows."""
    torch, dev = td
    s = Server(td, 2, 32, 64, tables_for(3, 5, 17, 11), 17)
    k, v = (normal(torch, (3, 2, 40, 64), "bf16", 51 + j, dev) for j in range(2))
    s.append(k, v, [40] * 3, 64, False)
    one_k, one_v = (normal(torch, (3, 2, 1, 64), "bf16", 53 + j, dev, 5.0) for j in range(2))
    s.append(one_k, one_v, [1] * 3, 64, False)
    held = [t.clone() for t in (s.big, s.ks, s.vs)]
    cache = s.cache()
    vef.append_paged(one_k, one_v, *cache, rope_dims=64)
    assert all(torch.equal(a, b) for a, b in zip(held, (s.big, s.ks, s.vs)))
    stream = torch.cuda.Stream(dev)
    stream.wait_stream(torch.cuda.current_stream(dev))
    vef.append_paged(one_k, one_v, *cache, rope_dims=64, stream=stream)
    stream.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(held, (s.big, s.ks, s.vs)))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        vef.append_paged(one_k, one_v, *cache, rope_dims=64)
    for step in range(30):
        for x in (one_k, one_v):
            x.copy_(normal(torch, x.shape, "bf16", 60 + step, dev))
        cache[5].add_(1)
        graph.replay()
        s.lens = [n + 1 for n in s.lens]
        for b in range(3):
            y, err = osv.rotated(f64(one_k)[b], [s.lens[b] - 1], 64)
            s.want[0].append(s.tables[b], s.lens[b], y, err)
            s.want[1].append(s.tables[b], s.lens[b], f64(one_v)[b], np.zeros((2, 1, 64)))
    s.check()


def test_many_sequences(td):
    torch, dev = td
    B = 70001
    k, v, big = pool(torch, B, 1, 16, 16, "heads", dev)
    ks, vs = (torch.ones(B, 1, device=dev) for _ in range(2))
    table = torch.randperm(B, generator=torch.Generator().manual_seed(1)).to(torch.int32).view(B, 1).to(dev)
    x = normal(torch, (B, 1, 2, 16), "f16", 71, dev)
    lens = torch.full((B,), 2, dtype=torch.int32, device=dev)
    vef.append_paged(x, x, k, v, ks, vs, table, lens, rope_dims=16)
    packed = x.transpose(0, 1).reshape(1, 1, 2 * B, 16)
    k2, v2, big2 = pool(torch, B, 1, 16, 16, "heads", dev)
    ks2, vs2 = (torch.ones(B, 1, device=dev) for _ in range(2))
    cu = torch.arange(0, 2 * B + 1, 2, dtype=torch.int32, device=dev)
    vef.append_paged(packed, packed, k2, v2, ks2, vs2, table, lens, cu_seqlens=cu, rope_dims=16)
    assert torch.equal(big, big2) and torch.equal(ks, ks2) and torch.equal(vs, vs2)
    for b in (0, 32767, 65535, 65536, B - 1):
        want = osv.Cache(np.zeros((1, 1, 16, 16)), np.ones((1, 1)))
        want.append([0], 2, f64(x)[b], np.zeros((1, 2, 16)))
        P = int(table[b, 0])
        assert np.array_equal(values(v[P:P + 1])[:, :, :2], want.lo[:, :, :2])


def test_far_pages(td):
    """Pages and rows further apart than 32 bits of bytes reach."""
    torch, dev = td
    if torch.cuda.mem_get_info(dev)[0] < 24 << 30:
        pytest.skip("needs 24 GB of free device memory")
    n, stride = 6, 1 << 31
    big = torch.zeros(n * stride, dtype=torch.uint8, device=dev)
    f8 = torch.float8_e4m3fn
    k, v = (big.as_strided((n, 1, 16, 64), (stride, 64, 64, 1), 1024 * i).view(f8) for i in range(2))
    ck, cv, _ = pool(torch, n, 1, 16, 64, "heads", dev, fill=0)
    table = ints(torch, [[5, 0, 3]], dev)
    scales = [torch.ones(n, 1, device=dev) for _ in range(4)]
    x, y = (normal(torch, (1, 1, 45, 64), "f16", 81 + j, dev) for j in range(2))
    lens = ints(torch, [45], dev)
    vef.append_paged(x, y, k, v, scales[0], scales[1], table, lens, rope_dims=64)
    vef.append_paged(x, y, ck, cv, scales[2], scales[3], table, lens, rope_dims=64)
    assert torch.equal(k.view(torch.uint8), ck.view(torch.uint8)) and torch.equal(v.view(torch.uint8), cv.view(torch.uint8))
    q = normal(torch, (1, 3, 5, 64), "f16", 83, dev)
    assert torch.equal(vef.forward_paged(q, k, v, scales[0], scales[1], table, lens),
                       vef.forward_paged(q, ck, cv, scales[2], scales[3], table, lens))
    del big
    torch.cuda.empty_cache()


def test_refusals(td):
    torch, dev = td
    k, v, _ = pool(torch, 4, 2, 16, 64, "heads", dev)
    ks, vs = (torch.ones(4, 2, device=dev) for _ in range(2))
    table, lens = ints(torch, [[0, 1]], dev), ints(torch, [5], dev)
    x = normal(torch, (1, 2, 5, 64), "f16", 91, dev)
    call = lambda *a, **kw: vef.append_paged(*a, **kw)
    call(x, x, k, v, ks, vs, table, lens)
    for bad in ((x.float(), x.float(), k, v, ks, vs, table, lens), (x, x.bfloat16(), k, v, ks, vs, table, lens),
                (x, x, k.float(), v, ks, vs, table, lens), (x, x, k, v, ks.half(), vs, table, lens),
                (x, x, k, v, ks, vs, table.long(), lens), (x, x, k, v, ks, vs, table, None)):
        with pytest.raises(TypeError):
            call(*bad)
    for bad in ((x[:, :1], x[:, :1], k, v, ks, vs, table, lens), (x, x[:, :, :4], k, v, ks, vs, table, lens),
                (x, x, k, v[:3], ks, vs, table, lens), (x, x, k, v, ks[:3], vs, table, lens),
                (x, x, k, v, ks, vs, table, ints(torch, [5, 5], dev)), (x, x, k, v, ks, vs, table.cpu(), lens),
                (x, x, k[..., :48], v, ks, vs, table, lens)):
        with pytest.raises(ValueError):
            call(*bad)
    with pytest.raises(vef.VattnError):
        call(x, x, k, k, ks, vs, table, lens)
    with pytest.raises(vef.VattnError):
        call(x, x, k, v, ks, ks, table, lens)
    with pytest.raises(vef.VattnError):
        call(x, x, k[:1].expand(4, 2, 16, 64), v, ks, vs, table, lens)  # pages that share addresses
    with pytest.raises(vef.VattnError):
        call(x, x, k, v, ks, vs, table, lens, rope_dims=65)
    with pytest.raises(ValueError):
        call(x, x, k, v, ks, vs, table, lens, positions=ints(torch, [[1, 2]], dev))
    with pytest.raises(ValueError):
        call(x.expand(2, 2, 5, 64), x.expand(2, 2, 5, 64), k, v, ks, vs, table, lens, cu_seqlens=ints(torch, [0, 5], dev))
