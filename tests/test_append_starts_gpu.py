"""GPU tests of appends of packed rows whose starts do not ascend or lie outside
the rows, and of the bytes that no append may touch."""
import numpy as np
import pytest

from oracle import serving as osv
import vision_encoder_flash_gb300 as vef
from decoder_util import f64, normal
from serving_util import ints
from test_append_paged_gpu import Server, tables_for, td  # noqa: F401

pytestmark = pytest.mark.gpu


def held(cu, total):
    """(first row, rows) of each sequence, starts held to [0, total]; none where they are too many together."""
    at = [min(max(c, 0), total) for c in cu]
    parts = [(a, max(0, b - a)) for a, b in zip(at, at[1:])]
    return parts if sum(n for _, n in parts) <= total else [(a, 0) for a, _ in parts]


STARTS = [
    [0, 17, 17, 60, 90, 100],             # as they should be
    [-5, 7, 27, 27, 2 ** 31 - 1],         # held to the rows
    [0, 50, 0, 50, 0],                    # 100 rows of 100
    [0, 100, 60, 60],                     # one that ends before it begins, behind one that touches all its pages
    [0, 50, 40, 50, 30, 40],              # overlaps, 70 rows
    [40, 30, 20, 10, 0],                  # all end before they begin
    [2 ** 31 - 1, -2 ** 31, 60],          # such, held to the rows
    [0, 100, 0, 100],                     # more than there are: nothing
    [100, 0, 1] + [0, 1] * 49,            # fifty of one row
    [0] * 40 + [100, 90, 95],             # beyond 32 sequences
    [0, 100] * 40,                        # such, more than there are
    [60, 0, 60, 0] + [0] * 60 + [30],     # the last of many
]


@pytest.mark.parametrize("page", [16, 48])
@pytest.mark.parametrize("i", range(len(STARTS)))
def test_starts(td, i, page):  # noqa: F811
    """Every byte and scale against the oracle, for starts in any order."""
    torch, dev = td
    cu, total = STARTS[i], 100
    B, H, D = len(cu) - 1, 2, 64
    most = 160 // page + 2
    s = Server(td, H, page, D, tables_for(B, most, B * most + 1, 30 + i), B * most + 1)
    k, v = (normal(torch, (1, H, total, D), "bf16", 300 + 2 * i + j, dev) for j in range(2))
    parts = held(cu, total)
    s.lens = [n + (15 + 13 * b) % 40 for b, (_, n) in enumerate(parts)]  # some into pages begun before
    untouched = [t.clone() for t in (s.big, s.ks, s.vs)]
    vef.append_paged(k, v, *s.cache(), cu_seqlens=ints(torch, cu, dev), rope_dims=D)
    kn, vn = f64(k), f64(v)
    for b, (a, n) in enumerate(parts):
        if n:
            y, err = osv.rotated(kn[0, :, a:a + n], np.arange(s.lens[b] - n, s.lens[b]), D)
            s.want[0].append(s.tables[b], s.lens[b], y, err)
            s.want[1].append(s.tables[b], s.lens[b], vn[0, :, a:a + n], np.zeros((H, n, D)))
    s.check()
    if not any(n for _, n in parts):
        assert all(torch.equal(a, b) for a, b in zip(untouched, (s.big, s.ks, s.vs)))


@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("page,D,rope", [(16, 64, 64), (48, 80, 40), (256, 128, 128), (16, 48, 7)])
def test_bytes_that_no_append_touches(td, page, D, rope, packed):  # noqa: F811
    """Rows before and behind the new ones, other pages, padding and other scales: the same bytes."""
    torch, dev = td
    B, H, T = 3, 2, 37
    most = 120 // page + 2
    s = Server(td, H, page, D, tables_for(B, most, B * most + 3, 5), B * most + 3, "both")
    s.big.copy_(torch.randint(0, 256, s.big.shape, dtype=torch.uint8, device=dev))
    s.ks.fill_(64.0)  # more than the new values need: rows before them keep their bytes
    s.vs.fill_(64.0)
    s.lens = [37 + 20, 37 + 3, 37 + 61]
    shape = (1, H, B * T, D) if packed else (B, H, T, D)
    k, v = (normal(torch, shape, "bf16", 400 + j, dev) for j in range(2))
    before = [t.clone() for t in (s.big, s.ks, s.vs)]
    cu = ints(torch, [0, T, 2 * T, 3 * T], dev) if packed else None
    vef.append_paged(k, v, *s.cache(), cu_seqlens=cu, rope_dims=rope)
    same = torch.ones(s.big.shape[:2], dtype=torch.bool, device=dev)  # [page, row]
    anew = torch.zeros(s.big.shape[0], dtype=torch.bool, device=dev)
    for b, n in enumerate(s.lens):
        for r in range(n - T, n):
            same[s.tables[b][r // page], r % page] = False
            anew[s.tables[b][r // page]] |= r % page == 0
    assert torch.equal(s.big[same], before[0][same])
    assert torch.equal(s.big[..., D:], before[0][..., D:])
    for now, was in ((s.ks, before[1]), (s.vs, before[2])):
        assert torch.equal(now[~anew], was[~anew]) and bool((now[anew] < 1).all())
