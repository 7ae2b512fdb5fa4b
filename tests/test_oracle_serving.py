"""The serving oracle: roundings against torch's own conversion, scales."""
import numpy as np
import pytest

from oracle import serving as osv


def test_every_byte_rounds_to_itself_and_midpoints_to_even():
    torch = pytest.importorskip("torch")
    all_bytes = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).float().numpy()
    want = np.where(np.isnan(all_bytes), np.nan, all_bytes)
    assert np.array_equal(osv.e4m3_round(want), want, equal_nan=True)
    values = np.sort(want[np.isfinite(want)])
    middles = (values[1:] + values[:-1]) / 2
    got = osv.e4m3_round(middles)
    assert np.array_equal(got, torch.from_numpy(middles).float().to(torch.float8_e4m3fn).float().numpy())
    x = np.random.default_rng(1).normal(size=20000) * 10.0 ** np.random.default_rng(2).uniform(-4, 2, 20000)
    x = np.clip(x.astype(np.float32), -448, 448)
    assert np.array_equal(osv.e4m3_round(x), torch.from_numpy(x).to(torch.float8_e4m3fn).float().numpy())


@pytest.mark.parametrize("most,exponent", [(0.0, -32), (448.0, 0), (448.0001, 1), (224.0, -1), (224.1, 0), (1.75, -8),
                                           (1.0, -8), (1.7500001, -7), (2.0 ** -100, -32), (3e38, 120)])
def test_scales(most, exponent):
    assert osv.scale_for(most) == 2.0 ** exponent
    assert most <= 448 * osv.scale_for(most)


def test_append_grows_a_page():
    c = osv.Cache(np.zeros((2, 1, 16, 16)), np.ones((2, 1)))
    zero = np.zeros((1, 3, 16))
    c.append([1, 0], 3, np.full((1, 3, 16), 1.0), zero)          # row 0 of page 1: a new scale
    assert c.scale[1, 0] == 2.0 ** -8 and (c.lo[1, 0, :3] == 256).all() and c.scale[0, 0] == 1
    c.append([1, 0], 17, np.full((1, 14, 16), 7.0), np.zeros((1, 14, 16)))
    assert c.scale[1, 0] == 2.0 ** -6 and (c.lo[1, 0, :3] == 64).all() and (c.lo[1, 0, 3:] == 448).all()
    assert c.scale[0, 0] == 2.0 ** -6 and (c.lo[0, 0, 0] == 448).all() and not c.lo[0, 0, 1:].any()
