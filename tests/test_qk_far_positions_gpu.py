"""The rotation at the ends of the positions, with divisors and bases that make
the angles larger still, against angles of 60 digits."""
from decimal import Decimal, getcontext

import numpy as np
import pytest

from oracle import decoder as od
import vision_encoder_flash_gb300 as vef
from decoder_util import assert_within, f64

pytestmark = pytest.mark.gpu

PI = Decimal("3.14159265358979323846264338327950288419716939937510582097494459230781640628620899862803")


def reduced(positions, rope_dims, base, factors):
    """The angles modulo 2 pi, in f64."""
    getcontext().prec = 60
    out = np.zeros((len(positions), rope_dims // 2))
    for i in range(rope_dims // 2):
        f = (Decimal(base).ln() * Decimal(-2 * i) / Decimal(rope_dims)).exp()
        if factors is not None:
            f /= Decimal(float(factors[i]))
        for n, p in enumerate(positions):
            out[n, i] = float((Decimal(p) * f) % (2 * PI))
    return out


@pytest.mark.parametrize("base,factor", [(10000.0, None), (10000.0, 1 / 64.0), (500000.0, 0.3), (1e6, -0.01), (0.001, None),
                                         (3.0, 7.0), (1e-4, 0.125)])
@pytest.mark.parametrize("dim,rope", [(8, 8), (48, 48), (8, 6)])
def test_far_positions(dim, rope, base, factor):
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    dev = torch.device("cuda", 0)
    positions = [0, 1, 12345, 10 ** 6 + 1, 2 ** 24 + 1, 10 ** 9 + 7, 2 ** 30 + 5, 2 ** 31 - 2, 2 ** 31 - 1, -1, -(10 ** 6)]
    n = len(positions)
    x = torch.from_numpy(np.random.default_rng(dim).normal(size=(1, 2, n, dim))).float().to(dev)
    g = torch.from_numpy(np.random.default_rng(dim + 1).normal(size=(1, 2, n, dim))).float().to(dev)
    at = torch.tensor([positions], dtype=torch.int32, device=dev)
    factors = None if factor is None else torch.tensor([factor * (1 + i % 3) for i in range(rope // 2)], device=dev)
    how = dict(rope_dims=rope, positions=at, base=base, factors=factors)
    theta = reduced(positions, rope, base, None if factors is None else f64(factors))
    got, _ = vef.qk_norm_rope(x, x[:, :1], **how)
    a = f64(x)
    y = a / np.sqrt((a * a).mean(-1, keepdims=True) + float(np.float32(1e-6)))
    want = od.turn(y, theta[None, None])
    half = rope // 2
    pair = np.abs(y[..., :half]) + np.abs(y[..., half:2 * half])
    size = np.concatenate([pair, pair, np.abs(y[..., 2 * half:])], -1)
    # the row's sum and root, the products and the turn, and the angle: sine and cosine to 1.3 2^-24
    # of an angle within 2^-31 turns (2^-28 radians)
    assert_within(got, want, (dim / 2 + 16) * od.F32 * size, "out", u=od.F32)
    # its transpose, from the gradient
    dx, _, _, _ = vef.qk_norm_rope_backward(g, g[:, :1], x, x[:, :1], **how)
    r = 1 / np.sqrt((a * a).mean(-1, keepdims=True) + float(np.float32(1e-6)))
    gy = od.turn(f64(g), theta[None, None], inverse=True)
    back = r * gy - a * r ** 3 / dim * (gy * a).sum(-1, keepdims=True)
    pg = np.abs(f64(g))
    pair = pg[..., :half] + pg[..., half:2 * half]
    size = np.concatenate([pair, pair, pg[..., 2 * half:]], -1)
    bound = (1.5 * dim + 32) * od.F32 * (r * size + np.abs(a) * r ** 3 / dim * (size * np.abs(a)).sum(-1, keepdims=True))
    assert_within(dx, back, bound, "dx", u=od.F32)
