"""GPU tests of attention over the paged cache at the ends of the ranges that its
call admits: queries near bf16's largest, scales of values far from 1, against
the f64 oracle."""
import numpy as np
import pytest

import vision_encoder_flash_gb300 as vef
from decoder_util import dtype
from serving_util import ints
from test_paged_gpu import against_the_oracle, build, td  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("power", [125, 126, 127])
def test_queries_near_the_largest(td, power):  # noqa: F811
    """bf16 rows whose largest element is 2^power and more, up to bf16's largest."""
    torch, dev = td
    case = ("bf16", (2, 4, 1, 3, 64), 16, [100, 37], None, 0, False, "heads", "plain")
    q, cache, _, _ = build(td, case, 2000 + power)
    x = q.float()
    x = (x / x.abs().amax(-1, keepdim=True) * (2.0 - 2.0 ** -7)).to(torch.bfloat16)  # each row's largest: all bits set
    q = (x.double() * 2.0 ** power).to(torch.bfloat16)
    assert bool(torch.isfinite(q).all()) and float(q.float().abs().amax(-1).min()) >= 2.0 ** power
    scale = 2.0 ** -(power - 1)
    out = vef.forward_paged(q, *cache, scale=scale)
    against_the_oracle(out, q, cache, None, 0, None, scale, "bf16")
    assert vef.device_status() == 0


def far_scales(td, name, exponent, lens, heads, D=16, page=64):
    """A cache whose first 128 keys score 7.75 log2 units below the others, its pages shared by all of
    its sequences, with values in units of 2^exponent; and q, scale for it."""
    torch, dev = td
    most = -(-max(lens) // page)
    k = torch.zeros(most, 1, page, D, dtype=torch.uint8, device=dev)
    k[128 // page:, :, :, 0] = 0x38                                  # ones
    g = torch.Generator(device=dev).manual_seed(9)
    v = (torch.randn(most, 1, page, D, generator=g, device=dev) * 100).clamp(-440, 440).to(torch.float8_e4m3fn)
    ks, vs = torch.ones(most, 1, device=dev), torch.full((most, 1), 2.0 ** exponent, device=dev)
    table = torch.arange(most, dtype=torch.int32, device=dev).repeat(len(lens), 1)
    q = torch.zeros(len(lens), heads, 1, D, dtype=dtype(torch, name), device=dev)
    q[..., 0] = 1.0
    return q, [k.view(torch.float8_e4m3fn), v, ks, vs, table, ints(torch, lens, dev)], 7.75 * float(np.log(2.0))


@pytest.mark.parametrize("exponent", [-100, 100])
@pytest.mark.parametrize("n_seqs", [1, 40, 320])
def test_scales_of_values_at_both_ends(td, n_seqs, exponent):  # noqa: F811
    """Sums of weights over the smallest and the largest scales, whose first keys count least: in one share
    of the keys, a few and many."""
    torch, dev = td
    lens = [32768 - 11 * b for b in range(n_seqs)]
    q, cache, scale = far_scales(td, "bf16", exponent, lens, 3)
    out = vef.forward_paged(q, *cache, scale=scale)
    for b in {0, n_seqs // 2, n_seqs - 1}:
        s = slice(b, b + 1)
        against_the_oracle(out[s], q[s], cache[:4] + [cache[4][s], cache[5][s]], None, 0, None, scale, "bf16", f"sequence {b}")
    assert bool(out.any(-1).all())
    assert vef.device_status() == 0
