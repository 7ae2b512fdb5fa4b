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


def zeros_for(torch, cache, pages, pools=(0, 1)):
    """What the cache stands for where these pages' scales are 0: bytes of zeros, in units of the smallest
    scale that is not."""
    out = [t.clone() for t in cache]
    for i in pools:
        out[i].view(torch.uint8)[pages] = 0
        left = out[2 + i][out[2 + i] > 0]
        out[2 + i][pages] = float(left.min()) if left.numel() else 1.0
    return out


@pytest.mark.parametrize("name,exponent", [("f16", -6), ("bf16", -6), ("bf16", -90), ("bf16", 0)])
@pytest.mark.parametrize("H,T,D", [(1, 1, 64), (8, 2, 128), (4, 5, 80), (4, 8, 32), (4, 11, 64), (8, 7, 128), (5, 20, 96)])
def test_pages_whose_scale_is_zero(td, name, exponent, H, T, D):  # noqa: F811
    """Scales of 0 in both pools, or in one: zeros whatever the bytes (of values, NaN among them), beside pages whose
    scales are near 1 or far from it; first, in between and last; and a NaN of another page in the same step."""
    torch, dev = td
    for page, lens in ((16, [300, 90]), (64, [2500, 700])):
        case = (name, (2, 2 * H, 2, T, D), page, lens, None, 0, False, "heads", "plain")
        q, cache, _, how = build(td, case, 2100 + T)
        cache[3] *= 2.0 ** exponent
        last = [(n - 1) // page for n in lens]
        gone = torch.cat([cache[4][0, [0, 1, 2, last[0]]], cache[4][1, [1, last[1]]]]).long()
        for pools in ((0, 1), (1,), (0,)):
            zero = [t.clone() for t in cache]
            for i in pools:
                zero[i].view(torch.uint8)[gone] = torch.randint(0, 0x7f, (1,) + zero[i].shape[1:], dtype=torch.uint8, device=dev)
                if i == 1:
                    zero[i].view(torch.uint8)[gone, :, 3] = 0x7f
                zero[2 + i][gone] = 0
            want = zeros_for(torch, cache, gone, pools)
            out = vef.forward_paged(q, *zero, **how)
            against_the_oracle(out, q, want, None, 0, None, how["scale"], name, f"pools {pools}, pages of {page}")
        # a NaN in the last token's value: in the rows that see it alone, in a step that holds a page of zeros
        P, row = int(cache[4][0, last[0] - 1]), page - 1
        n = last[0] * page  # rows in use now: up to that one
        zero[5] = ints(torch, [n, lens[1]], dev)
        zero[3][gone] = 0
        zero[1].view(torch.uint8)[gone, :, 5] = 0x7f
        want = zeros_for(torch, cache, gone) if 0 in pools else zeros_for(torch, cache, gone, (1,))
        want[5] = zero[5]
        clean = vef.forward_paged(q, *zero, **how)
        against_the_oracle(clean, q, want, None, 0, None, how["scale"], name, f"{n} rows")
        zero[1].view(torch.uint8)[P, 0, row, 7] = 0xff
        out = vef.forward_paged(q, *zero, **how)
        bad = torch.isnan(out)
        assert bool(bad[0, :H, T - 1, 7].all()) and int(bad.sum()) == H
        against_the_oracle(torch.where(bad, clean, out), q, want, None, 0, None, how["scale"], name, f"{n} rows, a NaN")
    assert vef.device_status() == 0


@pytest.mark.parametrize("name", ["f16", "bf16"])
def test_all_scales_zero(td, name):  # noqa: F811
    """Every visible page of values in units of 0: zeros exactly."""
    torch, dev = td
    for T, lens in ((1, [3000]), (3, [100]), (9, [700])):
        case = (name, (1, 8, 2, T, 64), 16, lens, None, 0, False, "tokens", "plain")
        q, cache, _, how = build(td, case, 2200 + T)
        cache[1].view(torch.uint8)[:, :, 2] = 0x7f
        cache[3].zero_()
        assert not bool(vef.forward_paged(q, *cache, **how).any())
        assert not bool(torch.isnan(vef.forward_paged(q, *cache, **how)).any())
