"""GPU tests of attention over the paged cache at the ends of the ranges that its
call admits: queries near bf16's largest, against the f64 oracle."""
import pytest

import vision_encoder_flash_gb300 as vef
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
