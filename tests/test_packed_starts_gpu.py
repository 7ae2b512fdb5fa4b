"""GPU tests of packed prompts whose starts hold anything: the work that they make
is bounded by the rows that there are."""
import pytest

import vision_encoder_flash_gb300 as vef
from test_packed_gpu import rows, td  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n_seqs", [300, 5000, 1 << 20])
def test_prompts_of_all_rows_again_and_again(td, n_seqs):  # noqa: F811
    """Every other prompt has all rows: none is computed, and the list of them ends with the first that are too many."""
    torch, dev = td
    total = 100000
    q, k, v = rows(td, "f16", (8, 1), total, 8, 4900, "packed")
    out = torch.full_like(q, 7.0)
    cu = torch.zeros(n_seqs + 1, dtype=torch.int32, device=dev)
    cu[1::2] = total
    vef.forward_packed(q, k, v, cu, scale=0.3, out=out)
    assert bool((out == 7).all())
    assert vef.device_status() == 0


@pytest.mark.parametrize("n_seqs", [300, 5000])
def test_any_starts(td, n_seqs):  # noqa: F811
    """Starts from everywhere: either too many rows together, and nothing is computed, or each prompt as if alone."""
    torch, dev = td
    total = 20000
    q, k, v = rows(td, "bf16", (2, 1), total, 16, 4910, "packed")
    out = torch.full_like(q, 7.0)
    g = torch.Generator().manual_seed(n_seqs)
    cu = torch.randint(-2 ** 31, 2 ** 31 - 1, (n_seqs + 1,), generator=g, dtype=torch.int64).to(torch.int32).to(dev)
    vef.forward_packed(q, k, v, cu, scale=0.3, out=out)
    assert bool((out == 7).all())
    # descending but for one step up
    cu = torch.arange(n_seqs, -1, -1, dtype=torch.int32, device=dev)
    cu[n_seqs // 2] = total
    lo = int(cu[n_seqs // 2 - 1])
    vef.forward_packed(q, k, v, cu, scale=0.3, out=out)
    part = [x[:, :, lo:].contiguous() for x in (q, k, v)]
    assert torch.equal(out[:, :, lo:], vef.forward_window(*part, scale=0.3))
    assert bool((out[:, :, :lo] == 7).all())
    assert vef.device_status() == 0
