"""GPU tests of trees whose words name tokens that see nothing themselves: such a
token is at the position before the new ones, which a window may leave out."""
import pytest

import vision_encoder_flash_gb300 as vef
from test_paged_gpu import against_the_oracle, build, signed, td  # noqa: F401

pytestmark = pytest.mark.gpu

WORDS = [
    [0b0001, 0b0000, 0b0110, 0b1010],   # the third and the last see the second, which sees nothing
    [0b0000, 0b0001, 0b0101, 0b1111],   # the first sees nothing, all others see it
    [0b0010, 0b0000, 0b0010, 0b0010],   # nobody sees itself
]


@pytest.mark.parametrize("window", [None, 1, 2, 3, 4, 50])
@pytest.mark.parametrize("i", range(len(WORDS)))
def test_words_that_name_tokens_without_bits(td, i, window):  # noqa: F811
    torch, dev = td
    for sinks, lens in ((0, [90, 4]), (7, [33, 5]), (200, [60, 6])):
        case = ("f16", (2, 6, 2, 4, 64), 16, lens, window, sinks, False, "heads", "plain")
        q, cache, _, how = build(td, case, 2300 + i)
        words = [WORDS[i]] * 2
        how["tree_mask"] = torch.tensor([signed(w) for w in words], dtype=torch.int64, device=dev)
        out = vef.forward_paged(q, *cache, **how)
        against_the_oracle(out, q, cache, window, sinks, words, how["scale"], "f16", f"first keys {sinks}")
    assert vef.device_status() == 0
