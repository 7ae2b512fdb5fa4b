"""Limits of the decoder calls' sizes that no tensor of a test has: refused on
the host, before any CUDA call (no GPU needed)."""
import pytest

from test_decoder_abi import FAKE, G, backward, cached, lib, win_args, window  # noqa: F401


@pytest.mark.parametrize("kw", [dict(hq=0, hk=2 ** 32 + 1), dict(hq=0, hk=2 ** 30), dict(batch=2, hq=0, hk=2 ** 29),
                                dict(batch=2 ** 15, hq=0, hk=2 ** 15)])
def test_key_heads_without_query_heads(lib, kw):  # noqa: F811
    """No query head limits their number: it has to fit 30 bits by itself."""
    assert window(lib, win_args(**kw)) == 2
    assert backward(lib, win_args(**kw)) == 2
    assert cached(lib, win_args(**{"kv_len": FAKE + 30 * G, **kw})) == 2
    assert "n_kv_heads" in lib.vattn_last_error_string().decode()
