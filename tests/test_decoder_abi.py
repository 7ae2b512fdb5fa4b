"""The decoder calls are exported as declared and refuse bad arguments on the
host, before any CUDA call (no GPU needed)."""
import subprocess

import pytest

import vision_encoder_flash_gb300 as vef
from vision_encoder_flash_gb300 import _lib, decoder

G = 2 ** 30
FAKE = 16 * G  # never dereferenced: every refusal comes before any CUDA call


@pytest.fixture(scope="module")
def lib():
    from vision_encoder_flash_gb300 import build
    build.build()
    return vef.load_library()


def test_exports_every_declared_symbol(lib):
    names = [n for n in _lib.exported_symbols(_lib.DECODER_HEADER)]
    assert set(names) == {"vattn_qk_norm_rope", "vattn_qk_norm_rope_backward", "vattn_forward_window",
                          "vattn_backward_window", "vattn_forward_cached"}
    out = subprocess.run(["nm", "-D", "--defined-only", _lib.lib_path()], capture_output=True, text=True,
                         check=True).stdout
    for name in names:
        assert f" T {name}\n" in out and hasattr(vef, name[len("vattn_"):]), name


def rows(i, heads=2, n=16, dim=64, off=0, strides=None):
    """vattn_rows of the i-th of some buffers 1 GB apart."""
    return decoder._ROWS(FAKE + i * G + off, *(strides or (heads * n * dim, n * dim, dim)))


def qk_args(batch=1, hq=2, hk=2, n=16, dim=64, rope=64, pos0=0, positions=0, factors=0, wq=0, wk=0, base=1e4,
            eps=1e-6, dtype=2, wdtype=0):
    return decoder._QK(batch, hq, hk, n, dim, rope, pos0, positions, factors, wq, wk, base, eps, dtype, wdtype)


def qk(lib, args=None, q=None, k=None, qo=None, ko=None):
    s = lib.vattn_qk_norm_rope(q or rows(0), k or rows(1), qo or rows(2), ko or rows(3), args or qk_args(), 0)
    assert s == 0 or lib.vattn_last_error_string().decode() != ""
    return s


NAN, INF = float("nan"), float("inf")


@pytest.mark.parametrize("kw,status", [
    (dict(batch=-1), 1), (dict(hq=-1), 1), (dict(n=-5), 1), (dict(dim=0), 1), (dict(dim=129), 2), (dict(rope=65), 1),
    (dict(rope=-1), 1), (dict(base=0.0), 1), (dict(base=INF), 1), (dict(base=NAN), 1), (dict(eps=-1e-6), 1),
    (dict(eps=NAN), 1), (dict(dtype=3), 1), (dict(dtype=-1), 1), (dict(wdtype=1), 2), (dict(n=2 ** 30), 2),
    (dict(batch=2 ** 30), 2), (dict(pos0=-1), 1), (dict(pos0=2 ** 31 - 16), 2), (dict(positions=FAKE + 2), 3),
    (dict(factors=FAKE + 1), 3), (dict(wq=FAKE + 2), 3),
])
def test_qk_refuses_sizes_and_numbers(lib, kw, status):
    assert qk(lib, qk_args(**kw)) == status
    r = [rows(i) for i in range(6)]
    assert lib.vattn_qk_norm_rope_backward(*r, 0, 0, qk_args(**kw), 0) == status


def test_qk_refuses_tensors(lib):
    assert qk(lib, q=decoder._ROWS(0, 1, 1, 1)) == 1
    assert qk(lib, q=rows(0, off=1)) == 3
    assert qk(lib, qo=rows(0, off=64)) == 1                       # over q, not q itself
    assert qk(lib, qo=rows(1)) == 1 and qk(lib, ko=rows(0)) == 1  # over the other input
    assert qk(lib, qo=rows(2), ko=rows(2)) == 1
    assert qk(lib, qo=rows(2, strides=(0, 0, 64))) == 1           # heads of the result share addresses
    assert qk(lib, qo=rows(2, strides=(2048, 64, 32))) == 1
    assert qk(lib, q=rows(0, strides=(2048, -1024, 64))) == 1
    assert qk(lib, q=rows(0, strides=(2048, 2 ** 40, 64))) == 2
    # heads of one packed buffer [1, 16, heads, 64]: k's first head inside q's
    packed = (16 * 4 * 64, 64, 4 * 64)
    assert qk(lib, qo=rows(2, strides=packed), ko=rows(2, off=64 * 2, strides=packed)) == 1
    r = [rows(i) for i in range(6)]
    args = qk_args(wq=FAKE + 10 * G, wk=FAKE + 11 * G)
    assert lib.vattn_qk_norm_rope_backward(*r, FAKE + 12 * G + 2, 0, args, 0) == 3
    assert lib.vattn_qk_norm_rope_backward(*r, FAKE + 4 * G, 0, args, 0) == 1
    assert lib.vattn_qk_norm_rope_backward(*r, FAKE + 12 * G, FAKE + 12 * G + 128, args, 0) == 1


def test_empty_qk_is_a_no_op(lib):
    for kw in (dict(batch=0), dict(n=0), dict(hq=0, hk=0)):
        assert qk(lib, qk_args(**kw)) == 0


def win_args(batch=1, hq=4, hk=2, m=16, n=16, dim=64, window=0, sinks=0, kv_len=0, q_start=0, tree=0, scale=1.0,
             dtype=1):
    return decoder._WINDOW(batch, hq, hk, m, n, dim, window, sinks, kv_len, q_start, tree, scale, dtype)


def window(lib, args=None, q=None, k=None, v=None, out=None, lse=0):
    s = lib.vattn_forward_window(q or rows(0, 4), k or rows(1), v or rows(2), out or rows(3, 4), lse,
                                 args or win_args(), 0)
    assert s == 0 or lib.vattn_last_error_string().decode() != ""
    return s


def backward(lib, args=None, **kw):
    heads = dict(dout=4, q=4, k=2, v=2, out=4, dq=4, dk=2, dv=2)
    r = {n: kw.get(n) or rows(i, h) for i, (n, h) in enumerate(heads.items())}
    s = lib.vattn_backward_window(r["dout"], r["q"], r["k"], r["v"], r["out"], kw.get("lse", FAKE + 20 * G),
                                  r["dq"], r["dk"], r["dv"], args or win_args(), 0)
    assert s == 0 or lib.vattn_last_error_string().decode() != ""
    return s


def cached(lib, args=None, q=None, k=None, v=None, out=None):
    s = lib.vattn_forward_cached(q or rows(0, 4), k or rows(1), v or rows(2), out or rows(3, 4),
                                 args or win_args(kv_len=FAKE + 30 * G), 0)
    assert s == 0 or lib.vattn_last_error_string().decode() != ""
    return s


@pytest.mark.parametrize("kw,status", [
    (dict(batch=-1), 1), (dict(hq=-4), 1), (dict(m=-1), 1), (dict(n=-1), 1), (dict(dim=0), 1), (dict(dim=136), 2),
    (dict(dim=60), 2), (dict(dtype=0), 2), (dict(dtype=7), 2), (dict(hq=3), 1), (dict(hk=0), 1), (dict(n=2 ** 30), 2),
    (dict(batch=2 ** 29), 2), (dict(window=-1), 1), (dict(sinks=-1), 1), (dict(scale=0.0), 1), (dict(scale=-1.0), 1),
    (dict(scale=NAN), 1), (dict(scale=INF), 1), (dict(kv_len=FAKE + 2), 3), (dict(tree=FAKE + 4), 3),
])
def test_attention_refuses_sizes_and_numbers(lib, kw, status):
    assert window(lib, win_args(**kw)) == status
    assert backward(lib, win_args(**kw)) == status
    assert cached(lib, win_args(**{"kv_len": FAKE + 30 * G, **kw})) == status


def test_attention_refuses_what_belongs_to_another_call(lib):
    assert window(lib, win_args(tree=FAKE)) == 1 and backward(lib, win_args(tree=FAKE)) == 1
    assert cached(lib, win_args(kv_len=FAKE, q_start=FAKE)) == 1
    assert cached(lib, win_args(kv_len=0)) == 1
    assert cached(lib, win_args(kv_len=FAKE, m=65)) == 2


def test_attention_refuses_tensors(lib):
    null = decoder._ROWS(0, 1024, 1024, 64)
    for call in (window, cached):
        assert call(lib, q=null) == 1 and call(lib, v=null) == 1 and call(lib, out=null) == 1
        assert call(lib, q=rows(0, 4, off=8)) == 3                       # not on 16 bytes
        assert call(lib, k=rows(1, strides=(2048, 1024, 68))) == 3        # nor are its rows
        assert call(lib, out=rows(0, 4)) == 1 and call(lib, out=rows(1, 4, off=1024)) == 1
        assert call(lib, out=rows(3, 4, strides=(4096, 0, 64))) == 1
        assert call(lib, k=rows(1, strides=(2048, -1024, 64))) == 1
    assert window(lib, lse=FAKE + 3 * G + 64) == 1 and window(lib, lse=FAKE + 9 * G + 2) == 3
    assert backward(lib, lse=0) == 1 and backward(lib, lse=FAKE + 6 * G) == 1
    assert backward(lib, dq=rows(1, 4)) == 1 and backward(lib, dk=rows(2)) == 1 and backward(lib, dv=rows(6)) == 1
    assert backward(lib, dk=rows(6, strides=(0, 0, 64))) == 1


def test_window_refuses_rows_that_share_addresses(lib):
    for stride in (0, 56):
        for call, name, h in ((window, "q", 4), (window, "k", 2), (window, "v", 2), (backward, "dout", 4),
                              (backward, "q", 4), (backward, "k", 2), (backward, "v", 2)):
            i = dict(q=0, k=1, v=2)[name] if call is window else dict(dout=0, q=1, k=2, v=3)[name]
            assert call(lib, **{name: rows(i, h, strides=(h * 1024, 1024, stride))}) == 2
            assert "row stride" in lib.vattn_last_error_string().decode()


def test_empty_attention_is_a_no_op(lib):
    for kw in (dict(batch=0), dict(hq=0, hk=0), dict(m=0)):
        assert window(lib, win_args(**kw)) == 0
        assert cached(lib, win_args(kv_len=FAKE, **kw)) == 0
    assert backward(lib, win_args(batch=0)) == 0 and backward(lib, win_args(m=0, n=0)) == 0


def test_python_checks():
    torch = pytest.importorskip("torch")
    x = torch.zeros(1, 2, 4, 8)
    with pytest.raises(ValueError):
        vef.qk_norm_rope(x, x)                                    # not on a GPU
    with pytest.raises(TypeError):
        vef.qk_norm_rope(x.double(), x.double())
    with pytest.raises(TypeError):
        vef.forward_window(x, x, x)                               # f32
    with pytest.raises(TypeError):
        vef.forward_window([1], x, x)
    with pytest.raises(ValueError):
        vef.forward_cached(x.half(), x.half(), x.half(), torch.zeros(1, dtype=torch.int32))
    with pytest.raises(ValueError):
        vef.forward_window(x.half()[0], x.half(), x.half())
