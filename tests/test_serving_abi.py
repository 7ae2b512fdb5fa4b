"""The serving calls are exported as declared and refuse bad arguments on the
host, before any CUDA call (no GPU needed)."""
import subprocess

import pytest

import vision_encoder_flash_gb300 as vef
from vision_encoder_flash_gb300 import _lib, decoder, serving

G = 2 ** 30
FAKE = 16 * G  # never dereferenced: every refusal comes before any CUDA call
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def lib():
    from vision_encoder_flash_gb300 import build
    build.build()
    return vef.load_library()


def test_exports_every_declared_symbol(lib):
    names = [n for n in _lib.exported_symbols(_lib.SERVING_HEADER)]
    assert set(names) == {"vattn_append_paged", "vattn_forward_paged", "vattn_forward_packed"}
    out = subprocess.run(["nm", "-D", "--defined-only", _lib.lib_path()], capture_output=True, text=True,
                         check=True).stdout
    for name in names:
        assert f" T {name}\n" in out and hasattr(vef, name[len("vattn_"):]), name


def rows(i, heads=2, n=16, dim=64, off=0, strides=None):
    """vattn_rows of the i-th of some buffers 1 GB apart."""
    return decoder._ROWS(FAKE + i * G + off, *(strides or (heads * n * dim, n * dim, dim)))


def pages(k=FAKE + 10 * G, v=FAKE + 11 * G, ks=(2048, 1024, 64), vs=None, k_scale=FAKE + 12 * G, v_scale=FAKE + 13 * G,
          table=FAKE + 14 * G, kv_len=FAKE + 15 * G, n_pages=8, page=16, max_pages=4):
    return serving._PAGES(k, v, *ks, *(vs or ks), k_scale, v_scale, table, kv_len, n_pages, page, max_pages)


def append_args(batch=1, heads=2, n=16, dim=64, rope=64, cu=0, positions=0, factors=0, base=1e4, dtype=1):
    return serving._APPEND(batch, heads, n, dim, rope, cu, positions, factors, base, dtype)


def append(lib, args=None, cache=None, k=None, v=None):
    s = lib.vattn_append_paged(k or rows(0), v or rows(1), cache or pages(), args or append_args(), 0)
    assert s == 0 or lib.vattn_last_error_string().decode() != ""
    return s


def win_args(batch=1, hq=4, hk=2, m=16, n=0, dim=64, window=0, sinks=0, kv_len=0, q_start=0, tree=0, scale=1.0, dtype=1):
    return decoder._WINDOW(batch, hq, hk, m, n, dim, window, sinks, kv_len, q_start, tree, scale, dtype)


def paged(lib, args=None, cache=None, q=None, out=None):
    s = lib.vattn_forward_paged(q or rows(0, 4), cache or pages(), out or rows(3, 4), args or win_args(), 0)
    assert s == 0 or lib.vattn_last_error_string().decode() != ""
    return s


def packed(lib, args=None, q=None, k=None, v=None, out=None, lse=0, cu=FAKE + 20 * G, n_seqs=3):
    s = lib.vattn_forward_packed(q or rows(0, 4), k or rows(1), v or rows(2), out or rows(3, 4), lse, cu, n_seqs,
                                 args or win_args(n=16), 0)
    assert s == 0 or lib.vattn_last_error_string().decode() != ""
    return s


@pytest.mark.parametrize("kw,status", [
    (dict(batch=-1), 1), (dict(heads=-1), 1), (dict(n=-5), 1), (dict(dim=0), 1), (dict(dim=144), 2), (dict(dim=72), 2),
    (dict(rope=65), 1), (dict(rope=-1), 1), (dict(base=0.0), 1), (dict(base=INF), 1), (dict(base=NAN), 1),
    (dict(dtype=0), 2), (dict(dtype=3), 2), (dict(n=2 ** 30), 2), (dict(batch=2 ** 30), 2), (dict(cu=FAKE + 2), 3),
    (dict(positions=FAKE + 1), 3), (dict(factors=FAKE + 2), 3),
])
def test_append_refuses_sizes_and_numbers(lib, kw, status):
    assert append(lib, append_args(**kw)) == status


@pytest.mark.parametrize("kw,status", [
    (dict(n_pages=-1), 1), (dict(n_pages=2 ** 31 - 1), 1), (dict(page=0), 2), (dict(page=24), 2), (dict(page=1040), 2),
    (dict(max_pages=-1), 2), (dict(max_pages=2 ** 25), 2), (dict(k=0), 1), (dict(v=0), 1), (dict(k=FAKE + 10 * G + 8), 3),
    (dict(ks=(2048, 1024, 72)), 3), (dict(ks=(2048, 1024, 0)), 1), (dict(ks=(0, 1024, 64)), 1), (dict(ks=(2048, -1024, 64)), 1),
    (dict(vs=(1024, 1024, 64)), 1), (dict(v=FAKE + 10 * G), 1), (dict(v=FAKE + 10 * G + 4096), 1), (dict(k_scale=0), 1),
    (dict(v_scale=0), 1), (dict(v_scale=FAKE + 12 * G + 4), 1), (dict(k_scale=FAKE + 12 * G + 2), 3),
    (dict(k_scale=FAKE + 10 * G + 64), 1), (dict(table=0), 1), (dict(table=FAKE + 2), 3), (dict(kv_len=0), 1),
    (dict(kv_len=FAKE + 1), 3),
])
def test_both_refuse_caches(lib, kw, status):
    assert append(lib, cache=pages(**kw)) == status
    assert paged(lib, cache=pages(**kw)) == status


def test_append_refuses_tensors(lib):
    null = decoder._ROWS(0, 2048, 1024, 64)
    assert append(lib, k=null) == 1 and append(lib, v=null) == 1
    assert append(lib, k=rows(0, off=1)) == 3
    assert append(lib, k=rows(10)) == 1 and append(lib, v=rows(11)) == 1   # over the pools
    assert append(lib, k=rows(12)) == 1 and append(lib, v=rows(13)) == 1   # over the scales
    assert append(lib, k=rows(0, strides=(2048, -1024, 64))) == 1
    assert lib.vattn_append_paged(rows(0), rows(1), None, append_args(), 0) == 1
    assert lib.vattn_append_paged(rows(0), rows(1), pages(), None, 0) == 1
    # heads and sequences so many that their blocks pass a grid
    wide = pages(ks=(64 * 16 * 2 ** 20, 64 * 16, 64), k_scale=FAKE + 2 ** 50, v_scale=FAKE + 2 ** 51, v=FAKE + 2 ** 52)
    k = decoder._ROWS(FAKE + 2 ** 53, 0, 0, 64)
    assert append(lib, append_args(heads=2 ** 20, batch=2 ** 20), cache=wide, k=k, v=k) == 2


def test_append_of_nothing_is_a_no_op(lib):
    for kw in (dict(batch=0), dict(heads=0), dict(n=0)):
        assert append(lib, append_args(**kw)) == 0
    assert append(lib, cache=pages(n_pages=0)) == 0 and append(lib, cache=pages(max_pages=0)) == 0


@pytest.mark.parametrize("kw,status", [
    (dict(batch=-1), 1), (dict(hq=-4), 1), (dict(m=-1), 1), (dict(dim=0), 1), (dict(dim=144), 2), (dict(dim=72), 2),
    (dict(dtype=0), 2), (dict(hq=3), 1), (dict(hk=0), 1), (dict(batch=2 ** 29), 2), (dict(window=-1), 1),
    (dict(sinks=-1), 1), (dict(scale=0.0), 1), (dict(scale=NAN), 1), (dict(tree=FAKE + 4), 3), (dict(m=65), 2),
    (dict(kv_len=FAKE), 1), (dict(q_start=FAKE), 1),
])
def test_paged_refuses_sizes_and_numbers(lib, kw, status):
    assert paged(lib, win_args(**kw)) == status


def test_paged_refuses_tensors(lib):
    null = decoder._ROWS(0, 1024, 1024, 64)
    assert paged(lib, q=null) == 1 and paged(lib, out=null) == 1
    assert paged(lib, q=rows(0, 4, off=8)) == 3 and paged(lib, q=rows(0, 4, strides=(4096, 1024, 68))) == 3
    assert paged(lib, out=rows(0, 4)) == 1 and paged(lib, out=rows(10, 4)) == 1 and paged(lib, out=rows(11, 4)) == 1
    assert paged(lib, out=rows(12, 4)) == 1 and paged(lib, out=rows(13, 4)) == 1
    assert paged(lib, out=rows(3, 4, strides=(4096, 0, 64))) == 1
    assert lib.vattn_forward_paged(rows(0, 4), None, rows(3, 4), win_args(), 0) == 1
    assert lib.vattn_forward_paged(rows(0, 4), pages(), rows(3, 4), None, 0) == 1
    for kw in (dict(batch=0), dict(hq=0, hk=0), dict(m=0)):
        assert paged(lib, win_args(**kw)) == 0


@pytest.mark.parametrize("kw,status", [
    (dict(batch=2), 1), (dict(batch=0), 1), (dict(n=15), 1), (dict(kv_len=FAKE), 1), (dict(q_start=FAKE), 1),
    (dict(tree=FAKE), 1), (dict(dim=60), 2), (dict(hq=3), 1), (dict(scale=INF), 1), (dict(dtype=0), 2),
])
def test_packed_refuses_sizes_and_numbers(lib, kw, status):
    assert packed(lib, win_args(**{"n": 16, **kw})) == status


def test_packed_refuses_tensors(lib):
    null = decoder._ROWS(0, 1024, 1024, 64)
    assert packed(lib, q=null) == 1 and packed(lib, v=null) == 1 and packed(lib, out=null) == 1
    assert packed(lib, cu=0) == 1 and packed(lib, cu=FAKE + 2) == 3
    assert packed(lib, n_seqs=-1) == 1 and packed(lib, n_seqs=2 ** 24) == 2
    assert packed(lib, out=rows(1, 4)) == 1 and packed(lib, lse=FAKE + 3 * G) == 1
    assert packed(lib, k=rows(1, strides=(2048, 1024, 0))) == 2
    assert packed(lib, n_seqs=0, cu=0) == 0 and packed(lib, win_args(m=0, n=0)) == 0
    assert packed(lib, win_args(hq=0, hk=0, n=16)) == 0


def test_python_checks():
    torch = pytest.importorskip("torch")
    x = torch.zeros(1, 2, 4, 16).half()
    p = torch.zeros(3, 2, 16, 16, dtype=torch.uint8)
    s, t, n = torch.ones(3, 2), torch.zeros(1, 2, dtype=torch.int32), torch.zeros(1, dtype=torch.int32)
    for call in (lambda: vef.append_paged(x, x, p, p, s, s, t, n), lambda: vef.forward_paged(x, p, p, s, s, t, n),
                 lambda: vef.forward_packed(x, x, x, n)):
        with pytest.raises(ValueError):
            call()                                                # not on a GPU
    for call in (lambda: vef.append_paged(x.float(), x, p, p, s, s, t, n), lambda: vef.forward_paged([1], p, p, s, s, t, n),
                 lambda: vef.forward_packed(x.float(), x, x, n)):
        with pytest.raises(TypeError):
            call()
