"""Host-side checks of the head norms' and the 8-bit caches' entry points (no GPU)."""
import pytest

from slot_decode_window_gb300 import binding as B
from slot_decode_window_gb300 import build as BLD


@pytest.fixture(scope="module")
def lib():
    BLD.build()
    return B.load()


CACHE = (0x1000, 0x2000, 0x3000, 0x4000)


def _desc(**kw):
    base = dict(n_layers=2, n_slots=4, heads=8, kv_heads=2, head_dim=128, max_ctx=100, block=64, format=0)
    base.update(kw)
    return B.strata_kv8_desc(*(base[n] for n, _ in B.strata_kv8_desc._fields_))


@pytest.mark.parametrize("kw,status", [
    (dict(n_layers=0), B.STRATA_EINVAL), (dict(n_slots=0), B.STRATA_EINVAL), (dict(heads=0), B.STRATA_EINVAL),
    (dict(kv_heads=0), B.STRATA_EINVAL), (dict(max_ctx=0), B.STRATA_EINVAL), (dict(heads=7), B.STRATA_EINVAL),
    (dict(format=2), B.STRATA_EINVAL), (dict(format=-1), B.STRATA_EINVAL), (dict(head_dim=96), B.STRATA_EUNSUPPORTED),
    (dict(head_dim=0), B.STRATA_EUNSUPPORTED), (dict(block=48), B.STRATA_EUNSUPPORTED),
    (dict(block=8), B.STRATA_EUNSUPPORTED), (dict(heads=2048, kv_heads=2), B.STRATA_EUNSUPPORTED),
    (dict(heads=129, kv_heads=1), B.STRATA_EUNSUPPORTED),
    (dict(max_ctx=(1 << 24) + 1), B.STRATA_EUNSUPPORTED),
    (dict(n_slots=1 << 20, max_ctx=1 << 11), B.STRATA_EUNSUPPORTED),
])
def test_kv8_create_rejects_bad_desc_on_host(lib, kw, status):
    st, h = B.strata_kv8_create(_desc(**kw), B.strata_kv8_cache(*CACHE))
    assert st == status and h is None


@pytest.mark.parametrize("i", range(4))
def test_kv8_create_rejects_null_pointers(lib, i):
    c = list(CACHE)
    c[i] = None
    assert B.strata_kv8_create(_desc(), B.strata_kv8_cache(*c)) == (B.STRATA_EINVAL, None)
    if i < 2:  # codes that are not 128-byte aligned
        c[i] = 0x1010
        assert B.strata_kv8_create(_desc(), B.strata_kv8_cache(*c)) == (B.STRATA_EINVAL, None)


def test_kv8_calls_on_null(lib, monkeypatch):
    rows = B.strata_kv8_rows(1, 1, 1, 0x1000, 0x1000, 0x1000)
    assert B.strata_kv8_append(None, 0, 0x1000, 256, 0x1000, 256, 0, rows) == B.STRATA_EINVAL
    assert B.strata_kv8_read(None, 0, 0x1000, 256, 0x1000, 256, 0, rows) == B.STRATA_EINVAL
    assert B.strata_kv8_attend(None, 0, 0x1000, 1024, 0x2000, 1024, 0, 1.0, rows) == B.STRATA_EINVAL
    assert B.strata_kv8_sync(None) == B.STRATA_EINVAL
    assert B.strata_kv8_query(None)[0] == B.STRATA_EINVAL
    assert B.strata_kv8_destroy(None) == B.STRATA_OK
    assert B.strata_qknorm_destroy(None) == B.STRATA_OK
    monkeypatch.setenv("STRATA_FAULT", "alloc")
    assert B.strata_kv8_create(_desc(), B.strata_kv8_cache(*CACHE)) == (B.STRATA_ENOMEM, None)


@pytest.mark.parametrize("kw,status", [
    (dict(heads=0), B.STRATA_EINVAL), (dict(kv_heads=-1), B.STRATA_EINVAL), (dict(rotary_dim=-2), B.STRATA_EINVAL),
    (dict(rotary_dim=130), B.STRATA_EINVAL), (dict(interleaved=2), B.STRATA_EINVAL), (dict(norm=2), B.STRATA_EINVAL),
    (dict(eps=-1.0), B.STRATA_EINVAL), (dict(eps=float("nan")), B.STRATA_EINVAL),
    (dict(eps=float("inf")), B.STRATA_EINVAL), (dict(head_dim=96, rotary_dim=0), B.STRATA_EUNSUPPORTED),
    (dict(rotary_dim=20), B.STRATA_EUNSUPPORTED), (dict(heads=1025), B.STRATA_EUNSUPPORTED),
])
def test_qknorm_create_rejects_bad_desc_on_host(lib, kw, status):
    base = dict(heads=8, kv_heads=2, head_dim=128, rotary_dim=128, interleaved=0, norm=1, eps=1e-6)
    base.update(kw)
    d = B.strata_qknorm_desc(*(base[n] for n, _ in B.strata_qknorm_desc._fields_))
    st, h = B.strata_qknorm_create(d, None, None, [1.0] * 64)
    assert st == status and h is None


def test_qknorm_create_rejects_bad_frequencies(lib):
    d = B.strata_qknorm_desc(8, 2, 128, 128, 0, 1, 1e-6)
    assert B.strata_qknorm_create(d, None, None, None) == (B.STRATA_EINVAL, None)
    assert B.strata_qknorm_create(d, None, None, [float("inf")] * 64) == (B.STRATA_EINVAL, None)
