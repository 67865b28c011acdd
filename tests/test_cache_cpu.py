"""Refusals of the paged cache's calls, before anything touches a GPU."""
import ctypes

import pytest

from titans_long_term_b200 import PagedCache, mem

GOOD = dict(d=64, type=0, B=2, H=4, Hkv=2, page=16, num_pages=8, max_pages=4)


@pytest.mark.parametrize("other,status", [
    (dict(d=80), mem.EUNSUPPORTED), (dict(type=2), mem.EINVAL), (dict(B=0), mem.EINVAL), (dict(Hkv=3), mem.EINVAL),
    (dict(Hkv=0), mem.EINVAL), (dict(page=48), mem.EUNSUPPORTED), (dict(page=8), mem.EUNSUPPORTED),
    (dict(num_pages=0), mem.EINVAL), (dict(num_pages=1 << 26), mem.EUNSUPPORTED), (dict(max_pages=1 << 28), mem.EUNSUPPORTED), (dict(max_pages=-1), mem.EINVAL),
    (dict(B=1 << 20, H=64), mem.EINVAL)])
def test_bad_configurations(other, status):
    c = mem.CacheConfig(*{**GOOD, **other}.values())
    h = ctypes.c_void_p(1)
    assert mem.lib().titans_cache_init(ctypes.byref(c), ctypes.byref(h)) == status
    assert h.value is None
    assert mem.lib().titans_last_error_string().decode()


def test_null_arguments():
    L = mem.lib()
    assert L.titans_cache_init(None, None) == mem.EINVAL
    assert L.titans_cache_destroy(None) == mem.EINVAL
    assert L.titans_cache_sync_status(None, None) == mem.EINVAL
    p = mem.CachePages(16, 16, None, None)
    assert L.titans_cache_append(None, 16, 16, 1, ctypes.byref(p), 16, 16, None, None) == mem.EINVAL
    assert L.titans_cache_read(None, ctypes.byref(p), 16, 16, None, 1, 16, 16, None) == mem.EINVAL
    assert L.titans_cache_attend(None, 16, 1, ctypes.byref(p), 16, 16, None, 0, 0, 1.0, 16, None, 0, None) == mem.EINVAL


def test_binding_refuses():
    with pytest.raises(ValueError, match="dtype"):
        PagedCache(64, "int8", 1, 1, num_pages=1, max_pages=1)
    with pytest.raises(mem.TitansError):
        PagedCache(64, "bf16", 1, 1)  # no pages


def test_a_table_as_long_as_positions_reach():
    """Positions are 32-bit, also when rounded up to a whole tile of keys."""
    c = mem.CacheConfig(*{**GOOD, "page": 128, "max_pages": (1 << 24) - 1}.values())
    h = ctypes.c_void_p(1)
    assert mem.lib().titans_cache_init(ctypes.byref(c), ctypes.byref(h)) == mem.EUNSUPPORTED
    assert h.value is None
