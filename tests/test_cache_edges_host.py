"""The paged cache's host side at the ends of its range: each call's workspace,
and what the binding refuses."""

import ctypes

import pytest

from test_abi import A16
from test_cache_host import calls, desc

SIZES = ("extend", "fork", "copy_pages")


def size_of(lib, name, c, *n):
    return getattr(lib.library(), f"fa_cache_{name}_workspace_size")(ctypes.byref(c), *n)


def test_only_a_fork_pays_for_table_rows(lib):
    """extend, compact and copy_pages need a few cells per entry, slot and page, however wide the table is."""
    n, pages, slots = 65536, 65536, 4096
    wide, narrow = (desc(lib, pages=pages, slots=slots, max_pages=m) for m in (8192, 1))
    for name in ("extend", "copy_pages"):
        assert size_of(lib, name, wide, n) == size_of(lib, name, narrow, n) <= 4 * (6 * n + slots + pages) + 4096
    assert size_of(lib, "compact", wide) == size_of(lib, "compact", narrow) <= 4 * 5 * pages + 4096
    assert size_of(lib, "fork", wide, n) >= 4 * n * 8192


def test_each_call_takes_its_own_workspace(lib):
    """A workspace of the call's own size passes the check, one byte less does not.  (What stands in the
    lists is not reached without a device.)"""
    c = desc(lib, pages=300, slots=70, max_pages=500)
    n = 33
    need = {"extend": size_of(lib, "extend", c, n), "fork": size_of(lib, "fork", c, n),
            "compact": size_of(lib, "compact", c), "copy": size_of(lib, "copy_pages", c, n)}
    assert all(x > 0 and x % 256 == 0 for x in need.values())
    assert lib.library().fa_cache_workspace_size(ctypes.byref(c), n) == max(need.values())
    for name, x in need.items():
        assert calls(lib, c, n=n, nbytes=x - 1)[name]() == 5, name


def test_workspace_sizes_of_bad_descriptions(lib):
    bad = desc(lib, layers=0)
    assert size_of(lib, "compact", bad) == 0
    for name in SIZES:
        assert size_of(lib, name, bad, 2) == 0 and size_of(lib, name, desc(lib), -1) == 0
    assert lib.library().fa_cache_workspace_size(ctypes.byref(desc(lib)), -1) == 0


def test_tensors_of_a_cache_cannot_be_replaced(lib):
    """The library keeps the addresses, so an assignment it would not notice is refused; the same tensor
    may come back from an in-place operator."""
    import torch
    cache = lib.PagedCache.__new__(lib.PagedCache)
    cache.lengths = torch.zeros(3, dtype=torch.int32)
    cache.pages = 4
    cache._sizes = {}  # the description is made
    with pytest.raises(AttributeError, match="cannot be replaced"):
        cache.lengths = torch.zeros(3, dtype=torch.int32)
    with pytest.raises(AttributeError, match="cannot be replaced"):
        cache.pages = 5
    cache.lengths += 1
    cache.label = "a user's own attribute"
    assert cache.lengths.tolist() == [1, 1, 1] and cache.pages == 4


def test_plans_of_the_largest_batches(lib):
    """Counts of rows past 2^31 / 8 (undefined behaviour in 32 bits, which the sanitizer build reports)."""
    so = lib.library()
    c = desc(lib, heads_kv=1, head_dim=32, max_pages=4, page_size=16, slots=1)
    for batch in (1 << 20, 1 << 28, (1 << 31) - 1):
        assert so.fa_cache_attend_workspace_size(ctypes.byref(c), batch, 1, 0, 0) > 0
    # more rows than the 32-bit counts of tiles hold are refused before any launch
    a = [0, A16, A16, A16, 32, 32, 32, 32, None, (1 << 31) - 1, 1, 0.125, 0, 0, A16, 1 << 40, None]
    assert so.fa_cache_attend(ctypes.byref(c), *a) == 2


def test_lists_that_would_take_minutes_are_refused(lib):
    """A fork and a page copy look at every pair of entries: at most 2^20 entries."""
    c = desc(lib)
    for n in ((1 << 20) + 1, (1 << 31) - 1):
        for name in ("fork", "copy"):
            assert calls(lib, c, n=n, nbytes=1 << 50)[name]() == 2, (name, n)
