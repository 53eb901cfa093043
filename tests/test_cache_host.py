"""The paged cache's refusals, on the host: every call checks its arguments
before any launch (the addresses are fake and never touched)."""

import ctypes

import pytest
import torch

from test_abi import A16


def desc(lib, **kw):
    c = lib.CacheDesc()
    c.layers, c.pages, c.page_size, c.heads_kv, c.head_dim, c.slots, c.max_pages = 2, 10, 16, 2, 64, 3, 4
    c.k = c.v = c.table = c.lengths = c.refs = A16
    c.k_layer = c.v_layer = 10 * 2 * 16 * 64
    c.ks = c.vs = lib.Strides(2 * 16 * 64, 16 * 64, 64)
    for name, x in kw.items():
        setattr(c, name, lib.Strides(*x) if isinstance(x, tuple) else x)
    return c


def calls(lib, c, n=2, ws=A16, nbytes=1 << 30):
    """Every call on the description, with arguments that are fine."""
    so, r = lib.library(), ctypes.byref(c)
    return {
        "extend": lambda: so.fa_cache_extend(r, A16, A16, n, A16, ws, nbytes, None),
        "write": lambda: so.fa_cache_write(r, 0, A16, A16, 128, 64, 128, 64, A16, A16, None, n, n, None),
        "fork": lambda: so.fa_cache_fork(r, A16, A16, n, ws, nbytes, None),
        "free": lambda: so.fa_cache_free(r, A16, n, None),
        "compact": lambda: so.fa_cache_compact(r, A16, ws, nbytes, None),
        "copy": lambda: so.fa_cache_copy_pages(r, None, A16, A16, n, ws, nbytes, None),
        "attend": lambda: so.fa_cache_attend(r, 0, A16, A16, A16, 256, 64, 256, 64, None, n, 4, 0.125, 0, 0,
                                             ws, nbytes, None),
    }


@pytest.mark.parametrize("change,code", [
    (dict(layers=0), 1), (dict(pages=0), 1), (dict(page_size=0), 1), (dict(heads_kv=0), 1),
    (dict(slots=0), 1), (dict(max_pages=0), 1), (dict(k=None), 1), (dict(v=A16 + 8), 1),
    (dict(table=A16 + 2), 1), (dict(lengths=None), 1), (dict(refs=A16 + 1), 1),
    (dict(k_layer=0), 1), (dict(v_layer=4), 1), (dict(ks=(2048, 0, 64)), 1), (dict(vs=(2048, 1024, 60)), 1),
    (dict(vs=(-8, 1024, 64)), 1), (dict(ks=(2048, 1024, 0)), 1),
    (dict(head_dim=80), 2), (dict(head_dim=512), 2), (dict(max_pages=(1 << 20) + 1), 2),
    (dict(max_pages=1 << 20, page_size=2048), 2), (dict(pages=(1 << 30) + 1), 2),
])
def test_bad_descriptions_are_refused(lib, change, code):
    c = desc(lib, **change)
    for name, call in calls(lib, c).items():
        assert call() == code, name
    so = lib.library()
    assert so.fa_cache_workspace_size(ctypes.byref(c), 2) == 0
    assert so.fa_cache_attend_workspace_size(ctypes.byref(c), 2, 4, 0, 0) == 0
    for call in (lambda: so.fa_cache_free(None, A16, 1, None),
                 lambda: so.fa_cache_compact(None, A16, A16, 1 << 30, None)):
        assert call() == 1


def test_refs_are_needed_where_pages_change_hands(lib):
    c = desc(lib, refs=None)
    got = {name: call for name, call in calls(lib, c).items()}
    for name in ("extend", "fork", "free", "compact"):
        assert got[name]() == 1, name
    so, r = lib.library(), ctypes.byref(c)
    assert so.fa_cache_workspace_size(r, 2) > 0
    # zero entries launch nothing
    assert so.fa_cache_copy_pages(r, None, A16, A16, 0, A16, 1 << 30, None) == 0


def test_small_or_missing_workspaces(lib):
    c = desc(lib)
    need = lib.library().fa_cache_workspace_size(ctypes.byref(c), 2)
    assert need > 0 and need % 256 == 0
    for name in ("extend", "fork", "compact", "copy"):
        assert calls(lib, c, ws=None)[name]() == 5, name
        assert calls(lib, c, ws=A16 + 128)[name]() == 5, name
        assert calls(lib, c, nbytes=200)[name]() == 5, name


@pytest.mark.parametrize("name,args,code", [
    ("extend", (None, A16, 2, A16), 1), ("extend", (A16, A16, -1, A16), 1), ("extend", (A16, A16 + 1, 2, A16), 1),
    ("extend", (A16, A16, 2, None), 1),
    ("fork", (A16, None, 2), 1), ("fork", (A16, A16, -1), 1),
    ("copy_pages", (None, None, A16, 2), 1), ("copy_pages", (None, A16, A16, -1), 1),
    ("compact", (None,), 1),
])
def test_bad_lists_are_refused(lib, name, args, code):
    c = desc(lib)
    fn = getattr(lib.library(), "fa_cache_" + name)
    assert fn(ctypes.byref(c), *args, A16, 1 << 30, None) == code


def test_copy_between_unlike_caches_is_refused(lib):
    so, a = lib.library(), desc(lib)
    for change in (dict(layers=1), dict(page_size=8), dict(heads_kv=1), dict(head_dim=32)):
        b = desc(lib, **change)
        assert so.fa_cache_copy_pages(ctypes.byref(a), ctypes.byref(b), A16, A16, 2, A16, 1 << 30, None) == 1


@pytest.mark.parametrize("change,code", [
    (dict(layer=2), 1), (dict(layer=-1), 1), (dict(k=None), 1), (dict(v=A16 + 8), 1), (dict(k_row=4), 1),
    (dict(v_head=-8), 1), (dict(slots=None), 1), (dict(start=A16 + 2), 1), (dict(total=3), 1), (dict(n=-1, total=-1), 1),
    (dict(cu=A16 + 2), 1), (dict(n=0, total=0), 0), (dict(cu=A16, total=0), 0),
])
def test_bad_writes_are_refused(lib, change, code):
    a = dict(layer=0, k=A16, v=A16, k_row=128, k_head=64, v_row=128, v_head=64, slots=A16, start=A16, cu=None, n=2,
             total=2)
    a.update(change)
    assert lib.library().fa_cache_write(ctypes.byref(desc(lib)), *a.values(), None) == code


@pytest.mark.parametrize("change,code", [
    (dict(layer=2), 1), (dict(q=None), 1), (dict(o=A16 + 8), 1), (dict(lse=A16 + 2), 1), (dict(heads=3), 1),
    (dict(heads=0), 1), (dict(scale=0.0), 1), (dict(scale=float("inf")), 1), (dict(scale=float("nan")), 1),
    (dict(window=-1), 1), (dict(sinks=-1), 1), (dict(q_head=4), 1), (dict(o_head=0), 1), (dict(o_batch=0), 1),
    (dict(slots=A16 + 2), 1), (dict(batch=-1), 1), (dict(batch=0), 0),
    (dict(batch=(1 << 30), heads=2), 2), (dict(heads=65536), 2),
])
def test_bad_attends_are_refused(lib, change, code):
    a = dict(layer=0, q=A16, o=A16, lse=A16, q_batch=256, q_head=64, o_batch=256, o_head=64, slots=None, batch=2,
             heads=4, scale=0.125, window=0, sinks=0, ws=A16, nbytes=1 << 40)
    a.update(change)
    assert lib.library().fa_cache_attend(ctypes.byref(desc(lib)), *a.values(), None) == code


def test_binding_refuses_host_tensors_and_wrong_shapes(lib):
    kv = torch.zeros((1, 4, 2, 16, 64), dtype=torch.bfloat16)
    i = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    with pytest.raises(ValueError, match="CUDA"):
        lib.PagedCache(kv, kv, i(2, 3), i(2), i(4))
    with pytest.raises(ValueError, match="one shape"):
        lib.PagedCache(kv, kv[:, :3], i(2, 3), i(2), i(4))
    with pytest.raises(ValueError, match="expected"):
        lib.PagedCache(kv, kv, i(2, 3), i(3), i(4))
