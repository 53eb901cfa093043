"""The paged cache at the ends of its range: views of one pool, replaced tensors,
calls on another stream, arguments out of range."""

import random

import pytest
import torch

from cache_model import CacheModel
from test_gpu_cache import check_attend, ints, make, randn

pytestmark = pytest.mark.gpu


def view(lib, k, v):
    """A cache over views of a pool (its book-keeping is not looked at)."""
    return lib.PagedCache(k, v, ints([[-1] * 3]), ints([0]), torch.zeros(k.shape[1], dtype=torch.int32, device="cuda"))


# how the source and the destination lie in the pool [layers, pages, heads, P, d]
VIEWS = {
    "pages apart": (lambda t: t[:, 5:], lambda t: t[:, :20]),
    "pages apart, the other way": (lambda t: t[:, :18], lambda t: t[:, 7:]),
    "layers apart": (lambda t: t[1:], lambda t: t[:-1]),
    "layers and pages apart": (lambda t: t[:-1, 3:], lambda t: t[1:, :-2]),
    "every second page": (lambda t: t[:, ::2], lambda t: t),
    "into every third page": (lambda t: t, lambda t: t[:, 1::3]),
    "one page": (lambda t: t[:, 4:5], lambda t: t),
    "the same": (lambda t: t, lambda t: t),
    "heads of their own": (lambda t: t[:, :, :2], lambda t: t[:, :, 2:]),
    "layers of their own": (lambda t: t[:2], lambda t: t[2:]),
    "pages of their own": (lambda t: t[:, :11], lambda t: t[:, 11:]),
}


@pytest.mark.parametrize("order", ["head", "row", "wide"])
@pytest.mark.parametrize("how", VIEWS)
def test_copy_between_views_of_one_pool(lib, how, order):
    """A page that is read is not written in the same call, whichever names the
    two caches have for it; every other pair is made."""
    pick_from, pick_to = VIEWS[how]
    pool = make(lib, layers=4, pages=23, P=4, heads_kv=4, d=64, order=order, seed=3)
    # the memory a page takes, by an id per (layer, page, head)
    ids = torch.arange(4 * 23 * 4).view(4, 23, 4, 1, 1)
    r = random.Random(how)
    for turn in range(6):
        f, t = (view(lib, pick(pool.k), pick(pool.v)) for pick in (pick_from, pick_to))
        n = 9
        src, dst = [r.randrange(-1, f.pages + 1) for _ in range(n)], [r.randrange(-1, t.pages + 1) for _ in range(n)]
        of, to = pick_from(ids), pick_to(ids)
        read = {x for s in src if 0 <= s < f.pages for x in of[:, s].flatten().tolist()}
        want = [pool.k.clone(), pool.v.clone()]
        for i, (s, d) in enumerate(zip(src, dst)):
            if not (0 <= s < f.pages and 0 <= d < t.pages) or d in dst[:i]:
                continue
            if read & set(to[:, d].flatten().tolist()):
                continue
            for w, x in zip(want, (pool.k, pool.v)):
                pick_to(w)[:, d] = pick_from(x)[:, s]
        t.copy_pages(ints(src), ints(dst), source=f)
        torch.cuda.synchronize()
        assert torch.equal(pool.k, want[0]) and torch.equal(pool.v, want[1]), turn


def test_tensors_cannot_be_replaced(lib):
    """The library keeps the addresses: an assignment that it would not notice is refused."""
    cache = make(lib)
    other = make(lib, layers=3, pages=41, P=8, heads_kv=3, d=64, slots=7, max_pages=9)
    for name in ("k", "v", "table", "lengths", "refs", "layers", "pages", "heads_kv", "page_size", "head_dim",
                 "slots", "max_pages"):
        with pytest.raises(AttributeError, match="cannot be replaced"):
            setattr(cache, name, getattr(other, name))
    cache.name = "a user's own attribute"
    cache.lengths[0] = 3        # contents are the caller's
    cache.lengths += 1
    assert cache.lengths.tolist()[0] == 4


@pytest.mark.parametrize("layer", [2, -1, 2 ** 31, 2 ** 32, 2 ** 32 + 1, -2 ** 32, 2 ** 70])
def test_layers_out_of_range_are_refused(lib, layer):
    cache = make(lib, layers=2)
    model = CacheModel(cache)
    start = cache.extend(ints([0]), ints([1]))
    model.extend([0], [1])
    k, q = randn((1, 2, 32), 1), randn((6, 4, 32), 2)
    for call in (lambda: cache.write(layer, k, k, ints([0]), start), lambda: cache.attend(layer, q)):
        with pytest.raises(lib.FaError) as e:
            call()
        assert e.value.code == 1
    model.check(cache)
