"""The paged cache at the ends of its range: views of one pool, replaced tensors,
calls on another stream, arguments out of range."""

import random

import pytest
import torch

from cache_model import CacheModel
from test_gpu_cache import check_attend, filled, ints, make, randn, widened

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


def test_calls_follow_the_current_stream(lib):
    """Nothing between the first copy and the last call looks at the device: a call
    sent to another stream would find the poisoned arguments."""
    d, H, Hkv = 64, 4, 2
    cache = make(lib, pages=30, P=4, d=d, heads_kv=Hkv, layers=1, slots=3, max_pages=12)
    model = CacheModel(cache)
    good = [ints([0, 1, 2]), ints([13, 20, 1]), ints([0, 13, 33, 34]), randn((34, Hkv, d), 1), randn((34, Hkv, d), 2),
            randn((3, H, d), 3)]
    slots, tokens, cu, k, v, q = [torch.full_like(t, -1 if t.dtype == torch.int32 else float("nan")) for t in good]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(100_000_000)
        for to, t in zip((slots, tokens, cu, k, v, q), good):
            to.copy_(t)
        start = cache.extend(slots, tokens)
        cache.write(0, k, v, slots, start, cu_seqlens=cu)
        o, lse = cache.attend(0, q, slots)
    torch.cuda.synchronize()
    assert start.tolist() == model.extend([0, 1, 2], [13, 20, 1])
    model.write(0, good[3], good[4], [0, 1, 2], [0, 0, 0], [0, 13, 33, 34])
    model.check(cache)
    check_attend(cache, 0, good[5], [0, 1, 2], o, lse, d ** -0.5)


@pytest.mark.parametrize("lens,columns", [([500, 3, 70], None), ([9000, 500, 20000, 1], 40000)])
def test_two_calls_at_once(lib, lens, columns):
    """Calls that overlap on two streams, each with its own workspace: the bits of
    the calls one after the other."""
    caches = [filled(lib, lens, 16, 2, 128, seed=s) for s in (41, 42)]
    if columns:
        caches = [widened(lib, c, columns) for c in caches]
    qs = [randn((len(lens), 8, 128), s) for s in (43, 44)]
    want = [c.attend(0, q) for c, q in zip(caches, qs)]
    streams = [torch.cuda.Stream() for _ in caches]
    torch.cuda.synchronize()
    got = [[], []]
    for turn in range(10):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(caches[i].attend(0, qs[i]))
    torch.cuda.synchronize()
    for i in range(2):
        for o, lse in got[i]:
            assert torch.equal(o, want[i][0]) and torch.equal(lse, want[i][1])


@pytest.mark.parametrize("columns", [None, 40000])
def test_mostly_idle_slots(lib, columns):
    """A batch of a fixed size with most of its slots unused or empty."""
    r = random.Random(6)
    lens = [0] * 512
    for s in r.sample(range(512), 12):
        lens[s] = r.randint(1, 700)
    cache = filled(lib, lens, 16, 2, 128, seed=45)
    if columns:
        cache = widened(lib, cache, columns)
    slots = [s if lens[s] or r.random() < 0.5 else -1 for s in range(512)]
    q = randn((512, 4, 128), 46)
    o, lse = cache.attend(0, q, ints(slots))
    check_attend(cache, 0, q, slots, o, lse, 128 ** -0.5)


@pytest.mark.parametrize("B,Hkv,G,window,sinks", [(513, 2, 4, 0, 0), (5000, 2, 1, 0, 0), (2100, 1, 17, 40, 5)])
def test_rows_cut_in_batches_of_many_chunks(lib, B, Hkv, G, window, sinks):
    """More sequences than a joining block adds up by itself: long ones, whose rows
    are cut, at the ends of the batch and of the blocks' chunks of sequences."""
    r = random.Random(B)
    lens = [r.choice([0, 1, 16, 17, r.randrange(90)]) for _ in range(B)]
    long = [0, 511, 512, B // 2, B - 1]
    for b in long:
        lens[b] = r.randint(3000, 6000)
    cache = filled(lib, lens, 16, Hkv, 64, seed=47)
    q = randn((B, Hkv * G, 64), 48)
    o, lse = cache.attend(0, q, window=window, sinks=sinks)
    some = sorted(set(long + [r.randrange(B) for _ in range(20)]))
    check_attend(cache, 0, q[some], some, o[some], lse[some], 64 ** -0.5, window, sinks)
    empty = [b for b in range(B) if lens[b] == 0]
    assert (o[empty] == 0).all() and (lse[empty] == float("-inf")).all()
    again = cache.attend(0, q, window=window, sinks=sinks)
    assert torch.equal(o, again[0]) and torch.equal(lse, again[1])


@pytest.mark.parametrize("B,Hkv,G,d,room", [(1, 4, 4, 128, 2048), (32, 4, 4, 128, 512), (64, 4, 2, 64, 512), (12, 1, 8, 256, 2048),
                                            (16, 1, 8, 256, 1024), (13, 1, 1, 256, 1024)])
def test_both_sides_of_the_clusters_rule(lib, B, Hkv, G, d, room):
    """Tables with just as much room as a cluster per row takes, and one page more:
    ragged lengths up to the whole table, on both ways."""
    r = random.Random(B + d)
    lens = [r.randint(0, room) for _ in range(B - 1)] + [room]
    q = randn((B, Hkv * G, d), 49)
    small = filled(lib, lens, 16, Hkv, d, seed=50)
    for columns in (room // 16, room // 16 + 1):
        table = torch.full((B, columns), -1, dtype=torch.int32, device="cuda")
        table[:, :room // 16] = small.table[:, :room // 16]
        cache = lib.PagedCache(small.k, small.v, table, small.lengths, small.refs)
        o, lse = cache.attend(0, q)
        check_attend(cache, 0, q, None, o, lse, d ** -0.5)
