"""The paged cache: its calls against a sequential model, to the bit, and the
decode attention against a plain 64-bit form within the bounds that its
roundings give (P and the output to bf16, sums and statistics in fp32)."""

import random

import pytest
import torch

import plain64
from cache_model import CacheModel

pytestmark = pytest.mark.gpu


def randn(shape, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(shape, generator=g, device="cuda").to(torch.bfloat16)


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def make(lib, layers=2, pages=40, P=4, heads_kv=2, d=32, slots=6, max_pages=8, seed=0, order="head"):
    """An empty cache with random rows everywhere; order "row": [layers, pages, P, heads, d] in memory."""
    if order == "head":
        k, v = (randn((layers, pages, heads_kv, P, d), seed + i) for i in range(2))
    elif order == "row":
        k, v = (randn((layers, pages, P, heads_kv, d), seed + i).transpose(2, 3) for i in range(2))
    else:  # k and v of a layer in one buffer, wider rows than d
        kv = randn((pages, layers, 2, heads_kv, P, d + 8), seed)
        k, v = (kv[:, :, i, :, :, :d].transpose(0, 1) for i in range(2))
    return lib.PagedCache(k, v, torch.full((slots, max_pages), -1, dtype=torch.int32, device="cuda"),
                          torch.zeros(slots, dtype=torch.int32, device="cuda"),
                          torch.zeros(pages, dtype=torch.int32, device="cuda"))


def grow(cache, model, slots, tokens, seed):
    """extend and write on both sides."""
    start = cache.extend(ints(slots), ints(tokens))
    want = model.extend(slots, tokens)
    assert start.tolist() == want
    put = [max(t, 0) if w >= 0 else 0 for t, w in zip(tokens, want)]
    cu = [0]
    for t in put:
        cu.append(cu[-1] + t)
    for layer in range(cache.layers):
        k, v = (randn((cu[-1], cache.heads_kv, cache.head_dim), seed + 10 * layer + i) for i in range(2))
        cache.write(layer, k, v, ints(slots), start, cu_seqlens=ints(cu))
        model.write(layer, k, v, slots, want, cu)


@pytest.mark.parametrize("P,d,order,seed", [(4, 32, "head", 1), (1, 64, "row", 2), (3, 96, "wide", 3),
                                            (16, 128, "head", 4), (5, 192, "row", 5), (2, 256, "wide", 6)])
def test_random_calls_match_the_model(lib, P, d, order, seed):
    r = random.Random(seed)
    cache = make(lib, P=P, d=d, order=order, pages=37, slots=7, max_pages=6, seed=seed)
    model = CacheModel(cache)
    for turn in range(30):
        what = r.choice(["grow", "grow", "grow", "fork", "free", "compact", "copy"])
        some = [r.randrange(-1, 8) for _ in range(r.randint(1, 7))]
        if what == "grow":
            grow(cache, model, some, [r.choice([0, 1, 1, P, r.randrange(-1, 3 * P + 1)]) for _ in some], 100 * turn)
        elif what == "fork":
            to = [r.randrange(-1, 8) for _ in some]
            cache.fork(ints(some), ints(to))
            model.fork(some, to)
        elif what == "free":
            cache.free(ints(some[:2]))
            model.free(some[:2])
        elif what == "compact":
            assert cache.compact().tolist() == [model.compact()]
        else:
            src, dst = [r.randrange(-1, 38) for _ in range(6)], [r.randrange(-1, 38) for _ in range(6)]
            cache.copy_pages(ints(src), ints(dst))
            model.copy_pages(src, dst)
        model.consistent()
        model.check(cache)


def test_extend_grants_in_order_until_pages_run_out(lib):
    cache = make(lib, pages=6, P=4, slots=8, max_pages=4)
    model = CacheModel(cache)
    # 2 pages; too long for a row; out of range; 3 pages; 2 more than there are; again; none needed
    slots, tokens = [0, 1, 9, 2, 3, 0, 4, 5], [7, 17, 1, 12, 5, 1, 0, 1]
    start = cache.extend(ints(slots), ints(tokens))
    assert start.tolist() == model.extend(slots, tokens) == [0, -1, -1, 0, -1, -1, 0, -1]
    model.check(cache)
    # slot 0 grows inside its last page although no page is left for slot 2
    grow(cache, model, [2, 0], [8, 1], 5)
    model.check(cache)
    assert cache.lengths.tolist()[:3] == [8, 0, 12]


def test_every_sharer_of_a_last_page_gets_its_own(lib):
    cache = make(lib, pages=20, P=8, slots=4, max_pages=4)
    model = CacheModel(cache)
    grow(cache, model, [0], [13], 1)
    cache.fork(ints([0, 0, 0]), ints([1, 2, 3]))
    model.fork([0, 0, 0], [1, 2, 3])
    grow(cache, model, [3, 1], [1, 5], 2)       # two copy, two still share
    model.check(cache)
    grow(cache, model, [0, 2], [1, 1], 3)       # both copy, the old page becomes free
    model.consistent()
    model.check(cache)
    assert sorted(cache.refs.tolist())[-1] == 4  # the first page is still everybody's


def test_fork_permutes_and_chains(lib):
    cache = make(lib, pages=40, P=2, slots=5, max_pages=8)
    model = CacheModel(cache)
    grow(cache, model, [0, 1, 2, 3, 4], [3, 5, 1, 0, 16], 1)
    for src, dst in (([1, 2, 0], [0, 1, 2]), ([4, 4, 4, 0], [0, 1, 4, 3]), ([2, 3], [3, 3]), ([3, 2], [2, 3])):
        cache.fork(ints(src), ints(dst))
        model.fork(src, dst)
        model.consistent()
        model.check(cache)


@pytest.mark.parametrize("pages,seed", [(1, 0), (1023, 1), (4097, 2), (9000, 3)])
def test_compact_and_extend_over_many_pages(lib, pages, seed):
    """More pages than one pass of the scans; some slots hold scattered pages."""
    r = random.Random(seed)
    cache = make(lib, layers=1, pages=pages, P=1, heads_kv=1, d=32, slots=5, max_pages=max(1, pages))
    order = list(range(pages))
    r.shuffle(order)
    at = 0
    for s in range(4):
        n = r.randint(0, (pages - at) // 2)
        row = order[at:at + n]
        at += n
        cache.table[s, :n] = ints(row) if n else 0
        cache.lengths[s] = n
        if n:
            cache.refs[ints(row).long()] = 1
    model = CacheModel(cache)
    grow(cache, model, [4], [min(3, pages - at)], 9)
    model.check(cache)
    assert cache.compact().tolist() == [model.compact()]
    model.consistent()
    model.check(cache)
    assert cache.compact().tolist() == [model.compact()]  # nothing left to move
    model.check(cache)


def test_more_entries_than_threads(lib):
    """2500 slots in one call, the same slot again among them."""
    n = 2500
    cache = make(lib, layers=1, pages=4000, P=2, heads_kv=1, d=32, slots=n, max_pages=3)
    model = CacheModel(cache)
    slots = list(range(n))
    random.Random(3).shuffle(slots)
    slots[2000] = slots[10]
    tokens = [i % 5 for i in range(n)]
    start = cache.extend(ints(slots), ints(tokens))
    assert start.tolist() == model.extend(slots, tokens)
    model.check(cache)


def test_copy_between_caches(lib):
    a, b = make(lib, pages=9, seed=1), make(lib, pages=5, seed=5, order="row")
    ma, mb = CacheModel(a), CacheModel(b)
    src, dst = [8, 0, 3, 9, 2, 1], [0, 4, 4, 1, 5, 1]
    b.copy_pages(ints(src), ints(dst), source=a)
    mb.copy_pages(src, dst, ma)
    ma.check(a)
    mb.check(b)


# ---------------------------------------------------------------------------
# decode attention
# ---------------------------------------------------------------------------

def gather(cache, layer, slot):
    """K, V [heads_kv, n, d] float64 of a slot, and which rows have a page."""
    n = max(0, min(int(cache.lengths[slot]), cache.max_pages * cache.page_size))
    j = torch.arange(n, device="cuda")
    page = cache.table[slot].long()[j // cache.page_size]
    live = (page >= 0) & (page < cache.pages)
    page = torch.where(live, page, torch.zeros_like(page))
    pick = lambda t: torch.where(live[:, None], t[layer][page, :, j % cache.page_size].transpose(0, 1).double(),  # noqa: E731
                                 torch.zeros((), dtype=torch.float64, device="cuda"))
    return pick(cache.k), pick(cache.v), live


def check_attend(cache, layer, q, slots, o, lse, scale, window=0, sinks=0):
    torch.cuda.synchronize()
    B, H, d = q.shape
    G = H // cache.heads_kv
    for b in range(B):
        s = b if slots is None else slots[b]
        if not 0 <= s < cache.slots or int(cache.lengths[s]) <= 0:
            assert (o[b] == 0).all() and (lse[b] == float("-inf")).all()
            continue
        k, v, live = gather(cache, layer, s)
        n = k.shape[1]
        mask = plain64.visible(1, n, q.device, causal=False, window=window, sinks=sinks) & live[None, :]
        for h in range(cache.heads_kv):
            hs = slice(h * G, (h + 1) * G)
            r = plain64.head(q[b, hs].double(), k[h], v[h], scale, mask.expand(G, n))
            plain64.check_lse(lse[b, hs], r["lse"])
            plain64.check("o", o[b, hs], r["o"], r["o_tol"])


def filled(lib, lens, P, heads_kv, d, seed=0, order="head", layers=1, spare=3):
    """A cache whose slot b holds lens[b] tokens in shuffled pages; rows behind the ends are NaN or infinite."""
    need = [-(-n // P) for n in lens]
    pages = sum(need) + spare
    cache = make(lib, layers=layers, pages=pages, P=P, heads_kv=heads_kv, d=d, slots=len(lens),
                 max_pages=max(need + [1]) + 1, seed=seed, order=order)
    ids = list(range(pages))
    random.Random(seed).shuffle(ids)
    free = torch.ones(pages, dtype=torch.bool)
    for s, (n, c) in enumerate(zip(lens, need)):
        mine, ids = ids[:c], ids[c:]
        if c:
            cache.table[s, :c] = ints(mine)
            cache.refs[ints(mine).long()] = 1
            free[mine] = False
            if n % P:
                cache.k[:, mine[-1], :, n % P:] = float("nan")
                cache.v[:, mine[-1], :, n % P:] = float("inf")
        cache.lengths[s] = n
    cache.k[:, free.cuda()] = float("inf")
    cache.v[:, free.cuda()] = float("nan")
    return cache


# lengths, page size, heads, K / V heads, d, window, sinks, order of the pool
DECODE = [
    ([1], 16, 1, 1, 64, 0, 0, "head"),
    ([1, 0, 2, 15, 16, 17, 31, 32, 33], 16, 4, 2, 128, 0, 0, "head"),
    ([63, 64, 65, 127, 128, 129, 500], 1, 8, 2, 64, 0, 0, "head"),
    ([700, 3, 333], 24, 4, 1, 32, 0, 0, "row"),
    ([700, 3, 333], 7, 3, 3, 96, 0, 0, "wide"),
    ([257, 1000], 64, 16, 2, 192, 0, 0, "head"),
    ([257, 1000, 0, 5], 128, 8, 1, 256, 0, 0, "row"),
    ([300, 40], 16, 16, 1, 128, 0, 0, "head"),         # a full block of heads
    ([300, 40], 16, 17, 1, 64, 0, 0, "head"),          # one more
    ([300, 40], 16, 40, 1, 128, 0, 0, "head"),
    ([300, 40, 41, 45, 44], 16, 4, 2, 128, 40, 4, "head"),
    ([300, 40, 1, 0], 16, 4, 2, 64, 1, 0, "row"),      # the newest token alone
    ([300, 40, 12], 8, 4, 4, 256, 7, 100, "head"),     # first tokens beyond some sequences
    ([5000, 4097], 32, 4, 2, 128, 1000, 130, "head"),
    ([20000, 1, 70], 256, 4, 1, 128, 0, 0, "head"),
    ([9000], 16, 2, 2, 64, 0, 0, "head"),
]


@pytest.mark.parametrize("lens,P,H,Hkv,d,window,sinks,order", DECODE)
def test_attend_matches_64_bits(lib, lens, P, H, Hkv, d, window, sinks, order):
    cache = filled(lib, lens, P, Hkv, d, seed=len(lens) + d, order=order, layers=2)
    q = randn((len(lens), H, d), 50)
    for layer in (0, 1):
        o, lse = cache.attend(layer, q, window=window, sinks=sinks)
        check_attend(cache, layer, q, None, o, lse, d ** -0.5, window, sinks)


def test_attend_slots_strides_and_scale(lib):
    """Slots in any order, twice, and out of range; q a slice of a wider
    projection, O with heads of another stride."""
    cache = filled(lib, [100, 7, 0, 260], 8, 2, 128, seed=3)
    slots = [3, -1, 1, 1, 2, 4, 0, 2 ** 31 - 1]
    wide = randn((len(slots), 3, 8, 128), 60)
    q = wide[:, 1, 2:6]
    out = torch.full((len(slots), 4, 136), 5.0, dtype=torch.bfloat16, device="cuda")[:, :, :128]
    o, lse = cache.attend(0, q, ints(slots), scale=0.3, out=out)
    assert o is out
    check_attend(cache, 0, q, slots, o, lse, 0.3)
    assert (out.as_strided((len(slots), 4, 8), (4 * 136, 136, 1), 128) == 5.0).all()


def test_attend_holes_and_bad_lengths(lib):
    """Missing pages hold no keys; lengths beyond the table are cut, negative ones are none."""
    cache = filled(lib, [100, 90, 64, 64, 40], 16, 2, 64, seed=4)
    cache.table[0, 2] = -1
    cache.table[0, 6] = cache.pages
    cache.table[1, :] = -1
    cache.lengths[2] = 2 ** 31 - 1
    cache.lengths[3] = -5
    cache.table[4, 0] = -7
    q = randn((5, 4, 64), 61)
    for window, sinks in ((0, 0), (30, 20)):
        o, lse = cache.attend(0, q, window=window, sinks=sinks)
        if window == 0:
            assert (o[1] == 0).all() and (lse[1] == float("-inf")).all()
        check = [0, 2, 4]
        check_attend(cache, 0, q[check], check, o[check], lse[check], 0.125, window, sinks)
        assert (o[3] == 0).all() and (lse[3] == float("-inf")).all()


def test_attend_large_scores(lib):
    """Scores of several hundred: the running maximum keeps exp2 in range."""
    cache = filled(lib, [300, 1000], 16, 1, 128, seed=5)
    live = torch.isfinite(cache.k.float())
    cache.k.copy_(torch.where(live, cache.k * 8, cache.k))
    q = (randn((2, 4, 128), 62) * 8).to(torch.bfloat16)
    o, lse = cache.attend(0, q)
    torch.cuda.synchronize()
    for b in range(2):
        k, v, live = gather(cache, 0, b)
        r = plain64.head(q[b].double(), k[0], v[0], 128 ** -0.5, live.expand(4, -1))
        # scores up to ~1000, off by 2^-22 of themselves: P by 3e-4 more
        plain64.check_lse(lse[b], r["lse"], 1e-3)
        plain64.check("o", o[b], r["o"], r["o_tol"] + 1e-3 * v[0].abs().max())


@pytest.mark.parametrize("lens,H,Hkv,d", [
    ([60, 33, 1], 4, 2, 128),             # a cluster of blocks per row
    ([60] * 300 + [7], 4, 2, 64),         # rows whole in a share
    ([40000, 500, 9000, 3], 8, 2, 128),   # rows cut, and joined
    ([900] * 80, 16, 1, 256),
])
def test_attend_keeps_what_is_not_a_number(lib, lens, H, Hkv, d):
    """A visible key, or a query, that is not a number: O and LSE of the rows that
    see it are none either, and every other row is as it was."""
    cache = filled(lib, lens, 32, Hkv, d, seed=9)
    q = randn((len(lens), H, d), 64)
    o, lse = cache.attend(0, q)
    assert torch.isfinite(o).all() and torch.isfinite(lse).all()
    bad = torch.zeros(len(lens), H, dtype=torch.bool, device="cuda")
    for s in {0, len(lens) // 2}:  # the last token of K / V head 0
        at = lens[s] - 1
        cache.k[0, cache.table[s, at // 32], 0, at % 32, 5] = float("nan")
        bad[s, :H // Hkv] = True
    q[-1, -1, d - 1] = float("nan")
    bad[-1, -1] = True
    o1, lse1 = cache.attend(0, q)
    assert o1[bad].isnan().all() and lse1[bad].isnan().all()
    assert torch.equal(o1[~bad], o[~bad]) and torch.equal(lse1[~bad], lse[~bad])


def test_offsets_beyond_32_bits(lib):
    """Pages past 2^32 bytes and past 2^31 elements of the pool."""
    P, d, pages = 256, 128, 70000
    k = torch.empty((1, pages, 1, P, d), dtype=torch.bfloat16, device="cuda")
    v = torch.empty_like(k)
    assert k.numel() > 2 ** 31
    cache = lib.PagedCache(k, v, torch.full((2, 4), -1, dtype=torch.int32, device="cuda"), ints([0, 0]),
                           torch.ones(pages, dtype=torch.int32, device="cuda"))
    far = [pages - 1, 3, pages - 2, 65536, pages - 3]
    cache.refs[ints(far).long()] = 0
    start = cache.extend(ints([0, 1]), ints([700, 300]))
    assert cache.table.tolist() == [[3, 65536, pages - 3, -1], [pages - 2, pages - 1, -1, -1]]
    new_k, new_v = randn((1000, 1, d), 70), randn((1000, 1, d), 71)
    cache.write(0, new_k, new_v, ints([0, 1]), start, cu_seqlens=ints([0, 700, 1000]))
    q = randn((2, 4, d), 72)
    o, lse = cache.attend(0, q)
    check_attend(cache, 0, q, None, o, lse, d ** -0.5)
    gk, _, _ = gather(cache, 0, 1)
    assert torch.equal(gk[0], new_k[700:, 0].double())


# ---------------------------------------------------------------------------
# together
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("window,sinks,d", [(0, 0, 128), (50, 4, 64)])
def test_prefill_then_decode_equals_one_pass(lib, window, sinks, d):
    """Prompts through the windowed forward, their keys into the cache, then
    decode steps with forks and frees in between: each new token's output is the
    row that the whole sequence would give."""
    layers, H, Hkv, P, slots = 2, 4, 2, 16, 4
    lens = [70, 129]
    cache = lib.PagedCache.allocate(layers, 60, P, Hkv, d, slots, 20)
    cu = ints([0, lens[0], sum(lens)])
    hist = {}
    start = cache.extend(ints([0, 1]), ints(lens))
    for layer in range(layers):
        q, k, v = randn((sum(lens), H, d), layer), randn((sum(lens), Hkv, d), 10 + layer), randn((sum(lens), Hkv, d), 20 + layer)
        lib.forward_general(q, k, v, layout="thd", cu_seqlens_q=cu, cu_seqlens_k=cu, max_seqlen_q=129,
                            max_seqlen_k=129, causal=True, window=window, sinks=sinks)
        cache.write(layer, k, v, ints([0, 1]), start, cu_seqlens=cu)
        hist[layer] = {0: [k[:70], v[:70]], 1: [k[70:], v[70:]]}
    live = [0, 1]
    for step in range(20):
        if step == 3:
            cache.fork(ints([0, 1]), ints([2, 3]))
            for layer in hist:
                hist[layer][2], hist[layer][3] = list(hist[layer][0]), list(hist[layer][1])
            live = [0, 1, 2, 3]
        if step == 9:
            cache.free(ints([1]))
            live = [0, 2, 3]
        if step == 12:
            cache.compact()
        n = len(live)
        start = cache.extend(ints(live), ints([1] * n))
        for layer in range(layers):
            q, k, v = (randn((n, h, d), 1000 * step + 10 * layer + i) for i, h in enumerate((H, Hkv, Hkv)))
            cache.write(layer, k, v, ints(live), start)
            o, lse = cache.attend(layer, q, ints(live), window=window, sinks=sinks)
            for i, s in enumerate(live):
                h = hist[layer][s]
                h[0], h[1] = torch.cat([h[0], k[i:i + 1]]), torch.cat([h[1], v[i:i + 1]])
                m = len(h[0])
                ref = plain64.padded(q[i][None, :, None], h[0].transpose(0, 1)[None], h[1].transpose(0, 1)[None],
                                     d ** -0.5, lambda _: plain64.visible(1, m, q.device, window=window, sinks=sinks))
                plain64.check("o", o[i], ref["o"][0, :, 0], ref["o_tol"][0, :, 0])
                plain64.check_lse(lse[i], ref["lse"][0, :, 0])
    assert lib.last_device_status() == 0


def test_captured_step(lib):
    """A whole decode step in a graph, replayed while the cache grows across page
    ends; two graphs of the same cache take turns."""
    P, H, Hkv, d = 4, 4, 2, 64
    caches = [filled(lib, [5, 30, 12], P, Hkv, d, seed=9, spare=60, layers=1) for _ in range(2)]
    slots, ones = ints([0, 1, 2]), ints([1, 1, 1])
    q, k, v = randn((3, H, d), 1), randn((3, Hkv, d), 2), randn((3, Hkv, d), 3)

    def step(cache, window):
        start = cache.extend(slots, ones)
        cache.write(0, k, v, slots, start)
        return cache.attend(0, q, slots, window=window, sinks=1 if window else 0)

    step(caches[0], 0)   # warm: the first launches set attributes
    step(caches[1], 0)
    side, graphs, outs = torch.cuda.Stream(), [], []
    for window in (0, 6):
        side.wait_stream(torch.cuda.current_stream())
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            outs.append(step(caches[0], window))
        graphs.append(g)
    for turn in range(8):
        i = turn % 2
        for t, s in ((q, 1), (k, 2), (v, 3)):
            t.copy_(randn(t.shape, 100 * turn + s))
        graphs[i].replay()
        want = step(caches[1], (0, 6)[i])
        torch.cuda.synchronize()
        assert torch.equal(outs[i][0], want[0]) and torch.equal(outs[i][1], want[1])
        assert torch.equal(caches[0].table, caches[1].table)
    # slot 1's table row is full at 9 pages of 4: its later tokens are not granted
    assert caches[0].lengths.tolist() == [5 + 9, 36, 12 + 9]


def test_another_stream(lib):
    """Calls go to the current stream, in its order."""
    cache = make(lib, pages=30, P=4, d=64, layers=1, slots=2, max_pages=12)
    model = CacheModel(cache)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)
        grow(cache, model, [0, 1], [13, 20], 1)
        o, lse = cache.attend(0, randn((2, 2, 64), 5))
    side.synchronize()
    model.check(cache)
    check_attend(cache, 0, randn((2, 2, 64), 5), None, o, lse, 0.125)


def test_results_repeat(lib):
    """The same call gives the same bits."""
    cache = filled(lib, [30000, 5, 700, 12345], 16, 2, 128, seed=11)
    q = randn((4, 8, 128), 63)
    a = cache.attend(0, q)
    for _ in range(3):
        b = cache.attend(0, q)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_empty_calls(lib):
    cache = make(lib)
    model = CacheModel(cache)
    none = ints([])
    assert cache.extend(none, none).shape == (0,)
    cache.free(none)
    cache.fork(none, none)
    cache.copy_pages(none, none)
    kv = torch.empty((0, 2, 32), dtype=torch.bfloat16, device="cuda")
    cache.write(0, kv, kv, none, none)
    o, lse = cache.attend(0, torch.empty((0, 4, 32), dtype=torch.bfloat16, device="cuda"))
    assert o.shape == (0, 4, 32) and lse.shape == (0, 4)
    assert cache.compact().tolist() == [0]
    model.check(cache)


@pytest.mark.parametrize("B,P,H,Hkv,d,window,sinks", [
    (300, 16, 8, 2, 96, 0, 0), (700, 16, 4, 1, 96, 0, 0), (1100, 16, 2, 1, 32, 9, 2), (130, 8, 20, 1, 64, 50, 3), (257, 4, 2, 2, 256, 0, 0), (1000, 16, 4, 1, 128, 0, 0)])
def test_attend_many_sequences(lib, B, P, H, Hkv, d, window, sinks):
    """More sequences than a block looks at together: short, empty and one long one among them."""
    r = random.Random(B)
    lens = [r.choice([0, 1, 5, 16, 17, r.randrange(60)]) for _ in range(B)]
    lens[B // 2] = 9000
    cache = filled(lib, lens, P, Hkv, d, seed=B)
    q = randn((B, H, d), 64)
    slots = list(range(B))
    r.shuffle(slots)
    o, lse = cache.attend(0, q, ints(slots), window=window, sinks=sinks)
    some = sorted(set([0, 127 % B, 128 % B, B - 1, slots.index(B // 2)] + [r.randrange(B) for _ in range(25)]))
    check_attend(cache, 0, q[some], [slots[i] for i in some], o[some], lse[some], d ** -0.5, window, sinks)
    empty = [i for i in range(B) if lens[slots[i]] == 0]
    assert (o[empty] == 0).all() and (lse[empty] == float("-inf")).all()


def test_attend_leads_to_the_next_call_in_order(lib):
    """Rows that need no joining: the joining kernel has nothing to wait for, yet
    a write behind it must not reach the pages while they are read."""
    cache = filled(lib, [16] * 2000, 16, 1, 128, seed=21)
    q, start = randn((2000, 1, 128), 65), ints([0] * 2000)
    slots = ints(list(range(2000)))
    want = cache.attend(0, q, slots)
    junk = torch.full((2000, 1, 128), 1e4, dtype=torch.bfloat16, device="cuda")
    keep = cache.k.clone(), cache.v.clone()
    for _ in range(20):
        got = cache.attend(0, q, slots)
        cache.write(0, junk, junk, slots, start)
        torch.cuda.synchronize()
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
        cache.k.copy_(keep[0])
        cache.v.copy_(keep[1])


def widened(lib, cache, columns=40000):
    """The same cache with room for very long sequences: the work is then cut into
    equal shares, where short tables get a cluster of blocks per row."""
    table = torch.full((cache.slots, columns), -1, dtype=torch.int32, device="cuda")
    table[:, :cache.max_pages] = cache.table
    return lib.PagedCache(cache.k, cache.v, table, cache.lengths, cache.refs)


@pytest.mark.parametrize("lens,P,H,Hkv,d,window,sinks,order", DECODE)
def test_attend_in_equal_shares(lib, lens, P, H, Hkv, d, window, sinks, order):
    small = filled(lib, lens, P, Hkv, d, seed=len(lens) + d + 1, order=order)
    cache = widened(lib, small, 40000 if P <= 256 else 4000)
    q = randn((len(lens), H, d), 51)
    o, lse = cache.attend(0, q, window=window, sinks=sinks)
    check_attend(cache, 0, q, None, o, lse, d ** -0.5, window, sinks)
    o2, lse2 = cache.attend(0, q, window=window, sinks=sinks)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)


def test_equal_shares_with_holes_and_bad_lengths(lib):
    cache = widened(lib, filled(lib, [100, 90, 64, 64, 40], 16, 2, 64, seed=4))
    cache.table[0, 2] = -1
    cache.table[0, 6] = cache.pages
    cache.table[1, :] = -1
    cache.lengths[2] = -1
    cache.lengths[3] = -5
    cache.table[4, 0] = -7
    q = randn((5, 4, 64), 61)
    o, lse = cache.attend(0, q)
    check_attend(cache, 0, q[[0, 4]], [0, 4], o[[0, 4]], lse[[0, 4]], 0.125)
    for i in (1, 2, 3):
        assert (o[i] == 0).all() and (lse[i] == float("-inf")).all()


@pytest.mark.parametrize("B,Hkv,longest", [(1, 1, 700), (3, 8, 100), (30, 4, 60), (64, 4, 200), (40, 1, 2000)])
def test_attend_cluster_sizes(lib, B, Hkv, longest):
    """Rows in clusters of 8 down to 1 block, some with fewer tiles than warps."""
    r = random.Random(B)
    lens = [r.randint(0, longest) for _ in range(B - 1)] + [longest]
    cache = filled(lib, lens, 16, Hkv, 128, seed=B + 1)
    q = randn((B, 5 * Hkv, 128), 66)
    o, lse = cache.attend(0, q)
    check_attend(cache, 0, q, None, o, lse, 128 ** -0.5)


def test_extend_by_far_too_much(lib):
    """Token counts up to the largest int are refused entry by entry."""
    cache = make(lib, pages=20, P=4, slots=5, max_pages=8)
    model = CacheModel(cache)
    slots, tokens = [0, 1, 2, 3], [2 ** 31 - 1, 33, 32, -2 ** 31]
    assert cache.extend(ints(slots), ints(tokens)).tolist() == model.extend(slots, tokens) == [-1, -1, 0, -1]
    model.check(cache)
    # a slot at its end stays there, and a row of its pages cannot grow
    assert cache.extend(ints([2]), ints([1])).tolist() == [-1]
    assert cache.extend(ints([2]), ints([0])).tolist() == [32]
    model.check(cache)


def test_attend_into_its_own_queries(lib):
    """O may be Q's memory: every query is read before its row is written."""
    for lens, columns in (([300, 40, 7], None), ([300, 40, 7, 20000], 40000)):
        cache = filled(lib, lens, 16, 2, 128, seed=31)
        if columns:
            cache = widened(lib, cache, columns)
        q = randn((len(lens), 8, 128), 67)
        want = cache.attend(0, q)
        cache.attend(0, q, out=q)
        assert torch.equal(q, want[0])


@pytest.mark.parametrize("B,Hkv,G,d,lo,hi,seed", [
    (70, 2, 8, 128, 159, 713, 1), (28, 8, 4, 256, 1, 416, 2), (76, 2, 1, 256, 18, 646, 3), (17, 8, 2, 256, 1, 397, 4),
    (150, 4, 4, 64, 100, 900, 5), (64, 4, 4, 128, 190, 210, 6), (90, 4, 2, 128, 320, 320, 7), (148, 4, 1, 128, 96, 96, 8)])
def test_attend_rows_and_shares_of_like_length(lib, B, Hkv, G, d, lo, hi, seed):
    """Shares of a few tiles against rows of a few dozen: rows that begin or end
    with a share or a block, or fill one block exactly."""
    r = random.Random(seed)
    lens = [r.randint(lo, hi) for _ in range(B)]
    cache = widened(lib, filled(lib, lens, 16, Hkv, d, seed=seed))
    q = randn((B, Hkv * G, d), 68)
    o, lse = cache.attend(0, q)
    check_attend(cache, 0, q, None, o, lse, d ** -0.5)
