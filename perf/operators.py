"""Cases of the operators that train and serve a language model with windowed
attention and a paged key / value cache:

  window    causal attention in which a query sees the last `window` keys up to
            its own position and the first `sinks` keys of its sequence: forward
            alone (a chunk of a prompt against the keys so far) or forward and
            backward (training), padded or packed, with grouped K / V heads
  decode    attention of one new token per sequence over a paged cache, whole
            or with the same window and sinks
  pages     the cache's book-keeping: growing sequences (pages allocated lowest
            number first, a shared last page copied before it is written), writing
            the new keys and values, forking, freeing and compacting
  step      one decode step as a server runs it: grow every sequence by one
            token, then per layer write the new keys and values and attend

The cache: k and v are bf16 [layers, pages, heads_kv, page_size, d]; `table` int32
[slots, max_pages] holds page numbers (-1: none), `lengths` int32 [slots] the tokens
of each slot, `refs` int32 [pages] how many slots hold a page (0: free).  `book` is
the three of them in one buffer; `run` starts from `book0`, so that a pass can be
made again on the same state.
"""

import math
import random

import torch

own = False  # True: the framework's operators; False: their plain form


# ----------------------------------------------------------------------------
# cases
# ----------------------------------------------------------------------------

def listed():
    return [
        # a few short, ragged samples packed in one batch: fine-tuning at its smallest
        dict(name="window_small_packed", op="window", train=True, packed=True, batch=4, lo=1, hi=257, nq=0, nk=0,
             heads=4, heads_kv=2, d=64, window=96, sinks=2, mix=1),
        # the GPT-2 shape of the benchmark's training workload, with a window
        dict(name="window_gpt2_train", op="window", train=True, packed=False, batch=8, lo=0, hi=0, nq=1024, nk=1024,
             heads=12, heads_kv=12, d=64, window=256, sinks=4, mix=2),
        # long-context training: the benchmark's 16K sequence at d = 128 with grouped heads
        dict(name="window_16k_train", op="window", train=True, packed=False, batch=1, lo=0, hi=0, nq=16384, nk=16384,
             heads=16, heads_kv=4, d=128, window=1024, sinks=4, mix=3),
        # chunked prefill: one chunk of a long prompt against all keys so far
        dict(name="window_prefill_chunk", op="window", train=False, packed=False, batch=1, lo=0, hi=0, nq=2048, nk=32768,
             heads=16, heads_kv=4, d=128, window=4096, sinks=4, mix=4),
        # one user, short context: latency
        dict(name="decode_one", op="decode", batch=1, lo=500, hi=500, heads=16, heads_kv=4, d=128, page=16,
             window=0, sinks=0, mix=5),
        # a server's batch: every length from a greeting to a document
        dict(name="decode_ragged", op="decode", batch=64, lo=1, hi=8192, heads=16, heads_kv=4, d=128, page=16,
             window=0, sinks=0, mix=6),
        # two users with very long contexts
        dict(name="decode_long", op="decode", batch=2, lo=120000, hi=131072, heads=16, heads_kv=4, d=128, page=64,
             window=0, sinks=0, mix=7),
        # many streams that only see a window and the first tokens, one K / V head per query head
        dict(name="decode_window", op="decode", batch=128, lo=64, hi=16384, heads=16, heads_kv=16, d=64, page=32,
             window=1024, sinks=4, mix=8),
        # one step of a server, four layers
        dict(name="step_serving", op="step", batch=32, lo=16, hi=4096, layers=4, heads=16, heads_kv=4, d=128, page=16,
             window=0, sinks=0, mix=9),
        # beam search: surviving beams fork, then every beam grows by a token
        dict(name="pages_beams", op="pages", what="beams", batch=64, lo=30, hi=2000, layers=8, heads_kv=4, d=128, page=16,
             spare=0, mix=10),
        # sequences end, new prompts take their place: free, grow, write
        dict(name="pages_prefill", op="pages", what="prefill", batch=16, lo=1, hi=2048, layers=4, heads_kv=4, d=128, page=32,
             spare=0, mix=11),
        # a cache that has become sparse is packed into its first pages
        dict(name="pages_compact", op="pages", what="compact", batch=64, lo=64, hi=2048, layers=8, heads_kv=4, d=128, page=16,
             spare=3000, mix=12),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    mix = rng.randrange(1 << 30)
    kind = rng.choice(["window", "window", "decode", "decode", "step", "pages"])
    d = rng.choice([32, 64, 96, 128, 128, 192, 256])
    kv = rng.choice([1, 2, 4, 8])
    group = rng.choice([1, 2, 3, 4, 5, 8, 16])
    if kind == "window":
        heads, heads_kv = (kv * group, kv) if kv * group <= 16 else (group, 1)
        sinks = rng.choice([0, 1, 4, 4, rng.randint(1, 200)])
        window = _log_int(rng, 1, 4096)
        if rng.random() < 0.4:
            return dict(op="window", train=True, packed=True, batch=rng.randint(1, 16), lo=1, hi=_log_int(rng, 16, 2048),
                        nq=0, nk=0, heads=heads, heads_kv=heads_kv, d=d, window=window, sinks=sinks, mix=mix)
        train = rng.random() < 0.7
        nq = _log_int(rng, 16, 8192 if train else 2048)
        nk = nq if train else nq + _log_int(rng, 1, 24000)
        batch = max(1, min(rng.randint(1, 8), (1 << 30) // (heads * nq * nk)))
        window = min(window, max(1, (1 << 35) // (batch * heads * nq * d)))
        return dict(op="window", train=train, packed=False, batch=batch, lo=0, hi=0, nq=nq, nk=nk, heads=heads,
                    heads_kv=heads_kv, d=d, window=window, sinks=sinks, mix=mix)
    if kind == "decode":
        hi = _log_int(rng, 16, 131072)
        hi = min(hi, (1 << 27) // (kv * d))
        batch = max(1, min(_log_int(rng, 1, 128), (1 << 27) // (hi * kv * d)))
        window, sinks = (0, 0) if rng.random() < 0.6 else (_log_int(rng, 1, 4096), rng.choice([0, 1, 4, 100]))
        return dict(op="decode", batch=batch, lo=_log_int(rng, 1, hi), hi=hi, heads=kv * group, heads_kv=kv, d=d,
                    page=rng.choice([1, 8, 16, 16, 24, 32, 64, 128, 256]), window=window, sinks=sinks, mix=mix)
    if kind == "step":
        window, sinks = (0, 0) if rng.random() < 0.6 else (_log_int(rng, 1, 2048), rng.choice([0, 1, 4]))
        hi, layers = _log_int(rng, 16, 4096), rng.randint(1, 4)
        batch = max(1, min(_log_int(rng, 1, 64), (1 << 28) // (hi * layers * kv * d)))
        return dict(op="step", batch=batch, lo=1, hi=hi, layers=layers, heads=kv * group,
                    heads_kv=kv, d=d, page=rng.choice([8, 16, 32, 64]), window=window, sinks=sinks, mix=mix)
    what = rng.choice(["beams", "prefill", "compact"])
    page = rng.choice([8, 16, 32, 64])
    return dict(op="pages", what=what, batch=_log_int(rng, 1, 64), lo=1, hi=_log_int(rng, 16, 2048), layers=rng.randint(1, 8),
                heads_kv=min(kv, 4), d=d if d <= 128 else 128, page=page,
                spare=rng.randint(0, 32000 // page) if what == "compact" else 0, mix=mix)


def _lengths(c, n):
    """n lengths from lo to hi, spread over their logarithm; the last one is hi."""
    r = random.Random(c["mix"])
    return [_log_int(r, c["lo"], c["hi"]) for _ in range(n - 1)] + [c["hi"]]


def _visible(length, window, sinks):
    """Keys that the last position of a sequence sees."""
    return length if window <= 0 else min(length, window + min(sinks, max(0, length - window)))


def _pairs(nq, nk, window, sinks):
    """(query, key) pairs that the mask leaves, queries aligned to the last keys."""
    first = nk - nq
    return sum(_visible(p + 1, window, sinks) for p in range(max(first, 0), nk))


# ----------------------------------------------------------------------------
# inputs
# ----------------------------------------------------------------------------

def _randn(shape, gen):
    return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32).to(torch.bfloat16)


def _pool(shape, gen):
    """A cache's pages: filled layer by layer, so that no fp32 copy of all of it is made."""
    return torch.stack([_randn(shape[1:], gen) for _ in range(shape[0])])


def _book(rows, lengths, max_pages, pages):
    """table, lengths and refs (host lists) in one device buffer, and its views."""
    table = torch.full((len(rows), max_pages), -1, dtype=torch.int32)
    refs = torch.zeros(pages, dtype=torch.int32)
    for s, row in enumerate(rows):
        table[s, : len(row)] = torch.tensor(row, dtype=torch.int32)
        refs += torch.bincount(torch.tensor(row, dtype=torch.int64), minlength=pages).to(torch.int32)
    flat = torch.cat([table.reshape(-1), torch.tensor(lengths, dtype=torch.int32), refs]).cuda()
    n = table.numel()
    return flat, flat[:n].view(len(rows), max_pages), flat[n:n + len(rows)], flat[n + len(rows):]


def prepare(case, seed):
    c = case
    gen = torch.Generator(device="cuda").manual_seed(seed)
    host = random.Random(seed)
    s = dict(c=c, scale=c["d"] ** -0.5)
    if c["op"] == "window":
        H, Hkv, d = c["heads"], c["heads_kv"], c["d"]
        if c["packed"]:
            lens = _lengths(c, c["batch"])
            cu = [0]
            for n in lens:
                cu.append(cu[-1] + n)
            s["cu"] = torch.tensor(cu, dtype=torch.int32, device="cuda")
            s["lens"], s["longest"] = lens, max(lens)
            qs, ks = (cu[-1], H, d), (cu[-1], Hkv, d)
        else:
            qs, ks = (c["batch"], H, c["nq"], d), (c["batch"], Hkv, c["nk"], d)
        s["q"], s["k"], s["v"] = _randn(qs, gen), _randn(ks, gen), _randn(ks, gen)
        if c["train"]:
            s["do"] = _randn(qs, gen)
        return s
    P, n = c["page"], c["batch"]
    L = c.get("layers", 1)
    lens = _lengths(c, n)
    if c["op"] != "pages":
        slots, rows_of = n, list(range(n))
    elif c["what"] == "beams":
        slots, rows_of = n, list(range(n))
    else:
        slots, rows_of = 2 * n, list(range(n))
    need = [-(-x // P) for x in lens]
    max_pages = -(-c["hi"] // P) + 1
    # room for the sequences, for the growth of every slot, and the spare pages
    pages = sum(need) + (sum(need) if c.get("what") == "prefill" else 0) + 2 * n + c.get("spare", 0)
    order = list(range(pages))
    host.shuffle(order)
    rows, at = [[] for _ in range(slots)], 0
    for r, k in zip(rows_of, need):
        rows[r] = order[at:at + k]
        at += k
    lens_of = lens + [0] * (slots - n)
    s["book0"], _, _, _ = _book(rows, lens_of, max_pages, pages)
    s["book"], s["table"], s["lengths"], s["refs"] = _book(rows, lens_of, max_pages, pages)
    shape = (L, pages, c["heads_kv"], P, c["d"])
    s["k"], s["v"] = _pool(shape, gen), _pool(shape, gen)
    if c["op"] == "decode":
        s["q"] = _randn((n, c["heads"], c["d"]), gen)
        s["slots"] = torch.arange(n, dtype=torch.int32, device="cuda")
    elif c["op"] == "step":
        s["q"] = _randn((L, n, c["heads"], c["d"]), gen)
        s["slots"] = torch.arange(n, dtype=torch.int32, device="cuda")
        s["tokens"] = torch.ones(n, dtype=torch.int32, device="cuda")
        s["new"] = _randn((2, L, n, c["heads_kv"], c["d"]), gen)
    elif c["what"] == "beams":
        # a quarter of the beams survive and take the others' places
        parents = [host.randrange(max(1, n // 4)) * 4 % n for _ in range(n)]
        s["parents"] = torch.tensor(parents, dtype=torch.int32, device="cuda")
        s["slots"] = torch.arange(n, dtype=torch.int32, device="cuda")
        s["tokens"] = torch.ones(n, dtype=torch.int32, device="cuda")
        s["new"] = _randn((2, L, n, c["heads_kv"], c["d"]), gen)
    elif c["what"] == "prefill":
        # the second half of the slots receives prompts, every other old sequence ends
        s["ended"] = torch.tensor(list(range(0, n, 2)), dtype=torch.int32, device="cuda")
        s["slots"] = torch.arange(n, 2 * n, dtype=torch.int32, device="cuda")
        s["tokens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
        cu = [0]
        for x in lens:
            cu.append(cu[-1] + x)
        s["cu"] = torch.tensor(cu, dtype=torch.int32, device="cuda")
        s["new"] = _randn((2, L, cu[-1], c["heads_kv"], c["d"]), gen)
    if own:
        import io_aware_exact_20_b200 as fa
        s["cache"] = fa.PagedCache(s["k"], s["v"], s["table"], s["lengths"], s["refs"])
    return s


# ----------------------------------------------------------------------------
# plain forms
# ----------------------------------------------------------------------------

def _plain_attention(q, k, v, do, scale, mask):
    """q, do [B, H, N, d], k, v [B, Hkv, M, d], mask [B, 1, N, M] (True: seen), all fp32."""
    B, H, N, d = q.shape
    G = H // k.shape[1]
    kx, vx = k.repeat_interleave(G, 1), v.repeat_interleave(G, 1)
    x = (q @ kx.transpose(-1, -2)).mul_(scale).masked_fill_(~mask, -math.inf)
    m = x.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, torch.zeros_like(m), m)
    p = x.sub_(m).exp_()
    l = p.sum(-1, keepdim=True)
    lse = torch.where(l > 0, m + l.log(), torch.full_like(l, -math.inf)).squeeze(-1)
    p = p.div_(torch.where(l > 0, l, torch.ones_like(l)))
    o = p @ vx
    if do is None:
        return o, lse
    dp = do @ vx.transpose(-1, -2)
    dv = (p.transpose(-1, -2) @ do).view(B, -1, G, *v.shape[2:]).sum(2)
    ds = dp.sub_((p * dp).sum(-1, keepdim=True)).mul_(p).mul_(scale)
    dk = (ds.transpose(-1, -2) @ q).view(B, -1, G, *k.shape[2:]).sum(2)
    return o, lse, ds @ kx, dk, dv


def _plain_window(s):
    c = s["c"]
    q, k, v, do = s["q"].float(), s["k"].float(), s["v"].float(), s["do"].float() if c["train"] else None
    dev = q.device
    if c["packed"]:
        cu, N = s["cu"].long(), s["longest"]
        n = cu[1:] - cu[:-1]
        at = torch.arange(N, device=dev)
        live = at[None, :] < n[:, None]                                  # [B, N]
        row = torch.where(live, cu[:-1, None] + at[None, :], torch.zeros_like(cu[:-1, None]))
        q, k, v, do = (t[row].transpose(1, 2) for t in (q, k, v, do))   # [B, heads, N, d]
        do = do * live[:, None, :, None]
        i, j = at[None, :, None], at[None, None, :]
        mask = (live[:, :, None] & live[:, None, :])
    else:
        i = (torch.arange(c["nq"], device=dev) + c["nk"] - c["nq"])[None, :, None]
        j = torch.arange(c["nk"], device=dev)[None, None, :]
        mask = torch.ones((1, 1, 1), dtype=torch.bool, device=dev)
    mask = (mask & (j <= i) & ((j > i - c["window"]) | (j < c["sinks"])))[:, None]
    out = _plain_attention(q, k, v, do, s["scale"], mask)
    if c["packed"]:
        out = [t.movedim(1, 2)[live] for t in out]                       # [T, heads(, d)]
        out[1] = out[1].transpose(0, 1).contiguous()                     # LSE [heads, T]
    return [out[0].bfloat16(), out[1]] + [t.bfloat16() for t in out[2:]]


def _plain_decode(s, layer, q, slots, length):
    """One query per slot over its pages; length [n]: the keys of each slot."""
    c = s["c"]
    P, N = c["page"], s["table"].shape[1] * c["page"]
    rows = s["table"][slots.long()].long().clamp_min(0)                  # [n, max_pages]
    pick = lambda t: t[layer][rows].transpose(1, 2).reshape(len(rows), c["heads_kv"], N, c["d"]).float()  # noqa: E731
    j = torch.arange(N, device=q.device)[None, :]
    last = length.long()[:, None]
    mask = j < last
    if c["window"] > 0:
        mask = mask & ((j >= last - c["window"]) | (j < c["sinks"]))
    k, v = pick(s["k"]), pick(s["v"])
    n, Hkv, d = len(rows), c["heads_kv"], c["d"]
    qg = q.float().view(n, Hkv, -1, d)
    x = (qg @ k.transpose(-1, -2)).mul_(s["scale"]).masked_fill_(~mask[:, None, None, :], -math.inf)
    m = x.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, torch.zeros_like(m), m)
    p = x.sub_(m).exp_()
    l = p.sum(-1, keepdim=True)
    o = (p @ v) / torch.where(l > 0, l, torch.ones_like(l))
    lse = torch.where(l > 0, m + l.log(), torch.full_like(l, -math.inf))
    return o.reshape(n, -1, d).bfloat16(), lse.reshape(n, -1)


def _plain_extend(s, slots, tokens):
    """Grows slots[i] by tokens[i]: the first new position of each, -1 where it is not granted."""
    table, lengths, refs, P = s["table"], s["lengths"], s["refs"], s["c"]["page"]
    n, (S, M) = len(slots), table.shape
    i = torch.arange(n, device=slots.device)
    sl = slots.long()
    inside = (sl >= 0) & (sl < S)
    sl = torch.where(inside, sl, torch.zeros_like(sl))
    again = ((slots[:, None] == slots[None, :]) & (i[None, :] < i[:, None])).any(1)
    length, more = lengths[sl].long(), tokens.long()
    have, want = (length + P - 1) // P, (length + more + P - 1) // P
    tail = table[sl, (have - 1).clamp_min(0)].long()
    shared = (length % P != 0) & (more > 0) & (refs[tail.clamp_min(0)] > 1)
    fine = inside & ~again & (more >= 0) & (want <= M)
    need = torch.where(fine, want - have + shared, torch.zeros_like(want))
    upto = need.cumsum(0)
    free = torch.argsort((refs != 0).int(), stable=True)
    granted = fine & ((need == 0) | (upto <= (refs == 0).sum()))
    # the new pages of entry i are its columns have - shared .. want - 1
    col = torch.arange(M, device=slots.device)[None, :]
    first = (have - shared.long())[:, None]
    new = granted[:, None] & (col >= first) & (col < want[:, None])
    which = ((upto - need)[:, None] + col - first).clamp(0, len(free) - 1)
    rows = torch.where(new, free[which], table[sl].long())
    copied = granted & shared
    src, used = tail[copied], (length % P)[copied]
    dst = rows[i, (have - 1).clamp_min(0)][copied]
    live = (torch.arange(P, device=slots.device)[None, :] < used[:, None])[None, :, None, :, None]
    s["k"][:, dst] = torch.where(live, s["k"][:, src], s["k"][:, dst])
    s["v"][:, dst] = torch.where(live, s["v"][:, src], s["v"][:, dst])
    refs.index_add_(0, src, torch.full_like(src, -1, dtype=torch.int32))
    refs[free[which][new]] = 1
    table[sl[granted]] = rows[granted].int()
    lengths[sl[granted]] = (length + more)[granted].int()
    return torch.where(granted, length, torch.full_like(length, -1)).int()


def _plain_write(s, layer, k, v, slots, start, cu=None):
    """Puts k, v [T, heads_kv, d] at positions start[i] .. of slots[i]; start[i] < 0: nothing."""
    T, P = len(k), s["c"]["page"]
    t = torch.arange(T, device=k.device)
    entry = t if cu is None else torch.searchsorted(cu[1:].contiguous(), t, right=True)
    pos = start[entry].long() + (0 if cu is None else t - cu[entry].long())
    put = start[entry] >= 0
    pos, entry, t = pos[put], entry[put], t[put]
    page = s["table"][slots[entry].long(), pos // P].long()
    s["k"][layer][page, :, pos % P] = k[t]
    s["v"][layer][page, :, pos % P] = v[t]


def _plain_free(s, slots):
    rows = s["table"][slots.long()].long()
    held = rows[rows >= 0]
    s["refs"].index_add_(0, held, torch.full_like(held, -1, dtype=torch.int32))
    s["table"][slots.long()] = -1
    s["lengths"][slots.long()] = 0


def _plain_fork(s, src, dst):
    """Slot dst[i] takes src[i]'s pages and length (all read before any is replaced); src[i] == dst[i]: it stays."""
    table, lengths, refs = s["table"], s["lengths"], s["refs"]
    moved = src != dst
    src, dst = src[moved].long(), dst[moved].long()
    rows, old, length = table[src], table[dst].long(), lengths[src]
    held = rows[rows >= 0].long()
    refs.index_add_(0, held, torch.ones_like(held, dtype=torch.int32))
    held = old[old >= 0]
    refs.index_add_(0, held, torch.full_like(held, -1, dtype=torch.int32))
    table[dst] = rows
    lengths[dst] = length


def _plain_compact(s):
    """Moves the used pages with the highest numbers into the free ones with the lowest; the pages in use."""
    refs = s["refs"]
    used = refs > 0
    count = used.sum()
    at = torch.arange(len(refs), device=refs.device)
    src = torch.nonzero(used & (at >= count))[:, 0]
    dst = torch.nonzero(~used & (at < count))[:, 0]
    s["k"][:, dst] = s["k"][:, src]
    s["v"][:, dst] = s["v"][:, src]
    refs[dst] = refs[src]
    refs[src] = 0
    now = at.clone()
    now[src] = dst
    s["table"].copy_(torch.where(s["table"] >= 0, now[s["table"].long().clamp_min(0)].int(), s["table"]))
    return count.int().reshape(1)


# ----------------------------------------------------------------------------
# one pass
# ----------------------------------------------------------------------------

def run(state):
    s, c = state, state["c"]
    if c["op"] == "window":
        if not own:
            return _plain_window(s)
        import io_aware_exact_20_b200 as fa
        kw = dict(layout="bhsd", causal=True, window=c["window"], sinks=c["sinks"], scale=s["scale"])
        if c["packed"]:
            kw.update(layout="thd", cu_seqlens_q=s["cu"], cu_seqlens_k=s["cu"], max_seqlen_q=s["longest"],
                      max_seqlen_k=s["longest"])
        o, lse = fa.forward_general(s["q"], s["k"], s["v"], **kw)
        if not c["train"]:
            return [o, lse]
        return [o, lse, *fa.backward_general(s["q"], s["k"], s["v"], o, lse, s["do"], **kw)]
    win = dict(window=c.get("window", 0), sinks=c.get("sinks", 0))
    if c["op"] == "decode":
        if own:
            return list(s["cache"].attend(0, s["q"], s["slots"], scale=s["scale"], **win))
        return list(_plain_decode(s, 0, s["q"], s["slots"], s["lengths"]))
    s["book"].copy_(s["book0"])
    out = {}
    if c["op"] == "step":
        if own:
            cache = s["cache"]
            out["start"] = cache.extend(s["slots"], s["tokens"])
            for layer in range(c["layers"]):
                cache.write(layer, s["new"][0, layer], s["new"][1, layer], s["slots"], out["start"])
                out["o%d" % layer], out["lse%d" % layer] = cache.attend(layer, s["q"][layer], s["slots"], scale=s["scale"], **win)
        else:
            out["start"] = _plain_extend(s, s["slots"], s["tokens"])
            _plain_layers(s, out)
    elif c["what"] == "beams":
        if own:
            cache = s["cache"]
            cache.fork(s["parents"], s["slots"])
            out["start"] = cache.extend(s["slots"], s["tokens"])
            for layer in range(c["layers"]):
                cache.write(layer, s["new"][0, layer], s["new"][1, layer], s["slots"], out["start"])
        else:
            _plain_fork(s, s["parents"], s["slots"])
            out["start"] = _plain_extend(s, s["slots"], s["tokens"])
            _plain_layers(s, out)
    elif c["what"] == "prefill":
        if own:
            cache = s["cache"]
            cache.free(s["ended"])
            out["start"] = cache.extend(s["slots"], s["tokens"])
            for layer in range(c["layers"]):
                cache.write(layer, s["new"][0, layer], s["new"][1, layer], s["slots"], out["start"], cu_seqlens=s["cu"])
        else:
            _plain_free(s, s["ended"])
            out["start"] = _plain_extend(s, s["slots"], s["tokens"])
            _plain_layers(s, out)
    else:
        out["used"] = s["cache"].compact() if own else _plain_compact(s)
    out.update(k=s["k"], v=s["v"], table=s["table"], lengths=s["lengths"], refs=s["refs"])
    return out


def _plain_layers(s, out):
    """Every layer's writes, and its attention in a decode step."""
    c, cu = s["c"], s.get("cu")
    for layer in range(c["layers"]):
        _plain_write(s, layer, s["new"][0, layer], s["new"][1, layer], s["slots"], out["start"], cu)
        if c["op"] == "step":
            out["o%d" % layer], out["lse%d" % layer] = _plain_decode(s, layer, s["q"][layer], s["slots"], s["lengths"])


# ----------------------------------------------------------------------------
# what a pass cannot do without
# ----------------------------------------------------------------------------

def work(case):
    c = case
    if c["op"] == "window":
        H, Hkv, d = c["heads"], c["heads_kv"], c["d"]
        seqs = [(n, n) for n in _lengths(c, c["batch"])] if c["packed"] else [(c["nq"], c["nk"])] * c["batch"]
        tq = sum(a for a, _ in seqs)
        # a K / V row that no query sees is not read, its gradient is written all the same
        seen = sum(min(b, a + min(c["window"], b) + c["sinks"]) for a, b in seqs)
        tk = sum(b for _, b in seqs)
        if c["packed"]:
            pairs = sum(_pairs(a, b, c["window"], c["sinks"]) for a, b in seqs)
        else:
            pairs = c["batch"] * _pairs(c["nq"], c["nk"], c["window"], c["sinks"])
        fwd_b = 2 * d * (2 * tq * H + 2 * seen * Hkv) + 4 * tq * H
        fwd_f = 4 * d * H * pairs
        if not c["train"]:
            return dict(bytes=fwd_b, flops=fwd_f)
        # q, k, v, dO read; o, lse, dq, dk, dv written
        return dict(bytes=2 * d * (4 * tq * H + 2 * seen * Hkv + 2 * tk * Hkv) + 4 * tq * H, flops=3.5 * fwd_f)
    row = 2 * c["heads_kv"] * c["d"]  # bytes of one token's keys (or values) in one layer
    lens = _lengths(c, c["batch"])
    P, n, L = c["page"], c["batch"], c.get("layers", 1)
    need = [-(-x // P) for x in lens]
    if c["op"] in ("decode", "step"):
        grow = 1 if c["op"] == "step" else 0
        vis = sum(_visible(x + grow, c["window"], c["sinks"]) for x in lens)
        ids = 4 * sum(-(-_visible(x + grow, c["window"], c["sinks"]) // P) for x in lens)
        by = L * (2 * row * vis + n * c["heads"] * (4 * c["d"] + 4)) + ids + 4 * n
        if grow:
            by += L * 4 * row * n + 20 * n
        return dict(bytes=by, flops=4 * c["d"] * c["heads"] * L * vis)
    if c["what"] == "beams":
        # table rows read and written, each beam's last page copied as far as it is in use, a token written
        used = sum(x % P for x in lens)
        return dict(bytes=8 * sum(need) + L * row * (4 * used + 4 * n) + 16 * n, flops=0)
    if c["what"] == "prefill":
        return dict(bytes=4 * (2 * sum(need) + sum(need[0::2])) + L * row * 4 * sum(lens) + 16 * n, flops=0)
    pages = sum(need) + 2 * n + c["spare"]
    # pages in use past the end of the packed part, as they lie in a shuffled pool
    moved = sum(need) * (pages - sum(need)) / pages
    return dict(bytes=4 * pages + 8 * sum(need) + L * row * P * 4 * moved, flops=0)


# ----------------------------------------------------------------------------
# the definition, in 64 bits
# ----------------------------------------------------------------------------

def _exact_rows(q, k, v, first, window, sinks, scale, do=None):
    """Rows first .. of one head's sequence, a block of rows at a time, over only the keys that the block can see."""
    nq, nk, dev = len(q), len(k), q.device
    o, lse = torch.zeros_like(q), torch.full((nq,), -math.inf, dtype=torch.float64, device=dev)
    dq, dk, dv = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
    step = 2048
    for a in range(0, nq, step):
        b = min(nq, a + step)
        lo, hi = first + a - window + 1, min(nk, first + b)
        if hi <= 0:
            continue
        keys = sorted(set(range(0, min(sinks, hi))) | set(range(max(0, lo), hi)))
        j = torch.tensor(keys, device=dev)
        pos = torch.arange(first + a, first + b, device=dev)[:, None]
        seen = (j <= pos) & ((pos - j < window) | (j < sinks))
        w = (q[a:b] @ k[j].T * scale).masked_fill(~seen, -math.inf)
        lse[a:b] = torch.logsumexp(w, 1)
        p = torch.where(seen, torch.exp(w - lse[a:b, None]), torch.zeros_like(w))
        o[a:b] = p @ v[j]
        if do is not None:
            g = do[a:b] @ v[j].T
            t = p * (g - (do[a:b] * o[a:b]).sum(1, keepdim=True)) * scale
            dq[a:b] = t @ k[j]
            dk.index_add_(0, j, t.T @ q[a:b])
            dv.index_add_(0, j, p.T @ do[a:b])
    return o, lse, dq, dk, dv


def _exact_window(c, s):
    G = c["heads"] // c["heads_kv"]
    q, k, v = s["q"].double(), s["k"].double(), s["v"].double()
    do = s["do"].double() if c["train"] else None
    o, dq, dk, dv = torch.zeros_like(q), torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
    lse = torch.zeros((c["heads"], q.shape[0]) if c["packed"] else q.shape[:3], dtype=torch.float64, device=q.device)
    at = 0
    for b in range(c["batch"]):
        if c["packed"]:
            rows = slice(at, at + s["lens"][b])
            at += s["lens"][b]
        for h in range(c["heads"]):
            iq, ik = ((rows, h), (rows, h // G)) if c["packed"] else ((b, h), (b, h // G))
            first = 0 if c["packed"] else c["nk"] - c["nq"]
            got = _exact_rows(q[iq], k[ik], v[ik], first, c["window"], c["sinks"], s["scale"], None if do is None else do[iq])
            o[iq], dq[iq] = got[0], got[2]
            lse[(h, rows) if c["packed"] else (b, h)] = got[1]
            dk[ik] += got[3]
            dv[ik] += got[4]
    return [o, lse, dq, dk, dv] if c["train"] else [o, lse]


def _exact_decode(c, s, layer, q, table, lengths):
    """table, lengths: host lists."""
    G, P = c["heads"] // c["heads_kv"], c["page"]
    o = torch.zeros(q.shape, dtype=torch.float64, device=q.device)
    lse = torch.full(q.shape[:2], -math.inf, dtype=torch.float64, device=q.device)
    for b, n in enumerate(lengths):
        pos = [j for j in range(n) if c["window"] <= 0 or j >= n - c["window"] or j < c["sinks"]]
        if not pos:
            continue
        page = torch.tensor([table[b][j // P] for j in pos], device=q.device)
        slot = torch.tensor([j % P for j in pos], device=q.device)
        for h in range(c["heads_kv"]):
            k, v = s["k"][layer][page, h, slot].double(), s["v"][layer][page, h, slot].double()
            w = q[b, h * G:(h + 1) * G].double() @ k.T * s["scale"]
            lse[b, h * G:(h + 1) * G] = torch.logsumexp(w, 1)
            o[b, h * G:(h + 1) * G] = torch.softmax(w, 1) @ v
    return o, lse


def exact(case, seed):
    c, s = case, prepare(case, seed)
    if c["op"] == "window":
        return _exact_window(c, s)
    table, lengths, refs = s["table"].tolist(), s["lengths"].tolist(), s["refs"].tolist()
    if c["op"] == "decode":
        return list(_exact_decode(c, s, 0, s["q"], table, lengths))
    # a server's book-keeping, one slot after the other
    P, k, v, out = c["page"], s["k"], s["v"], {}
    if c.get("what") == "compact":
        used = sum(r > 0 for r in refs)
        holes = [p for p in range(used) if refs[p] == 0]
        for p in range(used, len(refs)):
            if refs[p]:
                to = holes.pop(0)
                k[:, to], v[:, to] = k[:, p].clone(), v[:, p].clone()
        return dict(used=None, k=k.double(), v=v.double(), table=None, lengths=None, refs=None)
    if c.get("what") == "beams":
        before = [list(row) for row in table], list(lengths)
        for i, parent in enumerate(s["parents"].tolist()):
            table[i], lengths[i] = list(before[0][parent]), before[1][parent]
        refs = [0] * len(refs)
        for row in table:
            for p in row:
                if p >= 0:
                    refs[p] += 1
    if c.get("what") == "prefill":
        for x in s["ended"].tolist():
            for p in table[x]:
                if p >= 0:
                    refs[p] -= 1
            table[x], lengths[x] = [-1] * len(table[x]), 0
    shared = [r > 1 for r in refs]
    spare = [p for p, r in enumerate(refs) if r == 0]
    cu = s["cu"].tolist() if "cu" in s else None
    for i, x in enumerate(s["slots"].tolist()):
        n, start = s["tokens"].tolist()[i], lengths[x]
        if start % P and shared[table[x][start // P]]:
            old, to = table[x][start // P], spare.pop(0)
            k[:, to, :, :start % P], v[:, to, :, :start % P] = k[:, old, :, :start % P], v[:, old, :, :start % P]
            table[x][start // P] = to
        for page in range(-(-start // P), -(-(start + n) // P)):
            table[x][page] = spare.pop(0)
        lengths[x] += n
        a = i if cu is None else cu[i]
        at = torch.tensor([table[x][(start + t) // P] for t in range(n)], device="cuda")
        row = (start + torch.arange(n, device="cuda")) % P
        for layer in range(c["layers"]):
            k[layer][at, :, row] = s["new"][0, layer, a:a + n]
            v[layer][at, :, row] = s["new"][1, layer, a:a + n]
    if c["op"] == "step":
        for layer in range(c["layers"]):
            out["o%d" % layer], out["lse%d" % layer] = _exact_decode(c, s, layer, s["q"][layer], table, lengths)
    out.update(start=None, k=k.double(), v=v.double(), table=None, lengths=None, refs=None)
    return out
