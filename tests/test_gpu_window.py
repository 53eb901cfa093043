"""Sliding window with visible first tokens, forward and backward, against a
plain 64-bit form, element by element within the bounds that the kernels'
roundings give (plain64)."""

import pytest
import torch

import plain64

pytestmark = pytest.mark.gpu


def randn(shape, seed, std=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (std * torch.randn(shape, generator=g, device="cuda")).to(torch.bfloat16)


def run(lib, q, k, v, do, **kw):
    o, lse = lib.forward_general(q, k, v, **kw)
    dq, dk, dv = lib.backward_general(q, k, v, o, lse, do, **kw)
    torch.cuda.synchronize()
    assert lib.last_device_status() == 0
    return dict(o=o, lse=lse, dq=dq, dk=dk, dv=dv)


def compare(got, ref, names=("o", "dq", "dk", "dv")):
    plain64.check_lse(got["lse"], ref["lse"])
    for n in names:
        plain64.check(n, got[n], ref[n], ref[n + "_tol"])


# layout, B, H, Hkv, Nq, Nk, d, window, sinks, key lengths
CASES = [
    ("bhsd", 1, 1, 1, 1, 1, 64, 1, 0, None),
    ("bhsd", 2, 2, 1, 1, 300, 64, 7, 1, None),              # a single query row
    ("bhsd", 1, 2, 2, 129, 129, 64, 1, 0, None),            # each query sees its own key alone
    ("bhsd", 2, 4, 2, 300, 300, 64, 33, 4, None),
    ("bhsd", 1, 2, 2, 640, 640, 64, 128, 0, None),          # tiles that end with the window
    ("bhsd", 1, 2, 1, 640, 640, 128, 128, 128, None),       # first keys fill a tile
    ("bhsd", 1, 2, 1, 700, 700, 128, 200, 130, None),       # ... and one more and a bit
    ("bhsd", 1, 3, 1, 513, 513, 128, 64, 4, None),
    ("bhsd", 1, 2, 1, 257, 900, 128, 100, 5, None),         # fewer queries than keys
    ("bhsd", 1, 2, 1, 900, 257, 64, 100, 5, None),          # rows before the first key see nothing
    ("bhsd", 1, 2, 1, 900, 257, 128, 100, 0, None),
    ("bhsd", 2, 2, 2, 400, 400, 32, 50, 3, None),
    ("bhsd", 2, 2, 1, 400, 400, 96, 50, 3, None),
    ("bhsd", 1, 2, 1, 400, 400, 192, 50, 3, None),
    ("bhsd", 1, 2, 2, 600, 600, 256, 129, 4, None),
    ("bhsd", 1, 4, 1, 384, 384, 256, 1, 0, None),
    ("bshd", 2, 4, 2, 333, 333, 64, 90, 2, [333, 40]),      # lengths before most rows' windows:
    ("bshd", 2, 4, 2, 333, 333, 128, 20, 0, [100, 0]),      # those rows see nothing at all
    ("bshd", 2, 2, 1, 333, 400, 128, 20, 9, [5, 300]),
    ("bhsd", 1, 2, 1, 300, 300, 64, 299, 0, None),          # only the last row loses a key
    ("bhsd", 1, 1, 1, 300, 300, 128, 10, 299, None),        # first keys leave one that can hide
    ("bhsd", 1, 16, 1, 500, 500, 64, 77, 4, None),          # one K / V head for all
]


@pytest.mark.parametrize("layout,B,H,Hkv,Nq,Nk,d,window,sinks,lens", CASES)
def test_window_matches_64_bits(lib, layout, B, H, Hkv, Nq, Nk, d, window, sinks, lens):
    q, do = randn((B, H, Nq, d), 1), randn((B, H, Nq, d), 2)
    k, v = randn((B, Hkv, Nk, d), 3), randn((B, Hkv, Nk, d), 4)
    scale = d ** -0.5
    ref = plain64.padded(q, k, v, scale, lambda b: plain64.visible(
        Nq, Nk, q.device, window=window, sinks=sinks, kv_len=None if lens is None else lens[b]), do)
    turn = (lambda t: t) if layout == "bhsd" else (lambda t: t.transpose(1, 2).contiguous())
    got = run(lib, *(turn(t) for t in (q, k, v, do)), layout=layout, causal=True, scale=scale,
              window=window, sinks=sinks, seqlens_k=lens)
    if layout == "bshd":
        for n in ("o", "dq", "dk", "dv"):
            got[n] = got[n].transpose(1, 2)
    compare(got, ref)


@pytest.mark.parametrize("d,H,Hkv,window,sinks", [(64, 2, 2, 60, 3), (128, 4, 1, 130, 4), (256, 2, 1, 40, 0)])
def test_window_with_dropout(lib, d, H, Hkv, window, sinks):
    B, N, p, seed = 2, 400, 0.25, 77
    q, do = randn((B, H, N, d), 5), randn((B, H, N, d), 6)
    k, v = randn((B, Hkv, N, d), 7), randn((B, Hkv, N, d), 8)
    keep = lib.dropout_mask(B, H, N, p, seed)
    ref = plain64.padded(q, k, v, d ** -0.5, lambda b: plain64.visible(
        N, N, q.device, window=window, sinks=sinks), do, keep, 1 / (1 - p))
    got = run(lib, q, k, v, do, causal=True, window=window, sinks=sinks, dropout_p=p, seed=seed)
    compare(got, ref)


@pytest.mark.parametrize("d", [64, 128])
def test_window_with_a_block_mask(lib, d):
    """Masks combine by AND: a hidden block stays hidden, first tokens included."""
    N, window, sinks = 900, 200, 4
    q, k, v, do = (randn((1, 2, N, d), 10 + i) for i in range(4))
    nb = (N + 127) // 128
    bm = torch.ones((nb, nb), dtype=torch.uint8, device="cuda")
    bm[3:, 0] = 0
    bm[5, 4] = 0
    bm[6, 5:] = 0
    ref = plain64.padded(q, k, v, d ** -0.5, lambda b: plain64.visible(
        N, N, q.device, window=window, sinks=sinks, block_mask=bm), do)
    compare(run(lib, q, k, v, do, causal=True, window=window, sinks=sinks, block_mask=bm), ref)


@pytest.mark.parametrize("d,H,Hkv", [(64, 4, 2), (128, 2, 2), (256, 2, 1)])
def test_window_packed_batch(lib, d, H, Hkv):
    """Packed sequences of 0 to 700 queries, more and fewer keys than queries;
    rows of no sequence stay as they were."""
    lq, lk, window, sinks = [1, 0, 300, 129, 700, 64], [1, 5, 300, 500, 700, 20], 100, 3
    cq = [0] + torch.tensor(lq).cumsum(0).tolist()
    ck = [0] + torch.tensor(lk).cumsum(0).tolist()
    q, do = randn((cq[-1] + 9, H, d), 20), randn((cq[-1] + 9, H, d), 21)
    k, v = randn((ck[-1] + 5, Hkv, d), 22), randn((ck[-1] + 5, Hkv, d), 23)
    out = torch.full_like(q, 7.0)
    dq, dk, dv = torch.full_like(q, 7.0), torch.full_like(k, 7.0), torch.full_like(v, 7.0)
    kw = dict(layout="thd", cu_seqlens_q=cq, cu_seqlens_k=ck, max_seqlen_q=max(lq), max_seqlen_k=max(lk),
              causal=True, window=window, sinks=sinks)
    o, lse = lib.forward_general(q, k, v, out=out, **kw)
    lib.backward_general(q, k, v, o, lse, do, dq=dq, dk=dk, dv=dv, **kw)
    torch.cuda.synchronize()
    assert lib.last_device_status() == 0
    for b, (n, m) in enumerate(zip(lq, lk)):
        if n == 0:
            continue
        rq, rk = slice(cq[b], cq[b + 1]), slice(ck[b], ck[b + 1])
        part = lambda t, r: t[r].transpose(0, 1)[None]  # noqa: E731
        ref = plain64.padded(part(q, rq), part(k, rk), part(v, rk), d ** -0.5,
                             lambda _: plain64.visible(n, m, q.device, window=window, sinks=sinks), part(do, rq))
        got = dict(o=part(o, rq), dq=part(dq, rq), dk=part(dk, rk), dv=part(dv, rk), lse=lse[:, rq][None])
        compare(got, ref)
    for t in (o, dq, dk, dv):
        assert (t[-5:] == 7.0).all()


@pytest.mark.parametrize("d", [64, 128, 256])
def test_long_window_is_no_window(lib, d):
    """A window of all keys hides nothing, in the outputs' every bit; so is a
    window of any length over first keys that cover the sequence."""
    N = 500
    q, k, v = (randn((1, 2, N, d), 30 + i) for i in range(3))
    o, lse = lib.forward_general(q, k, v, causal=True)
    for w, s in ((N, 0), (2 ** 31 - 1, 4), (2 ** 40, 0), (0, 4), (None, None)):
        o2, lse2 = lib.forward_general(q, k, v, causal=True, window=w, sinks=s)
        assert torch.equal(o, o2) and torch.equal(lse, lse2)
    o2, lse2 = lib.forward_general(q, k, v, causal=True, window=5, sinks=N)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)


def test_strided_views(lib):
    """q, k, v as slices of one projection's output, d contiguous."""
    B, N, H, d, window, sinks = 2, 300, 3, 64, 70, 2
    qkv = randn((B, N, 3, H, d), 40)
    q, k, v = qkv[:, :, 0], qkv[:, :, 1], qkv[:, :, 2]
    do = randn((B, N, H, d), 41)
    t = lambda x: x.transpose(1, 2)  # noqa: E731
    ref = plain64.padded(t(q), t(k), t(v), d ** -0.5, lambda b: plain64.visible(
        N, N, q.device, window=window, sinks=sinks), t(do))
    got = run(lib, q, k, v, do, layout="bshd", causal=True, window=window, sinks=sinks)
    compare({n: x if n == "lse" else t(x) for n, x in got.items()}, ref)


def test_captured_and_replayed(lib):
    """Forward and backward in one graph, replayed on new contents, while an
    uncaptured run of the same tensors is kept."""
    N, d, window, sinks = 600, 128, 100, 4
    q, k, v, do = (randn((1, 4, N, d), 50 + i) for i in range(4))
    kw = dict(causal=True, window=window, sinks=sinks)
    eager = run(lib, q, k, v, do, **kw)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        o, lse = lib.forward_general(q, k, v, **kw)
        dq, dk, dv = lib.backward_general(q, k, v, o, lse, do, **kw)
    q.copy_(randn(q.shape, 60))
    g.replay()
    torch.cuda.synchronize()
    ref = plain64.padded(q, k, v, d ** -0.5, lambda b: plain64.visible(
        N, N, q.device, window=window, sinks=sinks), do)
    compare(dict(o=o, lse=lse, dq=dq, dk=dk, dv=dv), ref)
    assert eager["o"].shape == o.shape


@pytest.mark.parametrize("d,H,Hkv,N,window,sinks,p", [
    (128, 4, 2, 3000, 64, 4, 0.0), (64, 3, 3, 3001, 100, 130, 0.0), (256, 2, 1, 2600, 200, 3, 0.0),
    (96, 8, 1, 2500, 1, 257, 0.0), (64, 2, 1, 2049, 300, 1, 0.2)])
def test_first_keys_walks_in_pieces(lib, d, H, Hkv, N, window, sinks, p):
    """Sequences long enough that the first keys' gradients come from several
    units; the same bits every time."""
    q, do = randn((1, H, N, d), 70), randn((1, H, N, d), 71)
    k, v = randn((1, Hkv, N, d), 72), randn((1, Hkv, N, d), 73)
    keep = lib.dropout_mask(1, H, N, p, 9) if p else None
    ref = plain64.padded(q, k, v, d ** -0.5, lambda b: plain64.visible(
        N, N, q.device, window=window, sinks=sinks), do, keep, 1 / (1 - int(p * 65536) / 65536))
    kw = dict(causal=True, window=window, sinks=sinks, dropout_p=p, seed=9)
    got = run(lib, q, k, v, do, **kw)
    compare(got, ref)
    again = run(lib, q, k, v, do, **kw)
    assert torch.equal(got["dk"], again["dk"]) and torch.equal(got["dv"], again["dv"])


def test_first_keys_in_pieces_packed(lib):
    """Sequences with and without pieces, more keys than queries and fewer, and
    a forced split of the group."""
    d, H, Hkv, window, sinks = 128, 4, 1, 90, 140
    lq, lk = [2500, 1, 1400, 700, 1300], [2500, 900, 2300, 30, 1100]
    cq, ck = [0] + torch.tensor(lq).cumsum(0).tolist(), [0] + torch.tensor(lk).cumsum(0).tolist()
    q, do = randn((cq[-1], H, d), 80), randn((cq[-1], H, d), 81)
    k, v = randn((ck[-1], Hkv, d), 82), randn((ck[-1], Hkv, d), 83)
    kw = dict(layout="thd", cu_seqlens_q=cq, cu_seqlens_k=ck, max_seqlen_q=max(lq), max_seqlen_k=max(lk),
              causal=True, window=window, sinks=sinks)
    for parts in (0, 1, 2):
        lib.set_gqa_split(parts)
        try:
            r = run(lib, q, k, v, do, **kw)
        finally:
            lib.set_gqa_split(0)
        for b, (n, m) in enumerate(zip(lq, lk)):
            rq, rk = slice(cq[b], cq[b + 1]), slice(ck[b], ck[b + 1])
            part = lambda t, s: t[s].transpose(0, 1)[None]  # noqa: E731
            ref = plain64.padded(part(q, rq), part(k, rk), part(v, rk), d ** -0.5,
                                 lambda _: plain64.visible(n, m, q.device, window=window, sinks=sinks), part(do, rq))
            compare(dict(o=part(r["o"], rq), dq=part(r["dq"], rq), dk=part(r["dk"], rk), dv=part(r["dv"], rk),
                         lse=r["lse"][:, rq][None]), ref)


@pytest.mark.parametrize("d,Hkv,p", [(64, 2, 0.0), (128, 1, 0.0), (64, 1, 0.25), (256, 2, 0.0)])
def test_own_key_alone_has_no_score_gradient(lib, d, Hkv, p):
    """Window 1 without first tokens: O is V's row, dQ and dK are exactly zero, dV is dO."""
    H, N = 2, 300
    q, do = randn((1, H, N, d), 90), randn((1, H, N, d), 91)
    k, v = randn((1, Hkv, N, d), 92), randn((1, Hkv, N, d), 93)
    got = run(lib, q, k, v, do, causal=True, window=1, dropout_p=p, seed=3)
    assert (got["dq"] == 0).all() and (got["dk"] == 0).all()
    if not p:
        assert torch.equal(got["o"], v.repeat_interleave(H // Hkv, 1))


@pytest.mark.parametrize("d,H,Hkv", [(64, 2, 1), (128, 2, 2)])
def test_window_with_dropout_positions(lib, d, H, Hkv):
    """The keep bits are keyed by the block's place in a longer sequence; the
    window counts the call's own rows."""
    import numpy as np
    import oracle
    N, p, seed, row0, key0, window, sinks = 300, 0.3, 5, 77, 128, 60, 3
    q, do = randn((1, H, N, d), 94), randn((1, H, N, d), 95)
    k, v = randn((1, Hkv, N, d), 96), randn((1, Hkv, N, d), 97)
    keep = np.stack([oracle.dropout_keep(seed, p, 0, h, np.arange(row0, row0 + N), N, key0=key0) for h in range(H)])
    keep = torch.from_numpy(keep)[None].cuda()
    ref = plain64.padded(q, k, v, d ** -0.5, lambda b: plain64.visible(
        N, N, q.device, window=window, sinks=sinks), do, keep, oracle.dropout_scale(p))
    got = run(lib, q, k, v, do, causal=True, window=window, sinks=sinks, dropout_p=p, seed=seed,
              dropout_row0=row0, dropout_key0=key0)
    compare(got, ref)
