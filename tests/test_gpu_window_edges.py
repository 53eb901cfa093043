"""Sliding window at the ends of its range: one key, pieces of the first keys'
walks together with every other mask and layout, replayed graphs."""

import pytest
import torch

import plain64
from test_gpu_window import compare, randn, run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("layout,B,H,Hkv,d,p", [("bhsd", 2, 4, 2, 64, 0.0), ("bhsd", 3, 2, 2, 128, 0.0),
                                                ("bshd", 2, 4, 1, 128, 0.3), ("bhsd", 2, 2, 1, 256, 0.0),
                                                ("thd", 5, 4, 2, 64, 0.0), ("thd", 4, 2, 1, 128, 0.25)])
def test_own_key_alone_of_one_key(lib, layout, B, H, Hkv, d, p):
    """Window 1 without first tokens over sequences of one key: that key has
    probability 1 whatever the score, so dQ and dK are exactly zero here too."""
    shape = {"bhsd": lambda h: (B, h, 1, d), "bshd": lambda h: (B, 1, h, d), "thd": lambda h: (B, h, d)}[layout]
    q, do, k, v = randn(shape(H), 1), randn(shape(H), 2), randn(shape(Hkv), 3), randn(shape(Hkv), 4)
    kw = dict(layout=layout, causal=True, window=1, dropout_p=p, seed=5)
    if layout == "thd":
        cu = list(range(B + 1))
        kw.update(cu_seqlens_q=cu, cu_seqlens_k=cu, max_seqlen_q=1, max_seqlen_k=1)
    got = run(lib, q, k, v, do, **kw)
    assert (got["dq"] == 0).all() and (got["dk"] == 0).all()
    if not p:
        heads = {"bhsd": 1, "bshd": 2, "thd": 1}[layout]
        assert torch.equal(got["o"], v.repeat_interleave(H // Hkv, heads))


@pytest.mark.parametrize("H,Hkv,N,d,window,sinks", [
    (16, 1, 4200, 128, 300, 4),     # dQ converted by a launch of its own; first keys in pieces
    (16, 2, 4200, 128, 200, 0),     # split units alone
    (16, 1, 4200, 128, 0, 0),       # no window
    (8, 1, 4300, 256, 130, 140),
    (32, 4, 4099, 64, 600, 3),
])
def test_gradients_of_many_row_blocks(lib, H, Hkv, N, d, window, sinks):
    """Grouped heads long enough that dQ is converted apart from dK and dV."""
    q, do = randn((1, H, N, d), 11), randn((1, H, N, d), 12)
    k, v = randn((1, Hkv, N, d), 13), randn((1, Hkv, N, d), 14)
    got = run(lib, q, k, v, do, causal=True, window=window, sinks=sinks)
    mask = plain64.visible(N, N, q.device, window=window, sinks=sinks)
    G, kv = H // Hkv, {}
    for h in range(H):
        r = plain64.head(q[0, h].double(), k[0, h // G].double(), v[0, h // G].double(), d ** -0.5, mask, do[0, h].double())
        plain64.check_lse(got["lse"][0, h], r["lse"])
        for n in ("o", "dq"):
            plain64.check(n, got[n][0, h], r[n], r[n + "_tol"])
        for n in ("dk", "dk_tol", "dv", "dv_tol"):
            kv[n] = kv[n] + r[n] if h % G else r[n]
        if h % G == G - 1:
            for n in ("dk", "dv"):  # (rounded once more, as plain64.padded says)
                plain64.check(n, got[n][0, h // G], kv[n], kv[n + "_tol"] + plain64.BF16 * kv[n].abs())


@pytest.mark.parametrize("kw", [dict(scale=1e300), dict(scale=-1e39), dict(dropout_p=1e39), dict(dropout_row0=2 ** 63),
                                dict(dropout_key0=2 ** 64)])
def test_values_beyond_fp32_are_refused_by_the_library(lib, kw):
    q, k, v = (randn((1, 2, 64, 64), i) for i in range(3))
    o, lse = lib.forward_general(q, k, v, causal=True, window=9)
    with pytest.raises(lib.FaError) as e:
        lib.forward_general(q, k, v, causal=True, window=9, **kw)
    assert e.value.code == 1
    with pytest.raises(lib.FaError) as e:
        lib.backward_general(q, k, v, o, lse, q, causal=True, window=9, **kw)
    assert e.value.code == 1


def test_lengths_beyond_int_are_refused_by_the_library(lib):
    q = randn((8, 2, 64), 1)
    for n in (2 ** 31, 2 ** 32 + 8):
        with pytest.raises(lib.FaError) as e:
            lib.forward_general(q, q, q, layout="thd", cu_seqlens_q=[0, 8], cu_seqlens_k=[0, 8], max_seqlen_q=n,
                                max_seqlen_k=8, causal=True)
        assert e.value.code == 1


@pytest.mark.parametrize("layout,B,H,Hkv,d,lens,mask", [
    ("bshd", 2, 2, 1, 64, [2300, 700], False), ("bhsd", 1, 2, 2, 128, [90], False), ("bshd", 1, 2, 1, 128, None, True),
    ("bhsd", 2, 4, 2, 64, [0, 2299], True), ("bhsd", 1, 2, 1, 256, [1500], True)])
def test_first_keys_in_pieces_under_other_masks(lib, layout, B, H, Hkv, d, lens, mask):
    """The first keys' walks cut into pieces, with key lengths (some before the
    window, some that hide first keys) and a block mask (whole pieces of it empty)."""
    N, window, sinks = 2300, 150, 140
    q, do = randn((B, H, N, d), 21), randn((B, H, N, d), 22)
    k, v = randn((B, Hkv, N, d), 23), randn((B, Hkv, N, d), 24)
    bm = None
    if mask:
        nb = (N + 127) // 128
        bm = torch.ones((nb, nb), dtype=torch.uint8, device="cuda")
        bm[7:, 1] = 0       # the second tile of first keys is hidden from there on
        bm[10:15, 0] = 0
        bm[4, 3:5] = 0
    ref = plain64.padded(q, k, v, d ** -0.5, lambda b: plain64.visible(
        N, N, q.device, window=window, sinks=sinks, kv_len=None if lens is None else lens[b], block_mask=bm), do)
    turn = (lambda t: t) if layout == "bhsd" else (lambda t: t.transpose(1, 2).contiguous())
    got = run(lib, *(turn(t) for t in (q, k, v, do)), layout=layout, causal=True, window=window, sinks=sinks,
              seqlens_k=lens, block_mask=bm)
    if layout == "bshd":
        for n in ("o", "dq", "dk", "dv"):
            got[n] = got[n].transpose(1, 2)
    compare(got, ref)


@pytest.mark.parametrize("d,H,Hkv", [(64, 2, 2), (128, 4, 1)])
def test_first_keys_in_pieces_of_sequences_without_queries(lib, d, H, Hkv):
    """A packed batch in which sequences without queries, or shorter than a piece,
    stand between long ones: their keys' gradients are zero, and so is nobody else's row touched."""
    window, sinks = 100, 130
    lq, lk = [0, 2400, 0, 5, 2200, 0], [300, 2400, 1, 2000, 2300, 129]
    cq, ck = [0] + torch.tensor(lq).cumsum(0).tolist(), [0] + torch.tensor(lk).cumsum(0).tolist()
    q, do = randn((cq[-1], H, d), 31), randn((cq[-1], H, d), 32)
    k, v = randn((ck[-1], Hkv, d), 33), randn((ck[-1], Hkv, d), 34)
    r = run(lib, q, k, v, do, layout="thd", cu_seqlens_q=cq, cu_seqlens_k=ck, max_seqlen_q=max(lq), max_seqlen_k=max(lk),
            causal=True, window=window, sinks=sinks)
    for b, (n, m) in enumerate(zip(lq, lk)):
        rq, rk = slice(cq[b], cq[b + 1]), slice(ck[b], ck[b + 1])
        if n == 0:
            assert (r["dk"][rk] == 0).all() and (r["dv"][rk] == 0).all()
            continue
        part = lambda t, s: t[s].transpose(0, 1)[None]  # noqa: E731
        ref = plain64.padded(part(q, rq), part(k, rk), part(v, rk), d ** -0.5,
                             lambda _: plain64.visible(n, m, q.device, window=window, sinks=sinks), part(do, rq))
        compare(dict(o=part(r["o"], rq), dq=part(r["dq"], rq), dk=part(r["dk"], rk), dv=part(r["dv"], rk),
                     lse=r["lse"][:, rq][None]), ref)


def test_replay_leaves_eager_results_alone(lib):
    """Results of an uncaptured run are the caller's: a graph of the same tensors
    replayed twice, on other contents, does not touch them."""
    N, d, kw = 600, 128, dict(causal=True, window=100, sinks=4)
    q, k, v, do = (randn((1, 4, N, d), 50 + i) for i in range(4))
    eager = run(lib, q, k, v, do, **kw)
    keep = {n: t.clone() for n, t in eager.items()}
    g = torch.cuda.CUDAGraph()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(g, stream=side):
        o, lse = lib.forward_general(q, k, v, **kw)
        lib.backward_general(q, k, v, o, lse, do, **kw)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(o, keep["o"]) and torch.equal(lse, keep["lse"])
    q.copy_(randn(q.shape, 60))
    g.replay()
    torch.cuda.synchronize()
    assert not torch.equal(o, keep["o"])
    for n, t in eager.items():
        assert torch.equal(t, keep[n]), n


def test_two_backwards_at_once(lib):
    """Overlapping calls on two streams, each with its own workspace."""
    d, kw = 64, dict(causal=True, window=70, sinks=5)
    sets = [[randn((1, 4, 2300, d), 10 * i + j) for j in range(4)] for i in (7, 8)]
    want = [run(lib, *s, **kw) for s in sets]
    streams = [torch.cuda.Stream() for _ in sets]
    torch.cuda.synchronize()
    got = []
    for turn in range(4):
        for s, t in zip(streams, sets):
            with torch.cuda.stream(s):
                o, lse = lib.forward_general(*t[:3], **kw)
                got.append((o, lse) + tuple(lib.backward_general(*t[:3], o, lse, t[3], **kw)))
    torch.cuda.synchronize()
    assert lib.last_device_status() == 0
    for i, (o, lse, dq, dk, dv) in enumerate(got):
        w = want[i % 2]
        assert all(torch.equal(a, w[n]) for a, n in ((o, "o"), (lse, "lse"), (dk, "dk"), (dv, "dv")))
        # dQ is summed by atomics, in fp32: the order shows in a bf16 step at most (2^-7 of the value)
        assert ((dq.float() - w["dq"].float()).abs() <= 2.0 ** -7 * w["dq"].float().abs() + 1e-6).all()
