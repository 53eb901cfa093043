"""Sliding window at the ends of its range: one key, pieces of the first keys'
walks together with every other mask and layout, replayed graphs."""

import pytest
import torch

import plain64
from test_gpu_window import randn, run

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
