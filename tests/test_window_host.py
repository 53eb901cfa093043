"""Sliding window: refusals before any launch, and the plain 64-bit form's
gradients against central differences."""

import ctypes

import pytest
import torch

import plain64
from test_abi import A16, _desc


@pytest.mark.parametrize("change,code", [
    (dict(causal=1, window=5, sinks=2), None), (dict(causal=1, window=0, sinks=2), None),
    (dict(causal=1, window=(1 << 31) - 1, sinks=(1 << 31) - 1), None),
    (dict(causal=0, window=5), 1), (dict(causal=1, window=-1), 1), (dict(causal=1, window=5, sinks=-1), 1),
])
def test_window_arguments(lib, change, code):
    so = lib.library()
    a = _desc(lib, **change)
    ws = so.fa_bwd_ex_workspace_size(ctypes.byref(a))
    if code is None:
        assert ws > 0
        return
    assert ws == 0
    assert so.fa_fwd_ex(ctypes.byref(a), A16, A16, A16, A16, A16, None) == code
    assert so.fa_bwd_ex(ctypes.byref(a), A16, A16, A16, A16, A16, A16, A16, A16, A16, A16, 1 << 30,
                        None) == code


def test_binding_refuses_negative_windows(lib):
    for w, s in ((-1, 0), (4, -1)):
        with pytest.raises(ValueError, match="negative"):
            lib._window(w, s)
    assert lib._window(None, None) == (0, 0)
    assert lib._window(2 ** 40, 2 ** 33) == (2 ** 31 - 1, 2 ** 31 - 1)


def test_visible_keys_one_by_one():
    m = plain64.visible(4, 6, "cpu", window=2, sinks=1)
    # positions 2 .. 5, the last two keys and key 0
    want = [[1, 1, 1, 0, 0, 0], [1, 0, 1, 1, 0, 0], [1, 0, 0, 1, 1, 0], [1, 0, 0, 0, 1, 1]]
    assert m.int().tolist() == want
    # more queries than keys: the first rows come before every key, first tokens too
    m = plain64.visible(4, 2, "cpu", window=1, sinks=2)
    assert m.int().tolist() == [[0, 0], [0, 0], [1, 0], [1, 1]]


def test_gradients_against_differences():
    torch.manual_seed(0)
    n, m, d, scale, h = 7, 9, 4, 0.5, 1e-5
    q, k, v, do = (torch.randn(s, d, dtype=torch.float64) for s in (n, m, m, n))
    mask = plain64.visible(n, m, "cpu", window=3, sinks=2)
    r = plain64.head(q, k, v, scale, mask, do)
    for name, t in (("dq", q), ("dk", k), ("dv", v)):
        for at in range(t.numel()):
            f = []
            for s in (h, -h):
                t.view(-1)[at] += s
                f.append((plain64.head(q, k, v, scale, mask)["o"] * do).sum().item())
                t.view(-1)[at] -= s
            assert abs((f[0] - f[1]) / (2 * h) - r[name].reshape(-1)[at].item()) < 1e-7


def test_packed_description_equals_the_fields(lib):
    """The binding packs a description's fields in one step: the same bytes as
    setting them one by one, and the size of the C structure."""
    assert lib._DESC.size == ctypes.sizeof(lib.AttentionDesc)
    a = lib.AttentionDesc()
    values = iter(range(1, 100))
    flat = []
    for name, kind in lib.AttentionDesc._fields_:
        if kind is lib.Strides:
            s = [next(values) for _ in range(3)]
            setattr(a, name, lib.Strides(*s))
            flat += s
        else:
            v = next(values)
            setattr(a, name, v)
            flat.append(v)
    b = lib.AttentionDesc.from_buffer_copy(lib._DESC.pack(*flat))
    for name, kind in lib.AttentionDesc._fields_:
        x, y = getattr(a, name), getattr(b, name)
        if kind is lib.Strides:
            x, y = [(s.batch, s.head, s.row) for s in (x, y)]
        assert x == y, name
