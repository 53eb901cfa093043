"""The binding's packed description: values that the C types cannot hold reach the
library as what it refuses."""

import ctypes

import pytest

from test_abi import A16, _desc

INT32, INT64 = 2 ** 31, 2 ** 63


def values(lib, a):
    """A description's fields in order, as the binding packs them."""
    out = []
    for name, kind in lib.AttentionDesc._fields_:
        x = getattr(a, name)
        out += [x.batch, x.head, x.row] if kind is lib.Strides else [x or 0]
    return out


def place(lib, name):
    at = 0
    for field, kind in lib.AttentionDesc._fields_:
        if field == name:
            return at
        at += 3 if kind is lib.Strides else 1


def test_values_that_fit_are_packed_as_they_are(lib):
    a = _desc(lib)
    assert lib._pack(*values(lib, a)) == bytes(a)
    assert len(lib._DESC_CODES) == len(values(lib, a))


@pytest.mark.parametrize("name,value", [
    ("softmax_scale", 1e300), ("softmax_scale", -1e39), ("dropout_p", 1e39), ("batch", INT32), ("heads", 2 ** 32 + 4),
    ("seqlen_q", INT32), ("seqlen_k", 2 ** 32 + 64), ("heads_kv", 2 ** 40), ("q", INT64), ("dropout_row0", INT64),
    ("dropout_key0", 2 ** 64 + 8)])
def test_values_beyond_their_types_are_refused_by_the_library(lib, name, value):
    a = _desc(lib)
    v = values(lib, a)
    v[place(lib, name)] = value
    b = lib.AttentionDesc.from_buffer_copy(lib._pack(*v))
    so = lib.library()
    assert so.fa_fwd_ex(ctypes.byref(b), A16, A16, A16, A16, A16, None) == 1
    assert so.fa_bwd_ex_workspace_size(ctypes.byref(b)) == 0


def test_what_is_no_number_is_an_error_of_the_binding(lib):
    v = values(lib, _desc(lib))
    v[place(lib, "batch")] = "two"
    with pytest.raises(Exception):
        lib._pack(*v)
