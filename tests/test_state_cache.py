"""LayerState.ready keeps the C struct of a state between calls: it has to be formed
again whenever a field's tensor, its memory or the dims are others (host only: the
checks of the tensors are replaced by a record of their arguments)."""
import ctypes as ct

import pytest
import torch

from recurrent_state_quant_lq_amd import lq


@pytest.fixture
def seen(monkeypatch):
    calls = []
    monkeypatch.setattr(lq, "_check", lambda t, name, shape, dtype: calls.append((name, tuple(shape))))
    return calls


def state(B=2, W=4):
    return lq.LayerState.allocate(lq.make_dims(B, 3, 16, 16, W, 1), "cpu")


def pointers(st):
    return [getattr(st, n).data_ptr() for n in lq._STATE_FIELDS]


def held(c):
    return [ct.cast(getattr(c, n), ct.c_void_p).value for n in lq._STATE_FIELDS]


def test_the_struct_is_kept_for_the_same_tensors(seen):
    st = state()
    a = st.ready()
    n = len(seen)
    st.buf_k.fill_(1.0)
    assert st.ready() is a and len(seen) == n and held(a) == pointers(st)


@pytest.mark.parametrize("name", lq._STATE_FIELDS)
def test_a_field_replaced_twice(seen, name):
    """The first replacement may free the old tensor, whose address and id the second can have."""
    for _ in range(20):
        st = state()
        st.ready()
        shape, dt = getattr(st, name).shape, getattr(st, name).dtype
        setattr(st, name, None)
        setattr(st, name, torch.zeros(shape, dtype=dt))
        n = len(seen)
        keep = torch.zeros((4, *shape), dtype=dt)         # (memory of another size in between)
        setattr(st, name, None)
        setattr(st, name, torch.ones(shape, dtype=dt))
        assert held(st.ready()) == pointers(st)
        assert len(seen) > n
        del keep


def test_a_view_of_the_same_memory_is_checked(seen):
    st = state()
    st.ready()
    n = len(seen)
    st.buf_m = st.buf_m.view(-1)[:16]                     # the same address, too few values
    st.ready()
    assert len(seen) > n


def test_memory_exchanged_in_place(seen):
    st = state()
    st.ready()
    n = len(seen)
    st.buf_k.set_(torch.zeros_like(st.buf_k))
    assert held(st.ready()) == pointers(st) and len(seen) > n
    n = len(seen)
    st.sq.data = torch.ones_like(st.sq)
    assert held(st.ready()) == pointers(st) and len(seen) > n


def test_dims_changed(seen):
    st = state(W=4)
    st.ready()
    st.dims.W = 32
    n = len(seen)
    st.ready()
    assert ("buf_k", (2, 3, 32, 16)) in seen[n:]
    st.dims = lq.make_dims(1, 3, 16, 16, 4, 1)
    n = len(seen)
    st.ready()
    assert ("buf_k", (1, 3, 4, 16)) in seen[n:]


def test_a_codec_without_a_buffer(seen):
    st = state()
    st.buf_k = st.buf_m = st.buf_g = None
    c = st.ready(with_buffer=False)
    assert held(c)[:5] == pointers_of_codec(st) and held(c)[5:] == [None] * 3 and st.ready(with_buffer=False) is c


def pointers_of_codec(st):
    return [getattr(st, n).data_ptr() for n in lq._STATE_FIELDS[:5]]


@pytest.mark.parametrize("name", lq._STATE_FIELDS[1:])
def test_a_state_on_two_devices_is_refused(seen, name):
    st = state()
    setattr(st, name, torch.zeros_like(getattr(st, name), device="meta"))
    with pytest.raises(ValueError, match=name):
        st.ready()
