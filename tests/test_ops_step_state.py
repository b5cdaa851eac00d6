"""What the plans of clipping and AdamW look at in every call (CPU): stand-ins for CUDA tensors,
addresses that are never dereferenced."""
import ctypes

import pytest

from tests.test_ops_step_refusals import F, H, Tensor, _plans


def _addresses(at, n=2):
    return list((ctypes.c_uint64 * n).from_address(at))


def test_moments_are_looked_at_in_every_step(monkeypatch):
    # a moment's memory may move between steps (`.data = `, set_, a storage resized away and back)
    _, o, calls = _plans(monkeypatch)
    seen = []
    o._run = lambda *a: seen.append((_addresses(a[4]), _addresses(a[5]))) or 0
    g, p = [Tensor(F, (4, 6)), Tensor(H, (7,))], [Tensor(F, (4, 6)), Tensor(F, (7,))]
    for moved in (None, o.m[0], o.v[1]):
        if moved is not None:
            moved._at += 1 << 24
        o.step(p, g, 0.1)
        assert seen[-1] == ([t._at for t in o.m], [t._at for t in o.v])
    o.v[0]._index = 1  # on another GPU
    with pytest.raises(ValueError):
        o.step(p, g, 0.1)
    assert len(seen) == 3


def test_copies_may_be_an_iterator(monkeypatch):
    # as the other lists
    _, o, calls = _plans(monkeypatch)
    seen = []
    o._run = lambda *a: seen.append(_addresses(a[6])) or 0
    g, p = [Tensor(F, (4, 6)), Tensor(H, (7,))], [Tensor(F, (4, 6)), Tensor(F, (7,))]
    low = [Tensor(H, (4, 6), at=1 << 21), Tensor(H, (7,), at=1 << 22)]
    for some in (low, [None, low[1]], [low[0], None], [None, None]):
        for kind in (list, tuple, iter):
            o.step(iter(p), iter(g), 0.1, low=kind(some))
            assert seen[-1] == [t._at if t else 0 for t in some]
