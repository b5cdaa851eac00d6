"""What the plans look at and count in every call (CPU): stand-ins for CUDA tensors, or tensors of
the CPU for entry points that do nothing; addresses are never dereferenced."""
import ctypes

import pytest
import torch

import asr_tiled_tanh_gb300 as rn
from asr_tiled_tanh_gb300 import ops
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


@pytest.mark.parametrize("helper", [True, False])
def test_writes_are_counted(helper):
    a, b = torch.zeros(3), torch.zeros(4)
    with torch.inference_mode():
        c = torch.zeros(5)  # has no count
    plan = rn.GradClip([(3,)], device="cpu")
    if helper:
        plan._fast = ops._helper()
        assert plan._fast is not None  # it was built
    plan._wrote(a, None, [b, None, c, a[:2]], c)
    assert (a._version, b._version) == (2, 1)
    plan._wrote(None)
    with torch.inference_mode():
        plan._wrote([b], c)
    assert (a._version, b._version) == (2, 2)


def _on_the_cpu(monkeypatch, plan, *entries):
    """The plan takes tensors of the CPU; its C functions do nothing."""
    monkeypatch.setattr(ops, "_raw_stream", lambda i: 0)
    monkeypatch.setattr(ops, "_current_device", lambda: -1)
    plan._index, plan._take_list = -1, None
    for e in entries:
        setattr(plan, e, lambda *a: 0)
    return plan


def test_what_a_call_writes_of_its_arguments_counts(monkeypatch):
    z = lambda *k, dtype=F: torch.zeros(k, dtype=dtype)  # noqa: E731
    cpu = lambda plan, *e: _on_the_cpu(monkeypatch, plan, *e)  # noqa: E731
    ver = lambda *ts: [t._version for t in ts]  # noqa: E731

    c = cpu(rn.GradClip([(3,), (4,)], device="cpu"), "_clip")
    g, w, out = [z(3), z(4)], [z(3), z(4)], z(2)
    c.norm(g, out=out)
    assert ver(*g, out) == [0, 0, 1]
    c.clip(g, into=iter(w))
    assert ver(*g, *w) == [0, 0, 1, 1]
    c.clip(iter(g))
    assert ver(*g) == [1, 1]

    o = cpu(rn.AdamW([(3,), (4,)], device="cpu"), "_run")
    p, low = [z(3), z(4)], (z(3, dtype=H), None)
    before = ver(*o.m, *o.v)
    o.step(iter(p), g, 0.1, low=low)
    assert ver(*p, *g, low[0]) == [1, 1, 1, 1, 1]
    assert ver(*o.m, *o.v) == [k + 1 for k in before]

    n = cpu(rn.LayerNorm(1, 2, 3, dtype="f32", device="cpu"), "_fwd", "_bwd")
    x, y, dx, dg, db = z(1, 2, 3), z(1, 2, 3), z(1, 2, 3), z(3), z(3)
    n.fwd(x, y=y)
    n.bwd(x, y, dx=dx, dgamma=dg)
    n.bwd(x, y, dbeta=db)
    assert ver(x, y, dx, dg, db) == [0, 1, 1, 1, 1]
    n = cpu(rn.FrameNorm(1, 2, 4, 2, dtype="f32", device="cpu"), "_fwd", "_bwd")
    x, y, dx, dg, db = z(1, 2, 4), z(1, 2, 4), z(1, 2, 4), z(4), z(4)
    n.fwd(x, y=y)
    n.bwd(x, y, dx=dx, dgamma=dg, dbeta=db)
    assert ver(x, y, dx, dg, db) == [0, 1, 1, 1, 1]
    e = cpu(rn.LabelEmbedding(1, 2, 5, 3, "f32", "f32", device="cpu"), "_fwd", "_bwd")
    ids, table, rows = z(1, 2, dtype=torch.int32), z(5, 3), z(1, 2, 3)
    e.fwd(table, ids, out=rows)
    assert ver(table, rows) == [0, 1]
    e.bwd(rows, ids, dtable=table)
    assert ver(table, rows) == [1, 1]
    m = cpu(rn.Orthogonalizer(3, 4, out_dtype="f32", device="cpu"), "_run")
    G, out = z(3, 4), z(3, 4)
    m.run(G, out=out)
    assert ver(G, out) == [0, 1]


def test_a_graph_that_holds_old_weights_is_refused(monkeypatch):
    o = _on_the_cpu(monkeypatch, rn.AdamW([(3,)], device="cpu"), "_run")
    w, x = torch.ones(3, requires_grad=True), torch.ones(3, requires_grad=True)
    loss = (w * x).sum()
    o.step([w], [torch.ones(3)], 0.1)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        loss.backward()


def test_views_with_the_sign_left_to_do_are_refused(monkeypatch):
    # (the imaginary part of a conjugate is such a view: its memory has the other sign)
    c = _on_the_cpu(monkeypatch, rn.GradClip([(1,)], device="cpu"), "_clip")
    n = _on_the_cpu(monkeypatch, rn.LayerNorm(1, 1, 3, dtype="f32", device="cpu"), "_fwd")
    e = _on_the_cpu(monkeypatch, rn.LabelEmbedding(1, 2, 5, 3, "f32", "f32", device="cpu"), "_fwd")
    neg = torch.ones(1, dtype=torch.complex64).conj().imag
    assert neg.is_neg() and neg.is_contiguous()
    with pytest.raises(ValueError):
        c.norm([neg])
    with pytest.raises(ValueError):
        n.fwd(torch._neg_view(torch.ones(1, 1, 3)))
    with pytest.raises(ValueError):
        e.fwd(torch._neg_view(torch.ones(5, 3)), torch.zeros(1, 2, dtype=torch.int32))
    c.norm([neg.resolve_neg()])


def test_a_plan_of_updates_has_no_workspace():
    assert rn.AdamW([(300, 7)], device="cpu").ws.numel() == 0
    assert rn.GradClip([(300, 7)], device="cpu").ws.numel() > 0
    with pytest.raises(rn.RnntError):
        rn.AdamW([((1 << 36) + 1,)], m=[torch.empty(0)], v=[torch.empty(0)], device="cpu")
