"""What the Python plans of the operators around the loss take and refuse (CPU, nothing launched).

Tensors are stand-ins with a type, a shape, strides and a device; a call that passes the checks
ends in a recorder in place of the library's function.
"""
import ctypes

import pytest
import torch

import asr_tiled_tanh_gb300 as rn
from asr_tiled_tanh_gb300 import build, ops


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build_library()
    rn.load()


class Tensor:
    """A CUDA tensor as far as the checks look at it."""

    def __init__(self, dtype, shape, strides=None, index=0):
        self.dtype, self.shape = dtype, torch.Size(shape)
        self._strides, self._index = strides or torch.empty(shape, device="meta").stride(), index
        self.device, self.is_cuda = torch.device("cuda", index), True

    def dim(self):
        return len(self.shape)

    def get_device(self):
        return self._index

    def stride(self):
        return self._strides

    def data_ptr(self):
        return 1 << 20

    def __getitem__(self, key):
        assert key is None
        return Tensor(self.dtype, (1, *self.shape), (1 << 40, *self._strides), self._index)


def _on(plan, names, monkeypatch, index=0, current=0):
    """The plan as one of GPU `index`, its calls recorded."""
    calls = []
    for name in names:
        setattr(plan, name, lambda *a: calls.append(a) or 0)
    plan._index = index
    monkeypatch.setattr(ops, "_raw_stream", lambda i: 0)
    monkeypatch.setattr(ops, "_current_device", lambda: current, raising=False)
    return calls


F, H, I = torch.float32, torch.bfloat16, torch.int32


# The C side takes a stride of 0 for the dense one: a tensor that is expanded, and so holds less
# than dense rows, must not pass as one of stride 0.
@pytest.mark.parametrize("zero", [(0, 0), (0, 8), (None, 0)])
def test_frames_of_stride_zero_are_refused(zero, monkeypatch):
    B, T, C = 3, 5, 8
    zero = tuple(40 if z is None else z for z in zero)
    n = rn.FrameNorm(B, T, C, 2, x_strides=zero, y_strides=zero, device="cpu")
    calls = _on(n, ("_fwd", "_bwd"), monkeypatch)
    dense, flat = Tensor(H, (B, T, C)), Tensor(H, (B, T, C), (*zero, 1))
    for x, y in ((flat, dense), (dense, flat)):
        with pytest.raises(ValueError):
            n.fwd(x, y=y)
        with pytest.raises(ValueError):
            n.bwd(x, y, dx=dense, dgamma=Tensor(F, (C,)), dbeta=Tensor(F, (C,)))
    assert not calls
    n.fwd(dense, y=dense)
    assert len(calls) == 1


@pytest.mark.parametrize("zero", [(0, 6), (0, 0), (24, 0)])
def test_matrices_of_stride_zero_are_refused(zero, monkeypatch):
    N, R, K = 3, 4, 6
    o = rn.Orthogonalizer(R, K, batch=N, in_strides=zero, out_strides=zero, device="cpu")
    calls = _on(o, ("_run",), monkeypatch)
    for g, out in ((Tensor(F, (N, R, K), (*zero, 1)), Tensor(H, (N, R, K))),
                   (Tensor(F, (N, R, K)), Tensor(H, (N, R, K), (*zero, 1)))):
        with pytest.raises(ValueError):
            o.run(g, out=out)
    assert not calls
    o.run(Tensor(F, (N, R, K)), out=Tensor(H, (N, R, K)))
    assert len(calls) == 1


def _calls(index, monkeypatch, plan_index, current):
    """Every call of every plan, with tensors of GPU `index`: (plan's recorder, call) pairs."""
    e = rn.LabelEmbedding(2, 3, 7, 16, device="cpu")
    n = rn.FrameNorm(2, 5, 16, 4, device="cpu")
    o = rn.Orthogonalizer(4, 6, device="cpu")
    t = lambda dt, *shape: Tensor(dt, shape, None, index)
    ids, ul, c = t(I, 2, 3), t(I, 2), t(F, 16)
    at = dict(index=plan_index, current=current)
    re = _on(e, ("_fwd", "_bwd"), monkeypatch, **at)
    rnorm = _on(n, ("_fwd", "_bwd"), monkeypatch, **at)
    ro = _on(o, ("_run",), monkeypatch, **at)
    x = t(H, 2, 5, 16)
    return [(re, lambda: e.fwd(t(H, 7, 16), ids, ul, out=t(H, 2, 3, 16))),
            (re, lambda: e.bwd(t(H, 2, 3, 16), ids, ul, dtable=t(F, 7, 16))),
            (rnorm, lambda: n.fwd(x, c, c, ul, y=x)),
            (rnorm, lambda: n.bwd(x, x, c, c, ul, dx=x, dgamma=c, dbeta=c)),
            (ro, lambda: o.run(t(F, 4, 6), out=t(H, 4, 6)))]


@pytest.mark.parametrize("plan,tensors,current", [(0, 1, 0), (1, 0, 1), (1, 1, 0), (0, 0, 1),
                                                  (None, 0, 0)])
def test_another_gpu_is_refused(plan, tensors, current, monkeypatch):
    for record, call in _calls(tensors, monkeypatch, plan, current):
        with pytest.raises(ValueError):
            call()
        assert not record


@pytest.mark.parametrize("index", [0, 1])
def test_the_plans_own_gpu_is_taken(index, monkeypatch):
    for record, call in _calls(index, monkeypatch, index, index):
        call()
        assert len(record) == 1
        record.clear()


def test_a_given_stream_does_not_lift_the_check(monkeypatch):
    o = rn.Orthogonalizer(4, 6, device="cpu")
    calls = _on(o, ("_run",), monkeypatch, index=1, current=0)
    g, out = Tensor(F, (4, 6), None, 1), Tensor(H, (4, 6), None, 1)
    with pytest.raises(ValueError):
        o.run(g, out=out, stream=77)
    assert not calls


# Sizes at a limit: the largest is planned, the next is refused before anything is worked out of
# it (a frame of 2^30 floats divided by zero).
@pytest.mark.parametrize("C,dtype", [((1 << 28) + 1, 1), (1 << 29, 1), (1 << 30, 0), (1 << 30, 1)])
def test_frames_past_the_width_limit(C, dtype):
    lib, d = rn.load(), lambda c: ctypes.byref(ops.RnntNormDims(B=1, T=1, C=c, G=1, act=1,
                                                                dtype=dtype, eps=1e-5))
    assert lib.rnnt_norm_workspace_bytes(d(1 << 28)) > 0
    assert lib.rnnt_norm_workspace_bytes(d(C)) == lib.rnnt_norm_saved_bytes(d(C)) == 0
    assert lib.rnnt_norm_fwd(d(C), *[4096] * 7, 1 << 50, None, None) == 1
    assert lib.rnnt_norm_bwd(d(C), *[4096] * 10, 1 << 50, None, None) == 1


# 65,535 blocks of 32 columns are the most that one launch of the sums takes.
@pytest.mark.parametrize("D", [(1 << 20) + 1, 3_000_001, (1 << 31) - 1])
def test_rows_past_the_width_limit(D):
    lib, d = rn.load(), lambda n: ctypes.byref(ops.RnntEmbedDims(B=1, U1=1, V=2, D=n, table_dtype=0,
                                                                 row_dtype=0, scale=1.0))
    assert lib.rnnt_embed_workspace_bytes(d(1 << 20)) > 0
    assert lib.rnnt_embed_workspace_bytes(d(D)) == 0
    assert lib.rnnt_embed_fwd(d(D), *[4096] * 4, None, None) == 1
    assert lib.rnnt_embed_bwd(d(D), *[4096] * 5, 1 << 50, None, None) == 1


# A size past 32 bits would reach the C side as another one, and plan and tensors differ.
@pytest.mark.parametrize("make", [
    lambda: rn.LabelEmbedding((1 << 32) + 2, 3, 7, 16, device="cpu"),
    lambda: rn.LabelEmbedding(2, 3, (1 << 32) + 7, 16, device="cpu"),
    lambda: rn.FrameNorm(2, (1 << 32) + 5, 16, 4, device="cpu"),
    lambda: rn.FrameNorm(2, 5, (1 << 33) + 16, 4, device="cpu"),
    lambda: rn.FrameNorm(2, 5, 16, 4, x_strides=((1 << 64) + 80, 16), device="cpu"),
    lambda: rn.Orthogonalizer(4, (1 << 32) + 6, device="cpu"),
    lambda: rn.Orthogonalizer(4, 6, steps=(1 << 32) + 5, device="cpu")])
def test_sizes_past_the_fields_are_refused(make):
    with pytest.raises(ValueError):
        make()


def test_whole_numbers_for_real_fields():
    assert rn.LabelEmbedding(2, 3, 7, 16, scale=(1 << 24) + 1, device="cpu").dims.scale == 1 << 24
    assert rn.Orthogonalizer(4, 6, eps=0, device="cpu").dims.eps == 0
