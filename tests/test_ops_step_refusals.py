"""What the layer norm, the clipping and the AdamW update refuse on the host (CPU).

Addresses are fake and never dereferenced.
"""
import ctypes

import pytest
import torch

import asr_tiled_tanh_gb300 as rn
from asr_tiled_tanh_gb300 import build
from asr_tiled_tanh_gb300.ops import RnntAdamwOpts, RnntGradList, RnntLnDims

INVALID, WS = 1, 3
LN = dict(B=2, T=5, C=16, label_rows=0, x_dtype=1, y_dtype=1, eps=1e-5, x_frame=0, x_batch=0,
          y_frame=0, y_batch=0)


@pytest.fixture(scope="module")
def lib():
    build.build_library()
    return rn.load()


@pytest.mark.parametrize("bad", [
    dict(B=-1), dict(T=0), dict(C=0), dict(x_dtype=2), dict(y_dtype=-1), dict(eps=-1.0),
    dict(eps=float("nan")), dict(C=(1 << 20) + 1), dict(B=1 << 20, T=1 << 11), dict(x_frame=15),
    dict(y_frame=-16), dict(x_batch=79), dict(x_frame=16, x_batch=16), dict(y_batch=-80),
    dict(x_frame=31, x_batch=16), dict(x_frame=1 << 62), dict(x_batch=1 << 62),
    dict(y_frame=(1 << 47) // 5 + 1), dict(y_batch=1 << 47)])
def test_ln_dims(lib, bad):
    d = ctypes.byref(RnntLnDims(**{**LN, **bad}))
    assert lib.rnnt_ln_workspace_bytes(d) == lib.rnnt_ln_saved_bytes(d) == 0
    assert lib.rnnt_ln_fwd(d, *[4096] * 6, None, None) == INVALID
    assert lib.rnnt_ln_bwd(d, *[4096] * 9, 1 << 50, None, None) == INVALID


@pytest.mark.parametrize("good", [dict(x_frame=32, x_batch=16), dict(y_frame=40, y_batch=20),
                                  dict(B=1, x_batch=1), dict(T=1, x_frame=1, x_batch=16), dict(B=0),
                                  dict(C=1 << 20), dict(B=1 << 10, T=1 << 20)])
def test_ln_dims_that_are_fine(lib, good):
    d = ctypes.byref(RnntLnDims(**{**LN, **good}))
    assert lib.rnnt_ln_workspace_bytes(d) > 0 and lib.rnnt_ln_saved_bytes(d) > 0


def _each(call, base, required, misaligned):
    for n in required:
        assert call({**base, n: None}) == INVALID, n
    for n, by in misaligned.items():
        assert call({**base, n: base[n] + by}) == INVALID, n


def test_ln_pointers(lib):
    d = RnntLnDims(**LN)
    names = ("x", "gamma", "beta", "lengths", "y", "saved", "status")
    base = {n: 0x10000 * (i + 1) for i, n in enumerate(names)}
    _each(lambda a: lib.rnnt_ln_fwd(ctypes.byref(d), *[a[n] for n in names], None), base,
          ("x", "y"), dict(x=1, gamma=2, beta=1, lengths=2, y=1, saved=128, status=2))
    names = ("x", "dy", "gamma", "lengths", "saved", "dx", "dgamma", "dbeta", "ws")
    base = {n: 0x10000 * (i + 1) for i, n in enumerate(names)}
    need = lib.rnnt_ln_workspace_bytes(ctypes.byref(d))
    bwd = lambda a, ws=need, st=None: lib.rnnt_ln_bwd(  # noqa: E731
        ctypes.byref(d), *[a[n] for n in names], ws, st, None)
    _each(bwd, base, ("x", "dy", "saved", "dx", "ws"),
          dict(x=1, dy=1, gamma=2, lengths=1, saved=64, dx=1, dgamma=2, dbeta=2, ws=128))
    assert bwd(base, need - 1) == WS and bwd(base, need, 0x10002) == INVALID


def _list(counts, dtypes=None):
    n = len(counts)
    return RnntGradList(n, (ctypes.c_longlong * n)(*counts),
                        (ctypes.c_int * n)(*dtypes) if dtypes else None)


def _ptrs(*p):
    return (ctypes.c_void_p * len(p))(*p)


BAD_LISTS = [RnntGradList(-1, None, None), RnntGradList((1 << 16) + 1, None, None),
             RnntGradList(1, None, None), _list([-1]), _list([(1 << 36) + 1]), _list([4], [2])]


@pytest.mark.parametrize("i", range(len(BAD_LISTS)))
def test_lists(lib, i):
    l = ctypes.byref(BAD_LISTS[i])
    assert lib.rnnt_clip_workspace_bytes(l) == 0
    p, o = _ptrs(4096), RnntAdamwOpts(0.9, 0.999, 1e-8, 0.1, 0.0, None)
    assert lib.rnnt_clip(l, p, None, 1.0, 1e-6, 4096, 4096, 1 << 30, None) == INVALID
    assert lib.rnnt_adamw(l, ctypes.byref(o), p, p, p, p, None, None, None, 4096, None) == INVALID
    assert lib.rnnt_clip_workspace_bytes(None) == 0


def test_clip_arguments(lib):
    l = _list([100, 0, 8], [0, 1, 1])
    need = lib.rnnt_clip_workspace_bytes(ctypes.byref(l))
    g = _ptrs(0x1000, None, 0x2000)

    def call(grads=g, into=None, most=1.0, eps=1e-6, clip=4096, ws=4096, n=need):
        return lib.rnnt_clip(ctypes.byref(l), grads, into, most, eps, clip, ws, n, None)

    inf, nan = float("inf"), float("nan")
    for bad in (dict(grads=None), dict(clip=None), dict(ws=None), dict(clip=4098), dict(ws=4224),
                dict(most=-1.0), dict(most=nan), dict(eps=-1.0), dict(eps=nan), dict(eps=inf),
                dict(most=0.0, eps=0.0), dict(grads=_ptrs(None, None, 0x2000)),
                dict(grads=_ptrs(0x1002, None, 0x2000)), dict(grads=_ptrs(0x1000, None, 0x2001)),
                dict(into=_ptrs(0x1000, None, None)), dict(into=_ptrs(0x3002, None, 0x4000)),
                dict(into=_ptrs(0x1004, None, 0x2000)), dict(into=_ptrs(0x2008, None, 0x2000)),
                dict(into=_ptrs(0x2000, None, 0x1000))):
        assert call(**bad) == INVALID, bad
    assert call(n=need - 1) == WS


def test_adamw_arguments(lib):
    l = _list([100, 0, 8], [0, 1, 1])
    at = lambda k: _ptrs(k * 0x10000, None, k * 0x10000 + 0x1000)  # noqa: E731
    base = dict(params=at(1), grads=at(2), m=at(3), v=at(4), low=at(5), lr=None, clip=None,
                steps=4096)

    def call(opts=None, **k):
        a = {**base, **k}
        o = RnntAdamwOpts(*{**dict(b1=0.9, b2=0.999, eps=1e-8, lr=0.1, decay=0.0, decays=None),
                            **(opts or {})}.values())
        return lib.rnnt_adamw(ctypes.byref(l), ctypes.byref(o), *a.values(), None)

    inf, nan = float("inf"), float("nan")
    for bad in (dict(b1=1.0), dict(b1=-0.1), dict(b2=nan), dict(b2=1.0), dict(eps=-1.0),
                dict(eps=nan), dict(lr=nan), dict(lr=inf), dict(decay=nan), dict(decay=inf),
                dict(decays=(ctypes.c_float * 3)(0.1, nan, 0.1))):
        assert call(bad) == INVALID, bad
    for n in ("params", "grads", "m", "v", "steps"):
        assert call(**{n: None}) == INVALID, n
    for n in ("params", "m", "v"):
        assert call(**{n: _ptrs(0x70002, None, 0x80000)}) == INVALID, n
        assert call(**{n: _ptrs(0x70000, None, None)}) == INVALID, n
    assert call(grads=_ptrs(0x70000, None, 0x80001)) == INVALID
    assert call(low=_ptrs(0x70001, None, None)) == INVALID
    for n, off in (("lr", 2), ("clip", 1), ("steps", 2)):
        assert call(**{n: 4096 + off}) == INVALID, n
    # memory that is written and met again
    for n, p in (("m", _ptrs(0x10000, None, 0x90000)), ("v", _ptrs(0x10000 + 396, None, 0x90000)),
                 ("grads", _ptrs(0x10000, None, 0x90000)), ("low", _ptrs(0x40000, None, 0x90000)),
                 ("low", _ptrs(0x40000 - 198, None, 0x90000)),
                 ("params", _ptrs(0x90000, None, 0x90000 + 396)),
                 ("params", _ptrs(0x90000, None, 0x90000 - 28)),
                 ("grads", _ptrs(0x90000, None, 0x30000 + 396))):
        assert call(**{n: p}) == INVALID, (n, list(p))


def test_names_and_numbers(lib):
    for make in (lambda: rn.LayerNorm(1, 1, 1, dtype="f16", device="cpu"),
                 lambda: rn.LayerNorm(1, 1, 1, out_dtype="e4m3", device="cpu"),
                 lambda: rn.LayerNorm((1 << 32) + 2, 1, 16, device="cpu"),
                 lambda: rn.GradClip([(3,)], dtype="f64", device="cpu"),
                 lambda: rn.GradClip([(3,)], dtype=["f32", "f32"], device="cpu"),
                 lambda: rn.GradClip([(3,)], max_norm=-1, device="cpu"),
                 lambda: rn.GradClip([(3,)], max_norm=float("nan"), device="cpu"),
                 lambda: rn.GradClip([(3,)], max_norm=0, eps=0, device="cpu"),
                 lambda: rn.GradClip([(3,)], eps=float("inf"), device="cpu"),
                 lambda: rn.AdamW([(3,)], weight_decay=[0.1, 0.2], device="cpu"),
                 lambda: rn.AdamW([(3,)], grad_dtype=["f32", "bf16"], device="cpu"),
                 lambda: rn.AdamW([(3,)], betas=(1.0, 0.9), device="cpu"),
                 lambda: rn.AdamW([(3,)], eps=-1.0, device="cpu"),
                 lambda: rn.AdamW([(3,)], steps=-1, device="cpu")):
        with pytest.raises(ValueError):
            make()
    with pytest.raises(rn.RnntError):
        rn.LayerNorm(1, 0, 16, device="cpu")
    with pytest.raises(rn.RnntError):
        rn.GradClip([((1 << 36) + 1,)], device="cpu")


@pytest.mark.parametrize("seed", range(60))
def test_overlap_against_every_pair(lib, seed):
    import random
    r = random.Random(seed)
    spans, at = [], 4096
    for _ in range(r.choice([0, 1, 2, 5])):  # lists that lie one after another, or anywhere
        one = []
        for _ in range(r.randint(0, 12)):
            one.append((at, r.choice([0, 4, 64, 100]), r.random() < 0.6))
            at += r.choice([64, 100, 128])
        spans += r.choice([one, one[::-1], r.sample(one, len(one))])
    if seed % 2 and spans:  # one more that may meet others
        spans.insert(r.randint(0, len(spans)), (r.choice(spans)[0] + r.choice([-40, 0, 3, 63]),
                                                r.choice([1, 41, 5000]), r.random() < 0.5))
    if seed % 3 == 0:
        spans = sorted(spans, key=lambda s: s[0] % 1000)
    n = len(spans)
    expect = any(a[1] and b[1] and (a[2] or b[2]) and a[0] < b[0] + b[1] and b[0] < a[0] + a[1]
                 for i, a in enumerate(spans) for b in spans[:i])
    got = lib.rnnt_testing_overlap(n, _ptrs(*[s[0] for s in spans]),
                                   (ctypes.c_size_t * n)(*[s[1] for s in spans]),
                                   (ctypes.c_int * n)(*[int(s[2]) for s in spans]))
    assert got == int(expect)


class Tensor:
    """A CUDA tensor as far as the checks look at it."""

    def __init__(self, dtype, shape, dense=True, index=0, at=1 << 20):
        self.dtype, self.shape, self._dense, self._index = dtype, torch.Size(shape), dense, index
        self.device, self._at = torch.device("cuda", index), at

    def get_device(self):
        return self._index

    def is_contiguous(self):
        return self._dense

    def stride(self):
        return torch.empty(self.shape, device="meta").stride()

    def reshape(self, *shape):
        return self

    def data_ptr(self):
        return self._at


F, H = torch.float32, torch.bfloat16


def _plans(monkeypatch, current=0):
    from asr_tiled_tanh_gb300 import ops
    shapes = [(4, 6), (7,)]
    c = rn.GradClip(shapes, dtype=["f32", "bf16"], device="cpu")
    t = lambda dt: [Tensor(dt, k, at=(1 << 20) * (i + 1))  # noqa: E731
                    for i, k in enumerate(shapes)]
    o = rn.AdamW(shapes, grad_dtype=["f32", "bf16"], m=t(F), v=t(F), device="cpu")
    calls = []
    for plan, name in ((c, "_clip"), (o, "_run")):
        plan._index = 0
        setattr(plan, name, lambda *a: calls.append(a) or 0)
    monkeypatch.setattr(ops, "_raw_stream", lambda i: 0)
    monkeypatch.setattr(ops, "_current_device", lambda: current)
    for plan in (c, o):  # (the helper of lists takes no stand-ins)
        plan._take_list = None
    return c, o, calls


def test_tensors_of_another_type_layout_or_gpu_are_refused(monkeypatch):
    c, o, calls = _plans(monkeypatch)
    g = [Tensor(F, (4, 6)), Tensor(H, (7,))]
    p = [Tensor(F, (4, 6)), Tensor(F, (7,))]
    low = [Tensor(H, (4, 6)), Tensor(H, (7,))]
    out = Tensor(F, (2,))
    wrong = [[g[0]], [g[0], g[1], g[1]], [g[1], g[0]], [Tensor(F, (6, 4)), g[1]],
             [Tensor(F, (24,)), g[1]], [Tensor(F, (4, 6), dense=False), g[1]],
             [Tensor(F, (4, 6), index=1), g[1]], [Tensor(H, (4, 6)), g[1]]]
    for w in wrong:
        with pytest.raises(ValueError):
            c.norm(w, out=out)
        with pytest.raises(ValueError):
            c.clip(g, into=w, out=out)
        with pytest.raises(ValueError):
            o.step(p, w, 0.1)
        with pytest.raises(ValueError):
            o.step(w, g, 0.1)
        if w is not wrong[-1]:
            with pytest.raises(ValueError):
                o.step(p, g, 0.1, low=w)
    for bad in (dict(clip=Tensor(F, (1,))), dict(clip=Tensor(H, (2,))),
                dict(low=[None]), dict(low=[None, Tensor(F, (7,))])):
        with pytest.raises(ValueError):
            o.step(p, g, 0.1, **bad)
    with pytest.raises(ValueError):
        c.norm(g, out=Tensor(F, (3,)))
    assert not calls
    c.norm(g, out=out)
    c.clip(g, into=g, out=out)
    o.step(p, g, 0.1, low=low, clip=out)
    o.step(p, g, 0.1, low=[None, low[1]])
    assert len(calls) == 4


def test_another_current_gpu_is_refused(monkeypatch):
    c, o, calls = _plans(monkeypatch, current=1)
    g, p = [Tensor(F, (4, 6)), Tensor(H, (7,))], [Tensor(F, (4, 6)), Tensor(F, (7,))]
    with pytest.raises(ValueError):
        c.norm(g, out=Tensor(F, (2,)))
    with pytest.raises(ValueError):
        o.step(p, g, 0.1)
    assert not calls


def test_lists_are_refused_by_the_helper_too():
    c = rn.GradClip([(2, 3), (4,)], dtype=["f32", "bf16"], device="cpu")
    a, b = torch.zeros(2, 3), torch.zeros(4, dtype=torch.bfloat16)
    assert c._take_list is not None  # it was built
    c._index = 0
    for g in ([a, b], [a], [a, b, b], [b, a], [a, None], (a, b), [1, 2]):
        with pytest.raises((ValueError, AttributeError)):  # (no CUDA tensors, at best)
            c.norm(g, out=torch.zeros(2))
