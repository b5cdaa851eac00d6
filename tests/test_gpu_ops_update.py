"""Gradient clipping and the AdamW update against a plain implementation in 64 bits (GPU).

Tolerances.  u = 2^-24 is half a step of fp32, 2^-8 of bf16.  Squares are added in fp32 in groups
of at most 32 (each within 33 u of its sum, all terms positive) and then in fp64, so the norm is
17 u off and half a step more; the scale is its quotient, rounded once: 20 u and 22 u.  A moment is
two products and a sum of rounded factors: 5 u of the terms' sizes, 3 u more for a scaled gradient
(its square: 6 u).  1 - beta^t comes from an exponent that is 3 u off and stays within 8 u; the
step divides two such values by a root: 32 u of its size.  A weight adds half a step of its own.
"""
import numpy as np
import pytest
import torch

import asr_tiled_tanh_gb300 as rn

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
DT = {"f32": torch.float32, "bf16": torch.bfloat16}


@pytest.fixture(scope="module", autouse=True)
def _lib():
    rn.load(build_if_missing=True)


# (lists of one launch for everything, of several, of more tensors than a launch's tables hold)
LISTS = [[(1,)], [(3,), (), (0,), (5, 7)], [(64, 64), (64,), (32, 64), (33,)],
         [(2048,), (2049,), (2047,), (4096, 3)], [(513, 1025)], [(17,)] * 70,
         [(1000 + 37 * i,) for i in range(140)], [(1 << 21,), (7,), (1 << 20, 3)],
         [(1 + i % 37,) for i in range(530)], [(8192 * 31 - 5,)], [(8192 * 33,)]]


def _dtypes(shapes, kind):
    return [("f32", "bf16")[i % 2] if kind == "mixed" else kind for i in range(len(shapes))]


def _grads(shapes, dtypes, seed=0, size=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return [(size * torch.randn(k, device="cuda", generator=g)).to(DT[d])
            for k, d in zip(shapes, dtypes)]


def _norm64(ts):
    return np.sqrt(sum(float((t.double() ** 2).sum()) for t in ts))


def _check_clip(clip, grads, max_norm, eps):
    norm = _norm64(grads)
    scale = min(1.0, max_norm / (norm + eps))
    got = clip.double().cpu().numpy()
    assert abs(got[0] - norm) <= 20 * U * norm + 1e-45
    assert abs(got[1] - scale) <= 22 * U * scale
    return float(got[1])


def _check_scaled(into, grads, scale):
    for w, g in zip(into, grads):
        half = U if g.dtype is torch.float32 else 2.0 ** -8
        ref = g.double() * scale
        assert w.dtype is g.dtype
        assert torch.all((w.double() - ref).abs() <= half * ref.abs() + 1e-40)


@pytest.mark.parametrize("shapes", LISTS, ids=range(len(LISTS)))
@pytest.mark.parametrize("kind", ["f32", "bf16", "mixed"])
def test_norm_and_clip(shapes, kind):
    dtypes = _dtypes(shapes, kind)
    grads = _grads(shapes, dtypes, seed=len(shapes))
    keep = [g.clone() for g in grads]
    c = rn.GradClip(shapes, max_norm=0.5, dtype=dtypes)
    scale = _check_clip(c.norm(grads), grads, 0.5, 1e-6)
    assert all(torch.equal(a, b) for a, b in zip(grads, keep))
    into = [torch.full_like(g, float("nan")) for g in grads]
    _check_clip(c.clip(grads, into=into), keep, 0.5, 1e-6)
    assert all(torch.equal(a, b) for a, b in zip(grads, keep))
    _check_scaled(into, keep, scale)
    c.clip(grads)
    assert all(torch.equal(a, b) for a, b in zip(grads, into))


@pytest.mark.parametrize("sizes", [(300, 41, 5000), (200000, 33, 90001)])
def test_some_in_place_some_elsewhere(sizes):
    shapes = [(k,) for k in sizes]
    grads = tuple(_grads(shapes, ["f32", "bf16", "f32"], seed=4))
    keep = [g.clone() for g in grads]
    into = [grads[0], torch.zeros_like(grads[1]), grads[2]]
    c = rn.GradClip(shapes, max_norm=0.5, dtype=["f32", "bf16", "f32"])
    out = torch.zeros(2, device="cuda")
    assert c.clip(grads, into=into, out=out) is out
    _check_scaled(into, keep, _check_clip(out, keep, 0.5, 1e-6))
    assert torch.equal(grads[1], keep[1])


def test_a_norm_below_the_limit_leaves_the_gradients():
    shapes = [(100, 33), (5,)]
    grads = _grads(shapes, ["f32"] * 2)
    keep = [g.clone() for g in grads]
    c = rn.GradClip(shapes, max_norm=1e4)
    out = c.clip(grads)
    assert float(out[1]) == 1.0
    into = [torch.empty_like(g) for g in grads]
    c.clip(grads, into=into)
    assert all(torch.equal(a, b) and torch.equal(a, k) for a, b, k in zip(grads, into, keep))


@pytest.mark.parametrize("size", [1e-42, 1e-30, 1e-19, 3e-12, 1e18, 1e25, 3e36])
@pytest.mark.parametrize("kind", ["f32", "bf16"])
def test_entries_of_any_size(size, kind):
    shapes = [(40, 50), (3,), (2000,)]
    grads = _grads(shapes, [kind] * 3, seed=5, size=size)
    grads[2].zero_()
    out = rn.GradClip(shapes, max_norm=1.0, dtype=kind, eps=0.0).norm(grads)
    norm = _norm64(grads)
    assert abs(float(out[0]) - norm) <= 20 * U * norm + 2.0 ** -149
    scale = min(1.0, 1 / norm)
    assert abs(float(out[1]) - scale) <= 22 * U * scale + 2.0 ** -149


def test_small_entries_beside_large_ones():
    # 2^24 entries of 2^-13 beside one of 1: their squares add up to a quarter of its own
    g = torch.full((1 << 24,), 2.0 ** -13, device="cuda")
    g[12345] = 1.0
    out = rn.GradClip([(1 << 24,)]).norm([g])
    norm = _norm64([g])
    assert abs(float(out[0]) - norm) <= 20 * U * norm


def test_no_elements_and_zeros():
    for shapes in ([], [(0,), (4, 0)], [(0,)] * 600, [(2, 0)] * 600 + [(0, 3)]):
        c = rn.GradClip(shapes, max_norm=2.0)
        assert c.clip([torch.empty(k, device="cuda") for k in shapes]).tolist() == [0.0, 1.0]
    shapes = [(0,)] * 600 + [(7,)]  # one tensor with elements behind many without
    grads = [torch.full(k, 2.0, device="cuda") for k in shapes]
    c = rn.GradClip(shapes, max_norm=1.0)
    _check_clip(c.clip(grads), [torch.full((7,), 2.0, device="cuda")], 1.0, 1e-6)
    o = rn.AdamW(shapes)
    o.step([torch.zeros(k, device="cuda") for k in shapes], grads, 0.1)
    assert o.steps.tolist() == [1, 0]
    o = rn.AdamW([(0,)] * 600)
    o.step(grads[:600], grads[:600], 0.1)
    assert o.steps.tolist() == [0, 0]  # nothing to update
    z = [torch.zeros(100, 30, device="cuda")]
    assert rn.GradClip([(100, 30)], max_norm=2.0).clip(z).tolist() == [0.0, 1.0]


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("kind", ["f32", "bf16"])
def test_norms_that_are_not_finite(bad, kind):
    shapes = [(300,), (70, 70)]
    grads = _grads(shapes, [kind] * 2)
    grads[1][3, 4] = bad
    into = [torch.zeros_like(g) for g in grads]
    out = rn.GradClip(shapes, dtype=kind).clip(grads, into=into)
    if np.isnan(bad):
        assert torch.isnan(out).all() and all(torch.isnan(w).all() for w in into)
    else:
        assert out.tolist() == [float("inf"), 0.0]
        assert torch.isnan(into[1][3, 4]) and int(torch.count_nonzero(into[1])) == 1
        assert not into[0].any()


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("shift", [1, 2, 3])
def test_tensors_off_16_bytes(kind, shift):
    n = [5000, 17, 4096]
    bufs = [torch.full((k + 16,), 9.0, dtype=DT[kind], device="cuda") for k in n]
    outs = [torch.full((k + 16,), 9.0, dtype=DT[kind], device="cuda") for k in n]
    grads = [b[shift:shift + k] for b, k in zip(bufs, n)]
    for g, r in zip(grads, _grads([(k,) for k in n], [kind] * 3, seed=shift)):
        g.copy_(r)
    into = [b[k2:k2 + k] for b, k, k2 in zip(outs, n, (shift, 0, 5))]
    c = rn.GradClip([(k,) for k in n], dtype=kind)
    scale = _check_clip(c.clip(grads, into=into), grads, 1.0, 1e-6)
    _check_scaled(into, grads, scale)
    for v, b in zip(into, outs):
        v.fill_(9.0)
        assert torch.all(b == 9.0)


@pytest.mark.parametrize("times", [1, 9])  # one launch, and two
@pytest.mark.parametrize("kind", ["f32", "bf16"])
def test_views_of_one_buffer_without_gaps(kind, times):
    # tensors that begin anywhere, alike in both lists
    n = [1, 5001, 3, 8191, 8192, 2, 20001] * times
    flat, out = (torch.zeros(sum(n) + 9, dtype=DT[kind], device="cuda") for _ in range(2))
    flat.copy_(_grads([(sum(n) + 9,)], [kind], seed=3)[0])
    at = np.cumsum([0, *n])
    norms = []
    for move in (0, 1):
        grads = [flat[a:a + k] for a, k in zip(at, n)]
        into = [out[a + move:a + move + k] for a, k in zip(at, n)]
        out.fill_(9.0)
        c = rn.GradClip([(k,) for k in n], dtype=kind)
        norms += [c.norm(grads), c.clip(grads, into=into)]
        scale = _check_clip(norms[-1], grads, 1.0, 1e-6)
        _check_scaled(into, grads, scale)
        assert torch.all(out[:move] == 9.0) and torch.all(out[sum(n) + move:] == 9.0)
    assert all(torch.equal(a, norms[0]) for a in norms)  # wherever the products go


# ---- AdamW

OPT = dict(betas=(0.9, 0.999), eps=1e-8)


def _f32(x):
    return float(np.float32(x))


def _adam64(p, m, v, g, t, lr, decay, scale=1.0, betas=(0.9, 0.999), eps=1e-8):
    """One update in 64 bits, and the bounds of its three results."""
    lr, decay, eps = _f32(lr), _f32(decay), _f32(eps)
    b1, b2 = betas
    g = g.double() * scale
    m1 = b1 * m.double() + (1 - b1) * g
    v1 = b2 * v.double() + (1 - b2) * g * g
    mb = 8 * U * (b1 * m.double().abs() + (1 - b1) * g.abs())
    vb = 12 * U * v1
    step = m1 / (1 - b1 ** t) / ((v1 / (1 - b2 ** t)).sqrt() + eps)
    wide = (mb / (1 - b1 ** t)) / ((v1 / (1 - b2 ** t)).sqrt() + eps)
    p1 = p.double() - lr * (decay * p.double() + step)
    pb = U * p1.abs() + lr * (wide + 32 * U * step.abs() + 4 * U * decay * p.double().abs())
    return (p1, m1, v1), (pb, mb, vb)


def _within(got, ref, bound, what):
    for i, (a, r, b) in enumerate(zip(got, ref, bound)):
        err = (a.double() - r).abs()
        assert torch.all(err <= b + 1e-37), (what, i, float((err - b).max()))


def _state(shapes, seed=0, zero=False):
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda k: torch.randn(k, device="cuda", generator=g)  # noqa: E731
    p = [r(k) for k in shapes]
    m = [0.1 * r(k) * (not zero) for k in shapes]
    v = [0.01 * r(k) ** 2 * (not zero) for k in shapes]
    return p, m, v


@pytest.mark.parametrize("shapes", LISTS, ids=range(len(LISTS)))
@pytest.mark.parametrize("kind", ["f32", "bf16", "mixed"])
def test_adamw(shapes, kind):
    dtypes = _dtypes(shapes, kind)
    p, m, v = _state(shapes, seed=1)
    decays = [0.1 * (i % 3) for i in range(len(shapes))]
    o = rn.AdamW(shapes, grad_dtype=dtypes, weight_decay=decays, m=[t.clone() for t in m],
                 v=[t.clone() for t in v], steps=3, **OPT)
    q = [t.clone() for t in p]
    low = [None if i % 4 == 3 else torch.zeros(k, dtype=torch.bfloat16, device="cuda")
           for i, k in enumerate(shapes)]
    for t in (4, 5):
        grads = _grads(shapes, dtypes, seed=t, size=0.3)
        keep = [[x.clone() for x in s] for s in (q, o.m, o.v, grads)]
        o.step(q, grads, 1e-2, low=low)
        assert all(torch.equal(a, b) for a, b in zip(grads, keep[3]))
        for i in range(len(shapes)):
            ref, bound = _adam64(*[s[i] for s in keep], t, 1e-2, decays[i])
            _within((q[i], o.m[i], o.v[i]), ref, bound, (t, i))
            assert low[i] is None or torch.equal(low[i], q[i].bfloat16())
    assert o.steps.tolist() == [5, 0]


@pytest.mark.parametrize("t", [1, 2, 10, 1000, 100000, 10 ** 8])
@pytest.mark.parametrize("betas", [(0.9, 0.999), (0.95, 0.99999), (0.0, 0.0), (0.0, 0.99)])
def test_bias_corrections(t, betas):
    shapes = [(300,)]
    p, m, v = _state(shapes, seed=t % 97, zero=t == 1)
    grads = _grads(shapes, ["f32"])
    ref, bound = _adam64(p[0], m[0], v[0], grads[0], t, 0.125, 0.0, betas=betas)
    o = rn.AdamW(shapes, betas=betas, weight_decay=0.0, m=m, v=v, steps=t - 1)
    o.step(p, grads, 0.125)
    _within((p[0], m[0], v[0]), ref, bound, t)
    assert o.steps.tolist() == [t, 0]


def test_adamw_takes_the_clips_scale_and_a_device_learning_rate():
    shapes = [(50, 40), (77,)]
    p, m, v = _state(shapes, seed=8)
    grads = _grads(shapes, ["f32"] * 2, size=5.0)
    c = rn.GradClip(shapes, max_norm=1.0)
    clip = c.norm(grads)
    keep = [[x.clone() for x in s] for s in (p, m, v, grads)]
    o = rn.AdamW(shapes, m=m, v=v, steps=20)
    o.step(p, grads, torch.tensor(0.03, device="cuda"), clip=clip)
    for i in range(2):
        ref, bound = _adam64(*[s[i] for s in keep], 21, 0.03, 0.01, scale=float(clip[1]))
        _within((p[i], m[i], v[i]), ref, bound, i)


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_an_update_without_a_finite_norm_is_left_out(bad):
    shapes = [(17,)] * 70 + [(5000,)]
    p, m, v = _state(shapes, seed=8)
    grads = _grads(shapes, ["f32"] * 71)
    grads[70][123] = bad
    low = [torch.full(k, 3.0, dtype=torch.bfloat16, device="cuda") for k in shapes]
    keep = [[x.clone() for x in s] for s in (p, m, v, low)]
    c, o = rn.GradClip(shapes), rn.AdamW(shapes, m=m, v=v, steps=6)
    o.step(p, grads, 0.1, clip=c.norm(grads), low=low)
    assert all(torch.equal(a, b) for s, k in zip((p, m, v, low), keep) for a, b in zip(s, k))
    assert o.steps.tolist() == [6, 0]
    grads[70][123] = 1.0
    o.step(p, grads, 0.1, clip=c.norm(grads), low=low)
    assert o.steps.tolist() == [7, 0] and not torch.equal(p[3], keep[0][3])


@pytest.mark.parametrize("shift", [1, 2, 3])
@pytest.mark.parametrize("which", ["p", "m", "v", "g", "low", "all"])
def test_adamw_off_16_bytes(shift, which):
    shapes = [(4100,), (9,)]

    def place(name, dtype, values):
        out = []
        for x in values:
            at = shift if which in (name, "all") else 0
            buf = torch.full((x.numel() + 16,), 9.0, dtype=dtype, device="cuda")
            buf[at:at + x.numel()] = x
            bufs.append((buf, at, x.numel(), name))
            out.append(buf[at:at + x.numel()])
        return out

    bufs = []
    p, m, v = _state(shapes, seed=shift)
    g = _grads(shapes, ["bf16"] * 2, seed=shift)
    low = [torch.zeros(k, dtype=torch.bfloat16, device="cuda") for k in shapes]
    P, M, V = (place(k, torch.float32, x) for k, x in (("p", p), ("m", m), ("v", v)))
    G, L = place("g", torch.bfloat16, g), place("low", torch.bfloat16, low)
    o = rn.AdamW(shapes, grad_dtype="bf16", m=M, v=V)
    o.step(P, G, 0.01, low=L)
    for i in range(2):
        ref, bound = _adam64(p[i], m[i], v[i], g[i], 1, 0.01, 0.01)
        _within((P[i], M[i], V[i]), ref, bound, i)
        assert torch.equal(L[i], P[i].bfloat16())
    for buf, at, k, name in bufs:
        assert torch.all(buf[:at] == 9.0) and torch.all(buf[at + k:] == 9.0), name


def test_adamw_on_views_of_buffers_without_gaps():
    n = [1, 5001, 3, 8191, 8192, 2, 20001]
    total, at = sum(n), np.cumsum([0, *n])
    cut = lambda t: [t[a:a + k] for a, k in zip(at, n)]  # noqa: E731
    (p,), (m,), (v,) = _state([(total + 5,)], seed=2)
    g = _grads([(total + 5,)], ["bf16"], seed=9)[0]
    low = torch.full((total + 5,), 9.0, dtype=torch.bfloat16, device="cuda")
    keep = [x.clone() for x in (p, m, v, g)]
    o = rn.AdamW([(k,) for k in n], grad_dtype="bf16", m=cut(m), v=cut(v))
    o.step(cut(p), cut(g), 0.01, low=cut(low))
    ref, bound = _adam64(*[x[:total] for x in keep], 1, 0.01, 0.01)
    _within((p[:total], m[:total], v[:total]), ref, bound, "views")
    assert torch.equal(low[:total], p[:total].bfloat16()) and torch.all(low[total:] == 9.0)
    assert all(torch.equal(a[total:], b[total:]) for a, b in zip((p, m, v), keep))


def test_zero_gradients_only_decay():
    p, m, v = _state([(1000,)], zero=True)
    q = p[0].clone()
    o = rn.AdamW([(1000,)], weight_decay=0.5, m=m, v=v)
    o.step(p, [torch.zeros(1000, device="cuda")], 0.125)
    assert torch.equal(p[0], q - 0.125 * (0.5 * q)) and not m[0].any() and not v[0].any()


def test_a_captured_step_counts_its_replays():
    shapes = [(3000,), (40, 40)]
    grads = _grads(shapes, ["f32"] * 2)
    lr = torch.tensor(0.01, device="cuda")

    def make():
        p, _, _ = _state(shapes, seed=3)
        return p, rn.GradClip(shapes), rn.AdamW(shapes)

    def step(p, c, o):
        o.step(p, grads, lr, clip=c.norm(grads))

    p, c, o = make()
    for _ in range(4):
        step(p, c, o)
    ref = [t.clone() for t in p]
    q, c, o = make()
    s = torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(g, stream=s):
        step(q, c, o)
    for _ in range(4):
        g.replay()
    torch.cuda.synchronize()
    assert o.steps.tolist() == [4, 0]
    assert all(torch.equal(a, b) for a, b in zip(q, ref))


def test_the_same_bits_again_and_on_another_stream():
    shapes = [(1 << 20,), (333, 77)]
    grads = _grads(shapes, ["f32", "bf16"])
    c = rn.GradClip(shapes, dtype=["f32", "bf16"])
    ref = c.norm(grads)
    assert all(torch.equal(c.norm(grads), ref) for _ in range(5))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = c.norm(grads, stream=s)
    into = [torch.zeros_like(x) for x in grads]
    s.wait_stream(torch.cuda.current_stream())
    c.clip(grads, into=into, stream=s)
    s.synchronize()
    assert torch.equal(got, ref)
    _check_scaled(into, grads, float(ref[1]))


def test_tensors_past_32_bits_of_bytes():
    n = (1 << 30) + 5  # 4 GB of fp32
    g = torch.ones(n, device="cuda")
    g[-1] = 2.0
    c = rn.GradClip([(n,)], max_norm=float(np.sqrt(n + 3.0)) / 4, eps=0.0)
    out = c.clip([g])
    assert abs(float(out[0]) - np.sqrt(n + 3.0)) <= 20 * U * np.sqrt(n + 3.0)
    scale = float(out[1])
    assert float(g[0]) == scale and float(g[n // 2]) == scale and float(g[-1]) == 2 * scale
    assert float(g[-2]) == scale


def test_overlapping_tensors_are_refused():
    a = torch.zeros(100, device="cuda")
    g = [torch.zeros(60, device="cuda"), torch.zeros(60, device="cuda")]
    o = rn.AdamW([(60,), (60,)])
    for params in ([a[:60], a[:60]], [a[:60], a[40:]], [a[40:], a[:60]], [g[0], a[:60]],
                   [o.m[0], a[:60]], [a[:60], o.v[1]]):
        with pytest.raises(rn.RnntError):
            o.step(params, g, 0.1)
    p = [torch.zeros(60, device="cuda") for _ in range(2)]
    low = a.view(torch.bfloat16)
    with pytest.raises(rn.RnntError):
        o.step(p, g, 0.1, low=[low[:60], low[59:119]])
    o.step(p, [g[0], g[0]], 0.1)  # one gradient for two parameters is fine
    c = rn.GradClip([(60,), (60,)])
    with pytest.raises(rn.RnntError):
        c.clip([a[:60], a[40:]])
    with pytest.raises(rn.RnntError):
        c.clip(g, into=[a[:60], a[:60]])
    with pytest.raises(rn.RnntError):
        c.clip(g, into=[g[1], g[0]])
    c.norm([a[:60], a[40:]])  # reading is fine
    assert o.steps.tolist() == [1, 0]
