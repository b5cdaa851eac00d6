"""Clipping and the AdamW update at the ends of their ranges (GPU)."""
import numpy as np
import pytest
import torch

import asr_tiled_tanh_gb300 as rn

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def _lib():
    rn.load(build_if_missing=True)


def test_moments_whose_memory_moved():
    shapes = [(700,), (30, 5)]
    r = lambda: [torch.randn(k, device="cuda") for k in shapes]  # noqa: E731
    p, g = r(), r()
    q = [t.clone() for t in p]
    a, b = rn.AdamW(shapes), rn.AdamW(shapes)
    old = []
    for i in range(3):
        a.step(p, g, 0.1)
        b.step(q, g, 0.1)
        for t in (b.m[0], b.v[1]):  # (as a program that moved them to the host and back)
            old.append((t.data, t.data.clone()))
            t.data = t.data.clone()
    for x, y in ((p, q), (a.m, b.m), (a.v, b.v)):
        assert all(torch.equal(s, t) for s, t in zip(x, y))
    assert all(torch.equal(s, t) for s, t in old)  # nothing went to where they were


def test_the_count_stays_at_its_end():
    # (the corrections of these betas are 1 there)
    most = (1 << 31) - 1
    with pytest.raises(ValueError):
        rn.AdamW([(3,)], steps=most)
    g = torch.randn(300, device="cuda")
    p = torch.randn(300, device="cuda")
    m, v = 0.1 * torch.randn(300, device="cuda"), 0.1 + torch.rand(300, device="cuda")
    o = rn.AdamW([(300,)], weight_decay=0.0, m=[m], v=[v], steps=most - 1)
    for _ in range(3):
        q = p.double()
        o.step([p], [g], 0.125)
        step = m.double() / (v.double().sqrt() + 1e-8)  # (of the moments as they now are)
        bound = U * p.double().abs() + 0.125 * 32 * U * step.abs()
        assert torch.all((p.double() - (q - 0.125 * step)).abs() <= bound)
        assert o.steps.tolist() == [most, 0]


@pytest.mark.parametrize("n", [8, 400000])  # one launch, and several
def test_a_norm_past_the_range_is_infinite(n):
    shapes = [(n,), (3,)]
    g = [torch.full(k, 1e-3, device="cuda") for k in shapes]
    g[0][1] = g[1][2] = 3e38  # the norm: 4.2e38
    keep = [t.clone() for t in g]
    into = [torch.full_like(t, 5.0) for t in g]
    c, o = rn.GradClip(shapes), rn.AdamW(shapes)
    out = c.clip(g, into=into)
    assert out.tolist() == [float("inf"), 0.0] == c.norm(g).tolist()
    assert not any(t.any() for t in into)
    p = [torch.ones(k, device="cuda") for k in shapes]
    o.step(p, g, 0.1, clip=out)
    assert o.steps.tolist() == [0, 0] and all(torch.all(t == 1) for t in p)
    g[1][2] = 1e38  # 3.2e38
    out = c.norm(g)
    norm = np.sqrt(sum(float((t.double() ** 2).sum()) for t in g))
    assert abs(float(out[0]) - norm) <= 20 * U * norm
    assert abs(float(out[1]) - 1 / norm) <= 22 * U / norm + 2.0 ** -149
    assert torch.equal(g[0], keep[0])


@pytest.mark.parametrize("n", [8, 400000])
def test_an_unlimited_norm(n):
    # scale 1 while the norm is finite, 0 where it is not, NaN where it is none
    g = torch.ones(n, device="cuda")
    c = rn.GradClip([(n,)], max_norm=float("inf"))
    assert float(c.norm([g])[1]) == 1.0
    g[3] = 1e30
    assert float(c.norm([g])[1]) == 1.0
    g[3] = -float("inf")
    assert c.norm([g]).tolist() == [float("inf"), 0.0]
    g[3] = float("nan")
    assert torch.isnan(c.norm([g])).all()


@pytest.mark.parametrize("helper", [True, False])
def test_a_graph_that_holds_old_values_is_refused(helper):
    w, g = torch.ones(40, 3, device="cuda"), torch.ones(40, 3, device="cuda")
    low, x = w.bfloat16(), torch.ones(40, 3, device="cuda", requires_grad=True)
    c, o = rn.GradClip([(40, 3)], max_norm=2.0), rn.AdamW([(40, 3)])
    if not helper:
        c._fast = o._fast = None
    for held, call in ((w, lambda: o.step([w], [g], 0.1)),
                       (low, lambda: o.step([w], [g], 0.1, low=[low])),
                       (g, lambda: c.clip([g]))):
        loss = (x * held).sum()
        call()
        with pytest.raises(RuntimeError, match="modified by an inplace operation"):
            loss.backward()
    with torch.inference_mode():  # (has no count)
        p = torch.ones(40, 3, device="cuda")
    o.step([p], [g], 0.1)
    (x * g).sum().backward()  # what is only read stays
    assert torch.equal(x.grad, g)
