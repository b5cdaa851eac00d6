"""Group norm with an activation, channels last, against a plain 64-bit implementation (GPU).

Tolerances, relative 2-norm over the frames that exist.  fp32: every element passes through a
mean, a variance and a few products; x - mean loses the digits that a mean of r standard
deviations takes, so 64 2^-24 (1 + r), r the largest |mean| rstd.  bf16: the result's own
rounding is at most 2^-9; twice that, 2^-8, leaves as much again for the computation.  Parameter
gradients are fp32 sums of terms g xh that carry those errors: 64 2^-24 (1 + r) of the terms'
2-norm times the square root of their number.  relu has no derivative at 0: an element whose u
lies within u's own error of 0 may take either side's, so it is left out of dx, and its term is
allowed for in the sums.
"""
import numpy as np
import pytest
import torch

import asr_tiled_tanh_gb300 as rn

pytestmark = pytest.mark.gpu
DT = {"f32": torch.float32, "bf16": torch.bfloat16}
U32 = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def _lib():
    rn.load(build_if_missing=True)


def _act(act, u):
    s = 1 / (1 + np.exp(-np.clip(u, -700, 700)))
    if act == "silu":
        return u * s, s * (1 + u * (1 - s))
    if act == "relu":
        return np.maximum(u, 0), (u > 0).astype(float)
    return u, np.ones_like(u)


def _ref(x, gamma, beta, T_len, G, act, eps, dy=None):
    """(y, r) or (y, r, dx, dgamma, dbeta, terms, kink, kink terms) in 64 bits, group by group."""
    B, T, C = x.shape
    cg = C // G
    y, dx = np.zeros_like(x), np.zeros_like(x)
    dg, db, tg, tb_, kg, kb = (np.zeros(C) for _ in range(6))
    kink = np.zeros(x.shape, bool)
    r = 0.0
    for b in range(B):
        t = int(T_len[b])
        if t == 0:
            continue
        for g in range(G):
            cs = slice(g * cg, (g + 1) * cg)
            v = x[b, :t, cs]
            mean, var = v.mean(), v.var()
            rstd = 1 / np.sqrt(var + eps)
            r = max(r, abs(mean) * rstd)
            xh = (v - mean) * rstd
            u = xh * gamma[cs] + beta[cs]
            f, d = _act(act, u)
            y[b, :t, cs] = f
            if dy is None:
                continue
            gg = dy[b, :t, cs] * d
            dg[cs] += (gg * xh).sum(0)
            db[cs] += gg.sum(0)
            tg[cs] += ((gg * xh) ** 2).sum(0)
            tb_[cs] += (gg ** 2).sum(0)
            if act == "relu":
                k = np.abs(u) <= 64 * U32 * (1 + abs(mean) * rstd) * (1 + np.abs(xh * gamma[cs]))
                kink[b, :t, cs] = k
                kg[cs] += np.abs(k * dy[b, :t, cs] * xh).sum(0)
                kb[cs] += np.abs(k * dy[b, :t, cs]).sum(0)
            gg = gg * gamma[cs]
            dx[b, :t, cs] = rstd * (gg - gg.mean() - xh * (gg * xh).mean())
    return (y, r) if dy is None else (y, r, dx, dg, db, np.sqrt(tg), np.sqrt(tb_), kink, kg, kb)


def _inputs(B, T, C, dtype, seed, full=False, offset=1.0):
    g = torch.Generator().manual_seed(seed)
    x = (torch.randn(B, T, C, generator=g) * torch.rand(C, generator=g).add(0.3)
         + offset * torch.randn(C, generator=g)).to(DT[dtype])
    dy = torch.randn(B, T, C, generator=g).to(DT[dtype])
    gamma, beta = 1 + 0.3 * torch.randn(C, generator=g), 0.3 * torch.randn(C, generator=g)
    T_len = torch.randint(0, T + 1, (B,), generator=g, dtype=torch.int32)
    T_len[0] = T
    if B > 2:
        T_len[1], T_len[2] = 0, 1
    if full:
        T_len[:] = T
    return x, dy, gamma, beta, T_len


def _rel(got, ref):
    n = np.linalg.norm(ref)
    d = np.linalg.norm(got.double().cpu().numpy() - ref)
    return d / n if n else d


def _run(n, x, dy, gamma, beta, T_len, dev=None):
    """fwd and bwd with the frames past each length poisoned; checks the zeros there."""
    T = x.shape[1]
    gone = torch.arange(T)[None] >= T_len[:, None]
    xd, dyd = x.clone(), dy.clone()
    xd[gone], dyd[gone] = float("nan"), float("inf")
    a = [t.cuda() for t in (xd, gamma, beta, T_len)]
    y = torch.full(x.shape, float("nan"), dtype=x.dtype, device="cuda")
    dx = y.clone()
    n.fwd(*a, y=y)
    dx, dg, db = n.bwd(a[0], dyd.cuda(), *a[1:], dx=dx)
    assert torch.all(y[gone.cuda()] == 0) and torch.all(dx[gone.cuda()] == 0)
    return y, dx, dg, db


SHAPES = [(1, 1, 1, 1), (1, 1, 8, 2), (8, 1, 512, 32), (3, 7, 12, 4), (5, 333, 360, 24),
          (4, 200, 512, 32), (3, 100, 640, 32), (2, 50, 96, 1), (3, 65, 40, 40), (2, 31, 1000, 8),
          (2, 1500, 64, 4), (1, 4000, 48, 2), (1, 9000, 512, 1), (2, 2500, 256, 8),
          (300, 3, 64, 8), (2, 17, 24, 8), (1, 300, 2048, 1)]


@pytest.mark.parametrize("B,T,C,G", SHAPES)
@pytest.mark.parametrize("dtype,act", [("f32", "silu"), ("bf16", "silu"), ("f32", "relu"),
                                       ("bf16", "none")])
def test_forward_and_gradients(B, T, C, G, dtype, act):
    x, dy, gamma, beta, T_len = _inputs(B, T, C, dtype, B + T + C)
    n = rn.FrameNorm(B, T, C, G, act=act, dtype=dtype, eps=1e-5)
    y, dx, dg, db = _run(n, x, dy, gamma, beta, T_len)
    f = lambda t: t.double().numpy()
    # (one element per group has no spread: xh = 0 exactly, up to the mean's rounding)
    ry, r, rdx, rdg, rdb, tg, tb, kink, kg, kb = _ref(f(x), f(gamma), f(beta), T_len.numpy(), G,
                                                      act, 1e-5, f(dy))
    t32 = 64 * U32 * (1 + r)
    tol = t32 if dtype == "f32" else 2.0 ** -8 + t32
    assert n.status() == (0, 0)
    assert _rel(y, ry) <= tol
    # dx is what is left of g after two means are taken out: measured against g's own size
    scale = np.linalg.norm(rdx)
    if C // G * int(T_len.max()) > 2:
        assert np.linalg.norm((dx.double().cpu().numpy() - rdx)[~kink]) <= 4 * tol * scale
    cnt = np.sqrt(float(T_len.sum()))
    assert np.all(np.abs(dg.double().cpu().numpy() - rdg) <= 1e-30 + t32 * tg * cnt + kg)
    assert np.all(np.abs(db.double().cpu().numpy() - rdb) <= 1e-30 + t32 * tb * cnt + kb)


@pytest.mark.parametrize("B,T,C,G,dtype", [(4, 100, 64, 4, "bf16"), (9, 333, 360, 24, "f32")])
def test_same_bits_again(B, T, C, G, dtype):
    x, dy, gamma, beta, T_len = _inputs(B, T, C, dtype, 1)
    n = rn.FrameNorm(B, T, C, G, dtype=dtype)
    a, b = (_run(n, x, dy, gamma, beta, T_len) for _ in range(2))
    assert all(torch.equal(p, q) for p, q in zip(a, b))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("fx,bx,fy,by,off", [(72, 72 * 40, 64, 64 * 40, 0), (67, 67 * 40 + 5, 70, 70 * 41, 0),
                                             (80, 80 * 40, 72, 72 * 40, 8), (64, 64 * 40, 65, 65 * 40, 1)])
def test_strides_leave_the_gaps_alone(dtype, fx, bx, fy, by, off):
    B, T, C, G = 3, 40, 64, 8
    x, dy, gamma, beta, T_len = _inputs(B, T, C, dtype, 4)
    def place(t, b, f):
        buf = torch.full((b * B + off + 8,), 5.0, dtype=t.dtype, device="cuda")
        v = buf[off:].as_strided((B, T, C), (b, f, 1))
        v.copy_(t)
        return buf, v
    (xb, xv), (yb, yv) = place(x, bx, fx), place(dy, by, fy)
    ob, ov = place(torch.zeros_like(x), by, fy)
    gb, gv = place(torch.zeros_like(x), bx, fx)
    n = rn.FrameNorm(B, T, C, G, dtype=dtype, x_strides=(bx, fx), y_strides=(by, fy))
    d = rn.FrameNorm(B, T, C, G, dtype=dtype)
    y, dx, dg, db = _run(d, x, dy, gamma, beta, T_len)
    a = [t.cuda() for t in (gamma, beta, T_len)]
    n.fwd(xv, *a, y=ov)
    _, dg2, db2 = n.bwd(xv, yv, *a, dx=gv)
    f = lambda t: t.float()
    # other variants may sum in another order: equal to the dense result within its rounding
    tol = 1e-5 if dtype == "f32" else 2.0 ** -8
    for p, q in ((ov, y), (gv, dx), (dg2, dg), (db2, db)):
        assert (f(p) - f(q)).norm() <= tol * f(q).norm()
    for buf, v in ((ob, ov), (gb, gv)):
        v.fill_(5.0)
        assert torch.all(buf == 5.0)


def test_large_offsets_keep_the_variance():
    # a mean of 1000 standard deviations: the sum of squares would lose every digit
    x, dy, gamma, beta, T_len = _inputs(2, 500, 64, "f32", 8, full=True, offset=0.0)
    x = x + 1000.0
    n = rn.FrameNorm(2, 500, 64, 4, act="none", dtype="f32")
    y, dx, _, _ = _run(n, x, dy, gamma, beta, T_len)
    f = lambda t: t.double().numpy()
    ry, r, rdx, *_ = _ref(f(x), f(gamma), f(beta), T_len.numpy(), 4, "none", 1e-5, f(dy))
    assert _rel(y, ry) <= 64 * U32 * (1 + r)


def test_constant_groups_and_wild_values():
    # a group without spread: y = act(beta); infinities stay inside their own group and sample
    B, T, C, G = 2, 30, 32, 4
    x, dy, gamma, beta, T_len = _inputs(B, T, C, "f32", 3, full=True)
    x[:, :, :8] = 2.0
    x[1, 4, 9] = float("inf")
    n = rn.FrameNorm(B, T, C, G, act="relu", dtype="f32")
    y = n.fwd(x.cuda(), gamma.cuda(), beta.cuda(), T_len.cuda()).cpu()
    assert torch.allclose(y[:, :, :8], beta[:8].clamp(min=0).expand(B, T, 8), atol=1e-6)
    assert torch.isfinite(y[0]).all() and torch.isfinite(y[1, :, 16:]).all()
    assert torch.isnan(y[1, 4, 9]) or not torch.isfinite(y[1, 4, 9])


@pytest.mark.parametrize("act", ["silu", "none"])
def test_gradient_is_the_derivative(act):
    B, T, C, G = 2, 9, 12, 3
    x, dy, gamma, beta, T_len = _inputs(B, T, C, "f32", 6)
    n = rn.FrameNorm(B, T, C, G, act=act, dtype="f32", eps=1e-3)
    _, dx, dg, db = _run(n, x, dy, gamma, beta, T_len)
    f = lambda t: t.double().numpy()
    rs = np.random.RandomState(0)
    P, pg, pb = rs.randn(B, T, C), rs.randn(C), rs.randn(C)
    L = lambda h: float((_ref(f(x) + h * P, f(gamma) + h * pg, f(beta) + h * pb, T_len.numpy(), G,
                              act, 1e-3)[0] * f(dy)).sum())
    h = 1e-5  # central: error h^2, 1e-10 of third derivatives of order 100
    diff = (L(h) - L(-h)) / (2 * h)
    dot = float((f(dx.cpu()) * P).sum() + (f(dg.cpu()) * pg).sum() + (f(db.cpu()) * pb).sum())
    assert abs(dot - diff) <= 1e-4 * abs(diff) + 1e-4


def test_without_parameters_and_lengths():
    B, T, C, G = 2, 21, 48, 6
    x, dy, _, _, _ = _inputs(B, T, C, "f32", 7)
    one, zero, full = torch.ones(C), torch.zeros(C), torch.full((B,), T, dtype=torch.int32)
    n = rn.FrameNorm(B, T, C, G, dtype="f32")
    ref = _run(n, x, dy, one, zero, full)
    y = n.fwd(x.cuda())
    got = (y,) + n.bwd(x.cuda(), dy.cuda())
    assert all(torch.equal(p, q) for p, q in zip(got, ref))


def test_bad_lengths_are_reported_and_empty():
    B, T, C, G = 3, 10, 16, 2
    x, dy, gamma, beta, _ = _inputs(B, T, C, "f32", 7)
    T_len = torch.tensor([10, 11, -1], dtype=torch.int32)
    n = rn.FrameNorm(B, T, C, G, dtype="f32")
    a = [t.cuda() for t in (gamma, beta, T_len)]
    y = n.fwd(x.cuda(), *a)
    dx, dg, db = n.bwd(x.cuda(), dy.cuda(), *a)
    assert torch.all(y[1:] == 0) and torch.all(dx[1:] == 0) and y[0].abs().sum() > 0
    assert torch.isfinite(dg).all() and n.status()[0] == 4


def test_another_stream_and_a_graph():
    B, T, C, G = 4, 60, 64, 8
    x, dy, gamma, beta, T_len = (t.cuda() for t in _inputs(B, T, C, "bf16", 2))
    n = rn.FrameNorm(B, T, C, G)
    ref = [n.fwd(x, gamma, beta, T_len).clone()] + [t.clone() for t in
                                                    n.bwd(x, dy, gamma, beta, T_len)]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = [n.fwd(x, gamma, beta, T_len), *n.bwd(x, dy, gamma, beta, T_len)]
    s.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(got, ref))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        n.fwd(x, gamma, beta, T_len, y=got[0])
        n.bwd(x, dy, gamma, beta, T_len, dx=got[1], dgamma=got[2], dbeta=got[3])
    for _ in range(2):
        for t in got:
            t.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(got, ref))


# Rows of every alignment (16 bytes, two elements, one), threads of one, two and more groups,
# one group over many blocks, and more slabs than the card holds at a time.
CUTS = [(3, 70, 330, 2), (2, 65, 22, 1), (4, 40, 333, 1), (1, 1100, 1022, 1), (3, 90, 56, 8),
        (3, 90, 72, 8), (2, 120, 96, 24), (3, 1000, 512, 1), (2, 9000, 64, 4), (2, 700, 768, 2),
        (1500, 9, 512, 1), (700, 33, 120, 8)]


@pytest.mark.parametrize("B,T,C,G", CUTS)
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_cuts(B, T, C, G, dtype):
    test_forward_and_gradients(B, T, C, G, dtype, "silu")


# A whole number of samples' slabs would leave an eighth of the clusters idle: blocks change
# channels from slab to slab.
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_blocks_change_channels(dtype):
    test_forward_and_gradients(12, 2000, 512, 32, dtype, "silu")


# A cluster's blocks write their sums into one another's shared memory: blocks whose first slab
# has no frames, or one, get there before the others have begun.
@pytest.mark.parametrize("B,T,C,G", [(40, 2000, 512, 32), (3, 2600, 64, 8), (64, 500, 128, 1)])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_clusters_whose_first_samples_are_empty(B, T, C, G, dtype):
    x, dy, gamma, beta, _ = _inputs(B, T, C, dtype, 11)
    T_len = torch.zeros(B, dtype=torch.int32)
    T_len[B // 2:] = 1
    T_len[-1] = T
    n = rn.FrameNorm(B, T, C, G, dtype=dtype)
    f = lambda t: t.double().numpy()
    ry, r, rdx, rdg, rdb, tg, tb, *_ = _ref(f(x), f(gamma), f(beta), T_len.numpy(), G, "silu",
                                            1e-5, f(dy))
    t32 = 64 * U32 * (1 + r)
    tol = t32 if dtype == "f32" else 2.0 ** -8 + t32
    first = None
    for _ in range(3):
        y, dx, dg, db = _run(n, x, dy, gamma, beta, T_len)
        assert _rel(y, ry) <= tol
        assert np.linalg.norm(dx.double().cpu().numpy() - rdx) <= 4 * tol * np.linalg.norm(rdx)
        cnt = np.sqrt(float(T_len.sum()))
        assert np.all(np.abs(dg.double().cpu().numpy() - rdg) <= 1e-30 + t32 * tg * cnt)
        assert np.all(np.abs(db.double().cpu().numpy() - rdb) <= 1e-30 + t32 * tb * cnt)
        first = first or (y, dx, dg, db)
        assert all(torch.equal(p, q) for p, q in zip(first, (y, dx, dg, db)))
    assert n.status() == (0, 0)


# Where silu's derivative is small, each element of dx for itself: half a unit of its own last
# place, twice, and 64 2^-24 (1 + r) of every term it is made of, where u's error (that, of 1 + |u|)
# reaches act' through act''.
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("B,T,C,G", [(3, 130, 64, 4), (2, 70, 66, 2), (1, 3000, 512, 1)])
def test_each_element_on_the_negative_tail(B, T, C, G, dtype):
    x, dy, _, _, T_len = _inputs(B, T, C, dtype, 13, full=True, offset=0.3)
    g = torch.Generator().manual_seed(5)
    gamma, beta = torch.full((C,), 0.2), -3.6 - 5.8 * torch.rand(C, generator=g)
    n = rn.FrameNorm(B, T, C, G, dtype=dtype)
    _, dx, _, _ = _run(n, x, dy, gamma, beta, T_len)
    f = lambda t: t.double().numpy().reshape(B, T, G, C // G)
    v, d = f(x), f(dy)
    ga, be = (t.double().numpy().reshape(1, 1, G, C // G) for t in (gamma, beta))
    mean, rstd = v.mean((1, 3), keepdims=True), 1 / np.sqrt(v.var((1, 3), keepdims=True) + 1e-5)
    xh = (v - mean) * rstd
    u = xh * ga + be
    assert u.min() > -12 and u.max() < -2
    s = 1 / (1 + np.exp(-u))
    a1, a2 = s * (1 + u * (1 - s)), s * (1 - s) * (2 + u * (1 - 2 * s))
    gg = ga * d * a1
    m1, m2 = gg.mean((1, 3), keepdims=True), (gg * xh).mean((1, 3), keepdims=True)
    ref = rstd * (gg - m1 - xh * m2)
    size = ga * np.abs(d) * (np.abs(a1) + np.abs(a2) * (1 + np.abs(u)))
    size = size + size.mean((1, 3), keepdims=True) + np.abs(xh) * (size * np.abs(xh)).mean(
        (1, 3), keepdims=True)
    tol = 64 * U32 * (1 + (np.abs(mean) * rstd).max()) * rstd * size
    if dtype == "bf16":
        tol = tol + 2.0 ** -8 * np.abs(ref)
    assert np.all(np.abs(f(dx.cpu()) - ref) <= tol)


# Groups of so few channels that a thread holds three or more, over a cluster's blocks; groups that
# end inside a block's columns and go on in the next; as many groups as a slab takes.
@pytest.mark.parametrize("B,T,C,G", [(2, 3000, 24, 8), (2, 3000, 16, 16), (2, 9000, 48, 16),
                                     (2, 40, 8200, 8), (1, 5000, 3084, 12), (3, 500, 4104, 12),
                                     (2, 64, 130, 130), (1, 3000, 254, 127)])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_narrow_and_straddling_groups(B, T, C, G, dtype):
    test_forward_and_gradients(B, T, C, G, dtype, "silu")


# The gradient of a group of one value is 0, not what rounding leaves of terms that cancel.
@pytest.mark.parametrize("B,T,C", [(8, 1, 32), (5, 1, 8), (3, 1, 33), (4, 1, 22), (500, 1, 512),
                                   (6, 3000, 16), (6, 40, 33)])
@pytest.mark.parametrize("dtype,act", [("f32", "silu"), ("bf16", "none"), ("bf16", "silu")])
def test_groups_of_one_value_pass_nothing_on(B, T, C, dtype, act):
    x, dy, gamma, beta, T_len = _inputs(B, T, C, dtype, 17)
    T_len[1:] = 1  # (the first sample has every frame)
    n = rn.FrameNorm(B, T, C, C, act=act, dtype=dtype)
    y, dx, dg, _ = _run(n, x, dy, gamma, beta, T_len)
    assert torch.all(dx[1:, 0] == 0) and (T == 1 or torch.all(dx[0].float().norm(dim=0) > 0))
    ry, *_ = _ref(x[1:, :1].double().numpy(), gamma.double().numpy(), beta.double().numpy(),
                  np.ones(B - 1), C, act, 1e-5)
    tol = 64 * U32 if dtype == "f32" else 2.0 ** -8
    assert _rel(y[1:, :1], ry) <= tol
    assert T > 1 or torch.all(dg == 0)
