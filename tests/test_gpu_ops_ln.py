"""Layer norm of rows against a plain implementation in 64 bits (GPU).

Tolerances.  u = 2^-24 is half a step of fp32.  A row's sums add C / 256 or 32 terms one after
another, then meet in a tree: the mean is at most k u |x| off with k = 64 + C / 256, and x - mean,
taken times rstd, k u (1 + r) off where r is the row's |mean| rstd.  Every output is a sum of terms
that carry such errors, so its error is at most k u (1 + r) of the terms' sizes (not of their
sum, which may cancel), and half a step of its own type: 2^-24 or 2^-8.  Parameter gradients add
rows in chains of at most N / 64 terms: k counts these too.
"""
import numpy as np
import pytest
import torch

import asr_tiled_tanh_gb300 as rn

pytestmark = pytest.mark.gpu
DT = {"f32": torch.float32, "bf16": torch.bfloat16}
U = 2.0 ** -24
HALF = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8}


@pytest.fixture(scope="module", autouse=True)
def _lib():
    rn.load(build_if_missing=True)


def _alive(lengths, T, label_rows):
    return np.arange(T)[None] < np.asarray(lengths)[:, None] + int(label_rows)


def _check(got, ref, size, half, k, what):
    """got within k u of the terms' sizes, and half a step of the value."""
    got = got.double().cpu().numpy()
    err, tol = np.abs(got - ref), k * U * size + half * np.abs(ref) + 1e-38
    bad = ~(err <= tol)
    assert not bad.any(), (what, np.argwhere(bad)[0], err[bad][0], tol[bad][0])


def _compare(case, x, dy, gamma, beta, lengths, eps, y, dx, dg, db):
    """Everything against 64 bits; x and dy on the CPU, finite everywhere."""
    B, T, C, dtype, out, label_rows = case
    live = _alive(lengths, T, label_rows)[..., None]
    xd, gd = x.double().numpy(), dy.double().numpy()
    g = np.ones(C) if gamma is None else gamma.double().numpy()
    b = np.zeros(C) if beta is None else beta.double().numpy()
    mean, var = xd.mean(2, keepdims=True), xd.var(2, keepdims=True)
    rstd = 1 / np.sqrt(var + eps)
    r = 1 + np.abs(mean) * rstd
    xh = (xd - mean) * rstd
    k = 64 + C / 256
    _check(y, (xh * g + b) * live, (np.abs(g) * (np.abs(xh) + r) + np.abs(b)) * live, HALF[out], k,
           "y")
    if dx is None:
        return
    a = g * gd
    m1, m2 = a.mean(2, keepdims=True), (a * xh).mean(2, keepdims=True)
    s1, s2 = np.abs(a).mean(2, keepdims=True), (np.abs(a) * (np.abs(xh) + r)).mean(2, keepdims=True)
    size = rstd * (np.abs(a) + s1 + (np.abs(xh) + r) * s2)
    _check(dx, rstd * (a - m1 - xh * m2) * live, size * r * live, HALF[dtype], k, "dx")
    k += B * T / 64
    gd = gd * live
    for got, ref, size, what in ((dg, (gd * xh).sum((0, 1)), (np.abs(gd) * (np.abs(xh) + r)), "dg"),
                                 (db, gd.sum((0, 1)), np.abs(gd), "db")):
        if got is not None:
            _check(got, ref, size.sum((0, 1)), HALF["f32"], k, what)


def _inputs(B, T, C, dtype, out, label_rows=False, seed=0, offset=1.0, full=False):
    g = torch.Generator().manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    x = (n(B, T, C) * torch.rand(C, generator=g).add(0.3) + offset * n(C)).to(DT[dtype])
    dy = n(B, T, C).to(DT[out])
    top = T - 1 if label_rows else T
    lengths = torch.randint(0, top + 1, (B,), generator=g, dtype=torch.int32)
    lengths[0] = top
    if B > 2:
        lengths[1], lengths[2] = 0, min(1, top)
    if full:
        lengths[:] = top
    return x, dy, 1 + 0.3 * n(C), 0.3 * n(C), lengths


def _poison(t, lengths, label_rows, value):
    """A copy on the GPU whose rows that do not exist hold `value`."""
    t = t.clone()
    t[torch.from_numpy(~_alive(lengths, t.shape[1], label_rows))] = value
    return t.cuda()


SHAPES = [(1, 1, 1), (1, 1, 2), (8, 1, 512), (3, 7, 12), (7, 33, 360), (5, 40, 64), (4, 50, 96),
          (9, 31, 8), (4, 60, 512), (3, 21, 640), (3, 40, 1000), (2, 30, 1024), (300, 3, 24),
          (2, 17, 1032), (2, 9, 2048), (2, 25, 4096), (1, 5, 8200), (2, 3, 20000), (1, 2, 40004),
          (3, 11, 333), (2, 19, 1001), (70, 40, 130), (1, 3000, 32), (1, 2, 33), (3, 5, 4100)]


@pytest.mark.parametrize("B,T,C", SHAPES)
@pytest.mark.parametrize("dtype,out", [("f32", "f32"), ("bf16", "bf16"), ("f32", "bf16"),
                                       ("bf16", "f32")])
def test_matches_64_bits(B, T, C, dtype, out):
    case = (B, T, C, dtype, out, False)
    x, dy, gamma, beta, lengths = _inputs(*case, seed=C + T)
    n = rn.LayerNorm(B, T, C, dtype=dtype, out_dtype=out)
    y = torch.full((B, T, C), float("nan"), dtype=DT[out], device="cuda")
    dx = torch.full((B, T, C), float("nan"), dtype=DT[dtype], device="cuda")
    xg, dyg = _poison(x, lengths, False, float("nan")), _poison(dy, lengths, False, float("inf"))
    n.fwd(xg, gamma.cuda(), beta.cuda(), lengths.cuda(), y=y)
    dx, dg, db = n.bwd(xg, dyg, gamma.cuda(), lengths.cuda(), dx=dx)
    _compare(case, x, dy, gamma, beta, lengths.numpy(), 1e-5, y, dx, dg, db)
    assert n.status() == (0, 0)


# Widths for every number of lanes and units: parts of a warp, a warp, several; 16-byte units,
# pairs, channels apart; a block a row.
WIDTHS = [3, 4, 5, 6, 8, 10, 16, 18, 24, 32, 36, 48, 50, 72, 96, 100, 127, 144, 192, 250, 256, 264,
          320, 321, 384, 400, 480, 600, 640, 704, 767, 768, 770, 776, 1002, 1280, 1281, 1536, 2002,
          2047, 2560, 3000, 4094, 6144, 8190, 8192, 12288, 16386]


@pytest.mark.parametrize("C", WIDTHS)
@pytest.mark.parametrize("dtype,out", [("f32", "f32"), ("bf16", "bf16"), ("f32", "bf16"),
                                       ("bf16", "f32")])
def test_every_width(C, dtype, out):
    B, T = 3, 5
    case = (B, T, C, dtype, out, False)
    x, dy, gamma, beta, lengths = _inputs(*case, seed=C)
    n = rn.LayerNorm(B, T, C, dtype=dtype, out_dtype=out)
    xg, dyg = _poison(x, lengths, False, float("nan")), _poison(dy, lengths, False, float("inf"))
    y = n.fwd(xg, gamma.cuda(), beta.cuda(), lengths.cuda())
    _compare(case, x, dy, gamma, beta, lengths.numpy(), 1e-5, y,
             *n.bwd(xg, dyg, gamma.cuda(), lengths.cuda()))


@pytest.mark.parametrize("B,T,C", [(1, 1, 16), (4, 9, 512), (5, 1, 64), (3, 12, 77),
                                   (64, 101, 128)])
@pytest.mark.parametrize("given", [True, False])
def test_label_rows_and_parameters_left_out(B, T, C, given):
    case = (B, T, C, "bf16", "bf16", True)
    x, dy, gamma, beta, lengths = _inputs(*case, seed=3)
    if not given:
        gamma = beta = None
    on = lambda t: None if t is None else t.cuda()  # noqa: E731
    n = rn.LayerNorm(B, T, C, label_rows=True)
    xg, dyg = _poison(x, lengths, True, float("inf")), _poison(dy, lengths, True, float("nan"))
    y = n.fwd(xg, on(gamma), on(beta), lengths.cuda())
    dx, dg, db = n.bwd(xg, dyg, on(gamma), lengths.cuda())
    _compare(case, x, dy, gamma, beta, lengths.numpy(), 1e-5, y, dx, dg, db)


def test_every_row_without_lengths():
    case = (3, 20, 256, "f32", "f32", False)
    x, dy, gamma, beta, lengths = _inputs(*case, full=True)
    n = rn.LayerNorm(3, 20, 256, dtype="f32")
    y = n.fwd(x.cuda(), gamma.cuda(), beta.cuda())
    _compare(case, x, dy, gamma, beta, lengths.numpy(), 1e-5, y,
             *n.bwd(x.cuda(), dy.cuda(), gamma.cuda()))


def test_offsets_far_from_zero():
    # a mean of thousands of deviations: the variance is taken about the mean
    case = (2, 10, 512, "f32", "f32", False)
    x, dy, gamma, beta, lengths = _inputs(*case, full=True)
    x = x + 3000.0
    n = rn.LayerNorm(2, 10, 512, dtype="f32")
    y = n.fwd(x.cuda(), gamma.cuda(), beta.cuda())
    _compare(case, x, dy, gamma, beta, lengths.numpy(), 1e-5, y,
             *n.bwd(x.cuda(), dy.cuda(), gamma.cuda()))


def test_constant_rows():
    # no deviation: y is the offset alone, and eps bounds the gradient
    x = torch.full((2, 3, 96), 7.0, device="cuda")
    beta = torch.randn(96, device="cuda")
    n = rn.LayerNorm(2, 3, 96, dtype="f32")
    assert torch.equal(n.fwd(x, None, beta), beta.expand(2, 3, 96))
    dx, dg, db = n.bwd(x, torch.ones_like(x))
    assert torch.all(dg == 0) and torch.all(db == 6) and dx.abs().max() < 1e-3


def _strided(shape, layout, dtype, pad, shift):
    """An empty [B,T,C] view of a buffer full of 77, and the buffer."""
    B, T, C = shape
    f = C + pad
    strides = (T * f + 3 * pad, f, 1) if layout == "samples" else (f, B * f + 2 * pad, 1)
    span = (B - 1) * strides[0] + (T - 1) * strides[1] + C
    buf = torch.full((span + shift + 64,), 77.0, dtype=dtype, device="cuda")
    return buf[shift:shift + span + 0].as_strided(shape, strides, shift), buf


@pytest.mark.parametrize("layout", ["samples", "frames"])
@pytest.mark.parametrize("pad,shift", [(0, 0), (8, 8), (8, 1), (3, 0), (5, 3), (4, 2)])
@pytest.mark.parametrize("dtype,out", [("f32", "bf16"), ("bf16", "bf16")])
@pytest.mark.parametrize("C", [64, 500])
def test_strides_and_alignment(layout, pad, shift, dtype, out, C):
    B, T = 3, 11
    case = (B, T, C, dtype, out, False)
    x, dy, gamma, beta, lengths = _inputs(*case, seed=9)
    xs, xbuf = _strided((B, T, C), layout, DT[dtype], pad, shift)
    gs, _ = _strided((B, T, C), layout, DT[out], pad, shift)
    ys, ybuf = _strided((B, T, C), layout, DT[out], pad, shift)
    ds, dbuf = _strided((B, T, C), layout, DT[dtype], pad, shift)
    xs.copy_(_poison(x, lengths, False, float("nan")))
    gs.copy_(_poison(dy, lengths, False, float("nan")))
    n = rn.LayerNorm(B, T, C, dtype=dtype, out_dtype=out, x_strides=xs.stride()[:2],
                     y_strides=ys.stride()[:2])
    a = gamma.cuda(), lengths.cuda()
    n.fwd(xs, a[0], beta.cuda(), a[1], y=ys)
    _, dg, db = n.bwd(xs, gs, *a, dx=ds)
    _compare(case, x, dy, gamma, beta, lengths.numpy(), 1e-5, ys, ds, dg, db)
    for view, buf in ((ys, ybuf), (ds, dbuf)):  # nothing else was written
        view.fill_(77.0)
        assert torch.all(buf == 77.0)


def test_gamma_off_16_bytes():
    case = (2, 6, 512, "bf16", "bf16", False)
    x, dy, gamma, beta, lengths = _inputs(*case, full=True)
    g, b = (torch.cat([torch.zeros(1), t]).cuda()[1:] for t in (gamma, beta))
    n = rn.LayerNorm(2, 6, 512)
    y = n.fwd(x.cuda(), g, b)
    dgb = torch.zeros(2, 513, device="cuda")
    dx, dg, db = n.bwd(x.cuda(), dy.cuda(), g, dgamma=dgb[0, 1:], dbeta=dgb[1, :512])
    _compare(case, x, dy, gamma, beta, lengths.numpy(), 1e-5, y, dx, dg, db)


@pytest.mark.parametrize("C", [512, 77, 9000])
def test_what_the_c_side_may_leave_out(C):
    # no statistics kept, and either or both of the parameters' gradients not wanted
    B, T = 3, 4
    x, dy, gamma, beta, lengths = (t.cuda() for t in _inputs(B, T, C, "f32", "f32", seed=1))
    n = rn.LayerNorm(B, T, C, dtype="f32")
    y, ref = n.fwd(x, gamma, beta, lengths), n.bwd(x, dy, gamma, lengths)
    p = lambda t: None if t is None else t.data_ptr()  # noqa: E731
    out = torch.full_like(y, 5.0)
    assert n._fwd(n._d, p(x), p(gamma), p(beta), p(lengths), p(out), None, None,
                  n._stream(None)) == 0
    assert torch.equal(out, y)
    for want in ((0, 0), (1, 0), (0, 1)):
        dx, dg, db = torch.full_like(x, 5.0), *torch.full((2, C), 5.0, device="cuda")
        assert n._bwd(n._d, p(x), p(dy), p(gamma), p(lengths), n._saved, p(dx),
                      p(dg) if want[0] else None, p(db) if want[1] else None, *n._args,
                      n._stream(None)) == 0
        assert torch.equal(dx, ref[0])
        assert torch.equal(dg, ref[1]) if want[0] else torch.all(dg == 5.0)
        assert torch.equal(db, ref[2]) if want[1] else torch.all(db == 5.0)


def test_no_rows_at_all():
    B, T, C = 4, 5, 40
    n = rn.LayerNorm(B, T, C)
    x = torch.full((B, T, C), float("nan"), dtype=torch.bfloat16, device="cuda")
    z = torch.zeros(B, dtype=torch.int32, device="cuda")
    assert torch.all(n.fwd(x, None, None, z) == 0)
    dx, dg, db = n.bwd(x, x, None, z, dgamma=torch.ones(C, device="cuda"))
    assert torch.all(dx == 0) and torch.all(dg == 0) and torch.all(db == 0)
    assert n.status() == (0, 0)


def test_an_empty_batch():
    n = rn.LayerNorm(0, 5, 40, dtype="f32")
    x = torch.empty(0, 5, 40, device="cuda")
    assert n.fwd(x).shape == (0, 5, 40)
    one = lambda: torch.ones(40, device="cuda")  # noqa: E731
    _, dg, db = n.bwd(x, x, dgamma=one(), dbeta=one())
    assert torch.all(dg == 0) and torch.all(db == 0)


@pytest.mark.parametrize("label_rows,bad", [(False, -1), (False, 8), (True, -1), (True, 7)])
def test_lengths_out_of_range(label_rows, bad):
    B, T, C = 3, 7, 48
    case = (B, T, C, "f32", "f32", label_rows)
    x, dy, gamma, beta, lengths = _inputs(*case)
    lengths[1] = bad
    n = rn.LayerNorm(B, T, C, dtype="f32", label_rows=label_rows)
    y = n.fwd(x.cuda(), gamma.cuda(), beta.cuda(), lengths.cuda())
    dx, dg, db = n.bwd(x.cuda(), dy.cuda(), gamma.cuda(), lengths.cuda())
    assert n.status()[0] == 4
    assert torch.all(y[1] == 0) and torch.all(dx[1] == 0)
    lengths[1] = -1 if label_rows else 0  # as a sample without rows
    _compare(case, x, dy, gamma, beta, lengths.numpy(), 1e-5, y, dx, dg, db)


def test_gradients_are_differences_of_the_forward():
    # sum(dy * y) rises by <d, step> for steps of x, gamma and beta
    case = (2, 5, 96, "f32", "f32", False)
    x, dy, gamma, beta, lengths = _inputs(*case, seed=4)
    n = rn.LayerNorm(2, 5, 96, dtype="f32")
    L = lengths.cuda()
    f = lambda x, g, b: (n.fwd(x, g, b, L).double() * dy.cuda().double()).sum()  # noqa: E731
    at = [t.cuda() for t in (x, gamma, beta)]
    n.fwd(*at, L)
    grads = n.bwd(at[0], dy.cuda(), at[1], L)
    torch.manual_seed(1)
    for i in range(3):
        step = torch.randn_like(at[i])
        h = 1e-2  # differences: h^2 of the third derivative, u / h of the rounding
        hi, lo = list(at), list(at)
        hi[i], lo[i] = at[i] + h * step, at[i] - h * step
        diff = (f(*hi) - f(*lo)) / (2 * h)
        # 1e-2: h^2 times third derivatives of order 10 of the value's size
        assert abs(diff - (grads[i].double() * step).sum()) <= 1e-2 * grads[i].norm() * step.norm()


def test_the_same_bits_again_in_a_graph_and_on_another_stream():
    B, T, C = 6, 50, 512
    x, dy, gamma, beta, lengths = (t.cuda() for t in _inputs(B, T, C, "bf16", "bf16", seed=2))
    n = rn.LayerNorm(B, T, C)
    run = lambda **k: [n.fwd(x, gamma, beta, lengths, **k),  # noqa: E731
                       *n.bwd(x, dy, gamma, lengths, **k)]
    ref = run()
    assert all(torch.equal(a, b) for a, b in zip(run(), ref))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = run(stream=s)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, ref))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = run()
    for _ in range(2):
        for t in out:
            t.fill_(float("nan"))
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, ref))


@pytest.mark.parametrize("B,T,C,dtype", [(700, 90, 40, "f32"), (300, 60, 512, "bf16"),
                                         (150, 40, 1280, "bf16"), (200, 70, 333, "bf16"),
                                         (200, 70, 330, "f32"), (90, 60, 1500, "f32")])
def test_more_rows_than_the_grid(B, T, C, dtype):
    # teams that walk over many ragged samples
    x, dy, gamma, beta, lengths = _inputs(B, T, C, dtype, dtype, seed=6)
    n = rn.LayerNorm(B, T, C, dtype=dtype)
    xg = _poison(x, lengths, False, float("nan"))
    y = n.fwd(xg, gamma.cuda(), beta.cuda(), lengths.cuda())
    dx, dg, db = n.bwd(xg, _poison(dy, lengths, False, float("nan")), gamma.cuda(), lengths.cuda())
    _compare((B, T, C, dtype, dtype, False), x, dy, gamma, beta, lengths.numpy(), 1e-5, y, dx, dg,
             db)


@pytest.mark.parametrize("C,dtype", [(56, "f32"), (720, "bf16"), (1544, "bf16"), (131, "bf16")])
def test_a_first_call_may_be_captured(C, dtype):
    x, dy, gamma, beta, lengths = (t.cuda() for t in _inputs(4, 6, C, dtype, dtype, seed=2))
    n = rn.LayerNorm(4, 6, C, dtype=dtype)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = [n.fwd(x, gamma, beta, lengths), *n.bwd(x, dy, gamma, lengths)]
    g.replay()
    torch.cuda.synchronize()
    ref = [n.fwd(x, gamma, beta, lengths), *n.bwd(x, dy, gamma, lengths)]
    assert all(torch.equal(a, b) for a, b in zip(out, ref))


def test_rows_of_infinities_and_nan_stay_by_themselves():
    # (rows that share a warp)
    for C, dtype in ((16, "f32"), (64, "bf16"), (130, "bf16"), (512, "bf16")):
        x, dy, gamma, beta, lengths = (t.cuda() for t in _inputs(2, 40, C, dtype, dtype, full=True))
        n = rn.LayerNorm(2, 40, C, dtype=dtype)
        ref = n.fwd(x, gamma, beta), n.bwd(x, dy, gamma)[0]
        bad = x.clone()
        bad[0, 3, 1], bad[0, 7, 0], bad[1, 39, C - 1] = float("inf"), float("nan"), -float("inf")
        got = n.fwd(bad, gamma, beta), n.bwd(bad, dy, gamma)[0]
        hit = torch.zeros(2, 40, dtype=torch.bool, device="cuda")
        hit[0, 3] = hit[0, 7] = hit[1, 39] = True
        for a, b in zip(got, ref):
            assert torch.equal(a[~hit], b[~hit])
            assert torch.isnan(a[hit].float()).any(1).all()


def test_offsets_past_32_bits():
    # rows that begin beyond 2^32 bytes and 2^31 elements of their buffer
    B, T, C = 3, 2, 64
    xb = 1 << 30
    buf = torch.empty(2 * xb + 2 * C, dtype=torch.bfloat16, device="cuda")
    x = buf.as_strided((B, T, C), (xb, C, 1))
    src = torch.randn(B, T, C, device="cuda").bfloat16()
    x.copy_(src)
    n = rn.LayerNorm(B, T, C, x_strides=(xb, C))
    d = rn.LayerNorm(B, T, C)
    assert torch.equal(n.fwd(x), d.fwd(src))
    got, ref = n.bwd(x, src), d.bwd(src, src)
    assert got[0].stride() == x.stride()
    assert all(torch.equal(a, b) for a, b in zip(got, ref))
