"""Layer norm's gradients against differences of its forward pass in 64 bits.

Each row is moved alone along four directions of length 1: a random one, a = gamma dy itself (where
the gradient is large), the constant one (which only mean(a) answers) and the normalised row (which
only the xh term answers).  A central
difference of step h is off by h^2 of third derivatives, at most 10 |a| h^2 rstd^3 here, beside
2^-52 |a| sqrt(C) / h of rounding; a computed gradient g by k u r of its terms' sizes and half a
step of its type in every channel, as test_gpu_ops_ln.py derives them (u = 2^-24, k = 64 + C / 256,
r = 1 + |mean| rstd).  The same check has to fail for gradients that lack a term (CPU).
"""
import numpy as np
import pytest
import torch

import asr_tiled_tanh_gb300 as rn

DT = {"f32": torch.float32, "bf16": torch.bfloat16}
HALF = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8}
U, EPS = 2.0 ** -24, 1e-5
WIDTHS = [24, 96, 333, 640, 2048, 9000]


def _inputs(C, dtype, seed=0):
    g = torch.Generator().manual_seed(seed + C)
    n = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    x = (n(2, 5, C) * torch.rand(C, generator=g).add(0.3) + n(C)).to(DT[dtype])
    return x, n(2, 5, C).to(DT[dtype]), 1 + 0.3 * n(C), 0.3 * n(C), torch.tensor([5, 3])


def _forward(x, gamma, beta):
    xc = x - x.mean(-1, keepdims=True)
    return gamma * xc / np.sqrt((xc * xc).mean(-1, keepdims=True) + EPS) + beta


def _agree(inputs, dtype, dx, dgamma, dbeta):
    """Whether all differences agree (arrays of 64 bits)."""
    x, dy, gamma, beta = (t.double().numpy() for t in inputs[:4])
    C, good, rng = x.shape[2], True, np.random.default_rng(1)
    live = np.arange(x.shape[1])[None] < inputs[4].numpy()[:, None]
    mean = x.mean(-1, keepdims=True)
    rstd = 1 / np.sqrt(x.var(-1, keepdims=True) + EPS)
    xh, r, k = (x - mean) * rstd, 1 + np.abs(mean) * rstd, 64 + C / 256
    a = gamma * dy
    size = rstd * (np.abs(a) + np.abs(a).mean(-1, keepdims=True) + (np.abs(xh) + r)
                   * (np.abs(a) * (np.abs(xh) + r)).mean(-1, keepdims=True))
    each = k * U * r * size + HALF[dtype] * np.abs(dx) + 1e-38
    for b, t in np.ndindex(*live.shape):
        if not live[b, t]:
            good &= not dx[b, t].any()
            continue
        loss = lambda row: (dy[b, t] * _forward(row, gamma, beta)).sum()  # noqa: E731
        for d in (rng.standard_normal(C), a[b, t], np.ones(C), xh[b, t]):
            d = d / np.linalg.norm(d)
            s, n = rstd[b, t, 0], np.linalg.norm(a[b, t])
            h = 1e-4 / s
            diff = (loss(x[b, t] + h * d) - loss(x[b, t] - h * d)) / (2 * h)
            tol = 10 * n * h * h * s ** 3 + 2.0 ** -52 * n * np.sqrt(C) / h
            good &= abs(diff - dx[b, t] @ d) <= tol + each[b, t] @ np.abs(d)
    # in scale and offset the loss is linear: a step of 1 in each channel
    rows = dy * live[..., None]
    for got, diff, term in ((dgamma, (rows * (_forward(x, 1.0, 0.0))).sum((0, 1)),
                             (np.abs(rows) * (np.abs(xh) + r)).sum((0, 1))),
                            (dbeta, rows.sum((0, 1)), np.abs(rows).sum((0, 1)))):
        good &= bool((np.abs(got - diff) <= (k + 1) * U * term + HALF["f32"] * np.abs(diff)).all())
    return bool(good)


def _formula(inputs, means=1.0, along=1.0, deviation=1.0, scale=1.0):
    """(dx, dgamma, dbeta) in 64 bits, its terms by these factors."""
    x, dy, gamma, _ = (t.double().numpy() for t in inputs[:4])
    live = (np.arange(x.shape[1])[None] < inputs[4].numpy()[:, None])[..., None]
    rstd = 1 / np.sqrt(x.var(-1, keepdims=True) + EPS)
    xh, a = (x - x.mean(-1, keepdims=True)) * rstd, gamma * dy
    dx = scale * rstd ** deviation * (a - means * a.mean(-1, keepdims=True)
                                      - along * xh * (a * xh).mean(-1, keepdims=True))
    return dx * live, (dy * xh * live).sum((0, 1)), (dy * live).sum((0, 1))


def _rounded(t, dtype):
    return torch.from_numpy(t).to(DT[dtype]).double().numpy()


@pytest.mark.parametrize("C", WIDTHS)
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_the_check_tells_gradients_from_others(C, dtype):
    inputs = _inputs(C, dtype)

    def says(change=None, **k):
        dx, dg, db = _formula(inputs, **k)
        out = [_rounded(dx, dtype), dg, db]
        if change:
            change(out)
        return _agree(inputs, dtype, *out)
    assert says()
    for wrong in (dict(means=0.0), dict(along=0.0), dict(means=0.0, along=0.0), dict(scale=1.2),
                  dict(scale=0.97), dict(deviation=0.0), dict(deviation=2.0), dict(along=-1.0)):
        assert not says(**wrong), wrong

    def dead(out):
        out[0][1, 4, 0] = 1e-6

    def swapped(out):
        out[1], out[2] = out[2], out[1]

    def short(out):  # a row left out of the offset's gradient
        out[2] = out[2] - inputs[1].double().numpy()[0, 2]

    for change in (dead, swapped, short):
        assert not says(change), change.__name__


@pytest.mark.gpu
@pytest.mark.parametrize("C", WIDTHS)
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_gradients_are_differences(C, dtype):
    rn.load(build_if_missing=True)
    inputs = _inputs(C, dtype)
    x, dy, gamma, beta, lengths = (t.cuda() for t in inputs)
    n = rn.LayerNorm(2, 5, C, dtype=dtype, eps=EPS)
    n.fwd(x, gamma, beta, lengths.int())
    got = n.bwd(x, dy, gamma, lengths.int())
    assert _agree(inputs, dtype, *(t.double().cpu().numpy() for t in got))
