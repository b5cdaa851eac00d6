"""Rows without deviation and rows past fp32's range, whichever kernel takes them (GPU).

Widths: parts of a warp, a warp, several warps, a block a row; 16-byte units, pairs, channels
apart.
"""
import pytest
import torch

import asr_tiled_tanh_gb300 as rn

pytestmark = pytest.mark.gpu
DT = {"f32": torch.float32, "bf16": torch.bfloat16}
WIDTHS = [24, 96, 333, 512, 640, 770, 1000, 2048, 4100, 9000, 13001, 20000, 40004]


@pytest.fixture(scope="module", autouse=True)
def _lib():
    rn.load(build_if_missing=True)


def _inputs(B, T, C, dtype, seed=0):
    g = torch.Generator().manual_seed(seed + C)
    n = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    return ((n(B, T, C) + n(C)).to(DT[dtype]).cuda(), n(B, T, C).to(DT[dtype]).cuda(),
            (1 + 0.3 * n(C)).cuda(), (0.3 * n(C)).cuda())


@pytest.mark.parametrize("C", WIDTHS)
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_rows_whose_squares_leave_the_range_are_nan(C, dtype):
    x, dy, gamma, beta = _inputs(2, 9, C, dtype)
    n = rn.LayerNorm(2, 9, C, dtype=dtype)
    ref = n.fwd(x, gamma, beta), *n.bwd(x, dy, gamma)
    bad = x.clone()
    bad[0, 3, C // 2] = 1e25  # its square
    bad[1, 8] = 3e38  # and the sum of the row
    hit = torch.zeros(2, 9, dtype=torch.bool, device="cuda")
    hit[0, 3] = hit[1, 8] = True
    got = n.fwd(bad, gamma, beta), *n.bwd(bad, dy, gamma)
    for a, b in zip(got[:2], ref[:2]):
        assert torch.equal(a[~hit], b[~hit])
        assert torch.isnan(a[hit].float()).all()
    assert torch.isnan(got[2]).all()
    assert torch.equal(got[3], ref[3])  # (the sum of dy alone)


# Their sums of equal terms are rounded, unlike those of 7.0 or of any value in bf16.
VALUES = [0.1, -1e4 / 3, 7.7e-3, 123456.789, 1.0 + 2.0 ** -23, 1e-12, 1e15]


@pytest.mark.parametrize("C", WIDTHS)
def test_rows_of_one_value(C):
    B, T = 2, len(VALUES)
    x, dy, gamma, beta = _inputs(B, 2 * T, C, "f32")
    mixed = x.clone()  # rows of one value beside others
    for i, v in enumerate(VALUES):
        mixed[:, 2 * i] = v
    n = rn.LayerNorm(B, 2 * T, C, dtype="f32")
    ref, ref_dx = n.fwd(x, gamma, beta), n.bwd(x, dy, gamma)[0]
    y = n.fwd(mixed, gamma, beta)
    dx, dg, db = n.bwd(mixed, dy, gamma)
    assert torch.equal(y[:, ::2], beta.expand(B, T, C))  # no deviation: the offset alone
    assert torch.equal(y[:, 1::2], ref[:, 1::2]) and torch.equal(dx[:, 1::2], ref_dx[:, 1::2])
    # dx = rstd (a - mean(a)), xh being 0: within (64 + C / 256) u of the terms' sizes
    a = (gamma * dy[:, ::2]).double()
    rstd = 1e-5 ** -0.5
    size = rstd * (a.abs() + a.abs().mean(2, keepdim=True))
    err = (dx[:, ::2].double() - rstd * (a - a.mean(2, keepdim=True))).abs()
    assert torch.all(err <= (64 + C / 256) * 2.0 ** -24 * size)
    alone = rn.LayerNorm(B, T, C, dtype="f32")
    only = mixed[:, ::2].contiguous()
    assert torch.equal(alone.fwd(only, gamma, beta), beta.expand(B, T, C))
    assert not alone.bwd(only, torch.ones_like(only), gamma)[1].any()  # dgamma = sum dy xh


@pytest.mark.parametrize("C", WIDTHS)
def test_rows_of_one_value_without_eps_are_nan(C):
    T = len(VALUES)
    x = torch.tensor(VALUES, device="cuda")[None, :, None].expand(1, T, C).contiguous()
    n = rn.LayerNorm(1, T, C, dtype="f32", eps=0.0)
    assert torch.isnan(n.fwd(x)).all()
    assert torch.isnan(n.bwd(x, torch.ones_like(x))[0]).all()


@pytest.mark.parametrize("C", WIDTHS)
def test_rows_far_from_zero(C):
    # |mean| of 2^12 to 2^20 deviations (r).  The mean is held in fp32, half a step of itself off:
    # r u of the deviation, twice that with the step of its sum; a sum about it is k u of the
    # deviations off.  The deviation is as far off as the mean squared, and by its own sum.
    B, T, u = 1, 9, 2.0 ** -24
    g = torch.Generator().manual_seed(C)
    base = torch.randn(B, T, C, generator=g)
    shift = 2.0 ** torch.arange(12, 21).float()
    x = base + shift[None, :, None] * 1.1
    n = rn.LayerNorm(B, T, C, dtype="f32", eps=0.0)
    y = n.fwd(x.cuda()).double().cpu()
    xd = x.double()
    mean, dev = xd.mean(2, keepdim=True), xd.std(2, correction=0, keepdim=True)
    xh, r = (xd - mean) / dev, mean.abs() / dev
    k = 64 + C / 256
    bound = 2 * r * u + k * u + xh.abs() * ((2 * r * u) ** 2 + k * u + 2 * u)
    err = (y - xh).abs()
    assert torch.all(err <= bound), float((err / bound).max())


@pytest.mark.parametrize("C", WIDTHS + [12288, 100000])
def test_rows_of_one_bf16_value(C):
    T = len(VALUES)
    x = torch.tensor(VALUES, device="cuda").bfloat16()[None, :, None].expand(2, T, C).contiguous()
    beta = torch.randn(C, device="cuda")
    n = rn.LayerNorm(2, T, C, out_dtype="f32")
    assert torch.equal(n.fwd(x, None, beta), beta.expand(2, T, C))
    assert not n.bwd(x, torch.ones(2, T, C, device="cuda"))[1].any()
    assert torch.isnan(rn.LayerNorm(2, T, C, out_dtype="f32", eps=0.0).fwd(x)).all()


@pytest.mark.parametrize("C", [24, 333, 512, 2048, 9000])
def test_infinities_in_parameter_gradients(C):
    x, dy, gamma, _ = _inputs(2, 40, C, "f32")
    n = rn.LayerNorm(2, 40, C, dtype="f32")
    n.fwd(x, gamma)
    ref = n.bwd(x, dy, gamma)
    xh = (x.double() - x.double().mean(2, keepdim=True))[1, 7]
    bad = dy.clone()
    bad[1, 7, 3], bad[1, 7, 5] = float("inf"), -float("inf")
    bad[0, 2, 9], bad[1, 7, 9] = float("inf"), -float("inf")
    _, dg, db = n.bwd(x, bad, gamma)
    inf = float("inf")
    assert float(db[3]) == inf and float(db[5]) == -inf and torch.isnan(db[9])
    assert float(dg[3]) == inf * float(xh[3].sign()) and float(dg[5]) == -inf * float(xh[5].sign())
    other = torch.ones(C, dtype=torch.bool, device="cuda")
    other[[3, 5, 9]] = False
    assert torch.equal(db[other], ref[2][other]) and torch.equal(dg[other], ref[1][other])


@pytest.mark.parametrize("C", [1 << 20, (1 << 20) - 1])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_rows_of_one_value_of_the_greatest_width(C, dtype):
    # (bf16: with C past 2^16 a sum of equal values is rounded too)
    values = [0.1, -1e4 / 3, 1.0 + 2.0 ** -7, 123.456]
    x = torch.tensor(values, device="cuda").to(DT[dtype])[None, :, None].expand(1, 4, C)
    beta = torch.randn(C, device="cuda")
    n = rn.LayerNorm(1, 4, C, dtype=dtype, out_dtype="f32")
    assert torch.equal(n.fwd(x.contiguous(), None, beta), beta.expand(1, 4, C))
    assert not n.bwd(x.contiguous(), torch.ones(1, 4, C, device="cuda"))[1].any()
