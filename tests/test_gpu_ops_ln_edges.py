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
