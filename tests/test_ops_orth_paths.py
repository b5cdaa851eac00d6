"""Each path of the orthogonalised update's dispatch, named by what is planned for its size.

The plans are checked on the CPU, the results on the GPU against the same iteration in 64 bits, at
the tolerances of test_gpu_ops_orth.py: fp32 output 485 2^-22, bf16 output 2^-8.
"""
import pytest
import torch

import asr_tiled_tanh_gb300 as rn
from asr_tiled_tanh_gb300 import build, ops

from .test_gpu_ops_orth import DT, TOL, _grad, _ref


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build_library()
    rn.load()


SMS = 152  # the plan is for this many, whatever the device

# rows, cols, batch, output: K ranges of the Gram matrix, tile widths (gram, poly, update), update
# tiles in halves, products of more tiles than SMs (so that a block takes a second one)
PATHS = {
    (2500, 2500, 1, "bf16"): (1, (128, 128, 256), 48, "gpu"),
    (2777, 1403, 1, "bf16"): (2, (128, 64, 256), 0, ""),
    (1003, 2501, 1, "bf16"): (4, (128, 64, 256), 0, ""),
    (6000, 900, 1, "bf16"): (4, (128, 64, 256), 36, "u"),
    (900, 6003, 1, "bf16"): (4, (128, 64, 128), 72, "u"),
    (1403, 2777, 2, "bf16"): (1, (128, 128, 256), 0, "u"),
    (2200, 1100, 2, "bf16"): (1, (128, 128, 128), 20, "u"),
    (1000, 1000, 2, "bf16"): (2, (128, 64, 128), 0, ""),
    (640, 640, 2, "bf16"): (1, (64, 64, 64), 0, ""),
    (300, 300, 3, "bf16"): (1, (64, 64, 64), 0, ""),
    (4096, 512, 1, "f32"): (8, (128, 64, 128), 0, ""),
    (2000, 2000, 4, "f32"): (1, (128, 128, 128), 0, "gpu"),
    (1712, 1535, 2, "f32"): (1, (128, 128, 128), 32, "gpu"),
    (5200, 1003, 1, "f32"): (4, (128, 64, 128), 24, "u"),
    (1315, 3923, 1, "f32"): (2, (128, 64, 128), 37, "u"),
    (150, 9000, 4, "bf16"): (12, (128, 64, 128), 0, "u"),
    (129, 130, 50, "bf16"): (1, (128, 128, 64), 0, "u"),
    (300, 260, 8, "f32"): (1, (64, 64, 64), 0, ""),
}


def _planned(R, K, N, odt):
    p = ops.rnnt_testing_orth_plan(ops.RnntOrthDims(R, K, N, 0, int(odt == "bf16"), 5, 1e-7))
    more = "".join(c for c, u in zip("gpu", p.units) if u > SMS)
    assert p.thin == 0 and bool(p.exact) == (odt == "f32" or min(R, K) <= 256)
    return p.splits, tuple(p.bn), p.halved, more


@pytest.mark.parametrize("size", PATHS)
def test_the_plan_is_the_one_named(size):
    assert _planned(*size) == PATHS[size]


def test_every_width_is_named():
    assert {p[1][2] for s, p in PATHS.items() if s[3] == "bf16"} == {64, 128, 256}
    assert {p[1][2] for s, p in PATHS.items() if s[3] == "f32"} == {64, 128}
    assert {(p[1][0], p[0] > 1) for p in PATHS.values()} == {(64, False), (128, False), (128, True)}
    assert {p[1][1] for p in PATHS.values()} == {64, 128}


@pytest.mark.gpu
@pytest.mark.parametrize("size", PATHS)
def test_iterate(size):
    R, K, N, odt = size
    assert _planned(*size) == PATHS[size]
    G = torch.stack([_grad(R, K, R + K + i, "strong") for i in range(N)]).cuda()
    o = rn.Orthogonalizer(R, K, batch=N, out_dtype=odt)
    got = o.run(G)
    assert torch.equal(got, o.run(G)) and o.status() == (0, 0)
    for i in sorted({0, 1, N // 2, N - 1} & set(range(N))):
        ref = _ref(G[i], 5)
        assert (got[i].double().cpu() - ref).norm() <= TOL[odt] * ref.norm()


# Batches of strided matrices in and out: rows that are 16-byte aligned and rows that are not.
@pytest.mark.gpu
@pytest.mark.parametrize("R,K", [(300, 264), (264, 320), (2500, 1100)])
@pytest.mark.parametrize("idt,odt", [("f32", "bf16"), ("bf16", "f32"), ("f32", "f32")])
@pytest.mark.parametrize("gap", [3, 8])
def test_batch_and_strides(R, K, idt, odt, gap):
    N, ld = 3, K + gap
    ib, ob = R * ld + (5 if gap % 8 else 8), R * ld + 16
    G = torch.stack([_grad(R, K, 40 + i) * 10.0 ** (i - 1) for i in range(N)]).to(DT[idt])
    gbuf = torch.full((N * ib + 8,), float("nan"), dtype=DT[idt], device="cuda")
    obuf = torch.full((N * ob + 8,), 9.0, dtype=DT[odt], device="cuda")
    gv = gbuf.as_strided((N, R, K), (ib, ld, 1))
    ov = obuf.as_strided((N, R, K), (ob, ld, 1))
    gv.copy_(G)
    o = rn.Orthogonalizer(R, K, batch=N, dtype=idt, out_dtype=odt, in_strides=(ib, ld),
                          out_strides=(ob, ld))
    assert ops.rnnt_testing_orth_plan(o.dims).thin == 0
    o.run(gv, out=ov)
    assert o.status() == (0, 0)
    for i in range(N):
        ref = _ref(G[i], 5)
        assert (ov[i].double().cpu() - ref).norm() <= TOL[odt] * ref.norm()
    ov.fill_(9.0)
    assert torch.all(obuf == 9.0)


# One matrix of a batch that is all zeros, or holds a NaN: the others keep their results.
@pytest.mark.gpu
@pytest.mark.parametrize("odt", ["f32", "bf16"])
def test_matrices_of_a_batch_keep_to_themselves(odt):
    R, K = 300, 270
    G = torch.stack([_grad(R, K, i) for i in range(4)])
    ref = {i: _ref(G[i], 5) for i in (0, 3)}
    G[1] = 0
    G[2, 7, 9] = float("nan")
    out = rn.Orthogonalizer(R, K, batch=4, out_dtype=odt).run(G.cuda()).cpu()
    assert torch.all(out[1] == 0) and torch.isnan(out[2].float()).all()
    for i, r in ref.items():
        assert (out[i].double() - r).norm() <= TOL[odt] * r.norm()


# Products of one term (bf16 output, more than 256 rows and columns) over spectra and steps.
def _spectrum(R, K, kind):
    m, g = min(R, K), torch.Generator().manual_seed(R + K)
    i = torch.arange(1, m + 1, dtype=torch.float64)
    s = {"flat": torch.ones(m, dtype=torch.float64), "decay": 1 / i, "steep": i ** -2.0,
         "few": torch.where(i <= 3, 1.0, 1e-3), "one": torch.where(i <= 1, 1.0, 0.0)}[kind]
    u, _ = torch.linalg.qr(torch.randn(R, m, generator=g, dtype=torch.float64))
    v, _ = torch.linalg.qr(torch.randn(K, m, generator=g, dtype=torch.float64))
    return ((u * s) @ v.T).float()


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["flat", "decay", "steep", "few", "one"])
@pytest.mark.parametrize("R,K", [(300, 500), (640, 640), (1300, 400)])
def test_one_term_products_over_spectra(R, K, kind):
    G = _spectrum(R, K, kind)
    o = rn.Orthogonalizer(R, K, out_dtype="bf16")
    assert not ops.rnnt_testing_orth_plan(o.dims).exact
    ref = _ref(G, 5)
    assert (o.run(G.cuda()).double().cpu() - ref).norm() <= TOL["bf16"] * ref.norm()


# (past five steps the products take three terms: small singular values, and their errors, go on
# growing by 3.4445 a step)
@pytest.mark.gpu
@pytest.mark.parametrize("steps", [1, 2, 3, 4, 6, 8, 12, 32])
@pytest.mark.parametrize("kind", ["noise", "strong"])
def test_bf16_results_over_steps(steps, kind):
    R, K = 320, 500
    G = _grad(R, K, steps, kind)
    o = rn.Orthogonalizer(R, K, out_dtype="bf16", steps=steps)
    assert bool(ops.rnnt_testing_orth_plan(o.dims).exact) == (steps > 5)
    ref = _ref(G, steps)
    assert (o.run(G.cuda()).double().cpu() - ref).norm() <= TOL["bf16"] * ref.norm()


@pytest.mark.gpu
@pytest.mark.parametrize("steps", [6, 7, 8, 10])
@pytest.mark.parametrize("kind", ["flat", "decay", "steep"])
def test_bf16_results_of_more_steps_over_spectra(steps, kind):
    R, K = 640, 640
    G = _spectrum(R, K, kind)
    ref = _ref(G, steps)
    got = rn.Orthogonalizer(R, K, out_dtype="bf16", steps=steps).run(G.cuda()).double().cpu()
    assert (got - ref).norm() <= TOL["bf16"] * ref.norm()
