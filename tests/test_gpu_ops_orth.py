"""Orthogonalised update against the same iteration in 64 bits (GPU).

Tolerances, relative 2-norm.  A step multiplies a small singular value by at most a = 3.4445, so
an error of the first step grows by at most a^5 = 485 in five.  fp32 output: products good to
2^-22 give at most 485 2^-22 = 1.2e-4.  bf16 output: 2^-8, twice the result's own rounding of
about 2^-9, which leaves as much for the products.
"""
import numpy as np
import pytest
import torch

import asr_tiled_tanh_gb300 as rn

pytestmark = pytest.mark.gpu
DT = {"f32": torch.float32, "bf16": torch.bfloat16}
A, B, C = 3.4445, -4.7750, 2.0315
TOL = {"f32": 485 * 2.0 ** -22, "bf16": 2.0 ** -8}


@pytest.fixture(scope="module", autouse=True)
def _lib():
    rn.load(build_if_missing=True)


def _ref(G, steps, eps=1e-7):
    G = G.double().cuda()
    X = G / (G.norm() + eps)
    t = X.shape[0] > X.shape[1]
    X = X.T if t else X
    for _ in range(steps):
        S = X @ X.T
        X = A * X + (B * S + C * S @ S) @ X
    return (X.T if t else X).cpu()


def _grad(R, K, seed, kind="noise"):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g)
    if kind == "noise":
        return r(R, K)
    if kind == "decay":  # singular values like 1 / i over three decades
        m = min(R, K)
        u, _ = torch.linalg.qr(r(R, m))
        v, _ = torch.linalg.qr(r(K, m))
        return (u / torch.arange(1, m + 1).float()) @ v.T
    k = max(1, min(R, K) // 16)
    return 1e-4 * (r(R, k) @ r(k, K) + 0.05 * r(R, K))  # a few strong directions


SHAPES = [(1, 1), (1, 40), (33, 1), (8, 8), (16, 200), (64, 64), (65, 130), (130, 63), (128, 256),
          (300, 200), (512, 512), (640, 640), (1000, 333), (257, 1025), (2048, 512), (96, 5000),
          (4100, 90), (1024, 1040)]


@pytest.mark.parametrize("R,K", SHAPES)
@pytest.mark.parametrize("idt,odt", [("f32", "f32"), ("f32", "bf16"), ("bf16", "bf16"),
                                     ("bf16", "f32")])
def test_iterate(R, K, idt, odt):
    G = _grad(R, K, R + K, "strong" if min(R, K) > 16 else "noise").to(DT[idt])
    o = rn.Orthogonalizer(R, K, dtype=idt, out_dtype=odt)
    got = o.run(G.cuda()).double().cpu()
    ref = _ref(G, 5)
    assert (got - ref).norm() <= TOL[odt] * ref.norm()
    assert o.status() == (0, 0)


@pytest.mark.parametrize("kind", ["noise", "decay", "strong"])
@pytest.mark.parametrize("R,K", [(256, 256), (1024, 200), (200, 640)])
@pytest.mark.parametrize("odt", ["f32", "bf16"])
def test_spectra(R, K, kind, odt):
    G = _grad(R, K, 3, kind)
    o = rn.Orthogonalizer(R, K, out_dtype=odt)
    got = o.run(G.cuda())
    ref = _ref(G, 5)
    assert (got.double().cpu() - ref).norm() <= TOL[odt] * ref.norm()
    if kind == "noise" and R != K:  # singular values that started near one another: all near 1
        s = torch.linalg.svdvals(got.double().cpu())
        assert s.min() > 0.6 and s.max() < 1.25


@pytest.mark.parametrize("steps", [1, 2, 3, 4, 7, 12])
@pytest.mark.parametrize("odt", ["f32", "bf16"])
def test_steps(steps, odt):
    G = _grad(192, 320, steps, "strong")
    got = rn.Orthogonalizer(192, 320, out_dtype=odt, steps=steps).run(G.cuda()).double().cpu()
    ref = _ref(G, steps)
    # (past five steps nothing grows any more: the singular values stay near 1)
    assert (got - ref).norm() <= TOL[odt] * ref.norm()


@pytest.mark.parametrize("R,K", [(72, 130), (300, 100)])
@pytest.mark.parametrize("idt,odt", [("f32", "bf16"), ("bf16", "f32")])
def test_batch_and_strides(R, K, idt, odt):
    N = 3
    G = torch.stack([_grad(R, K, 40 + i) * 10.0 ** (i - 1) for i in range(N)]).to(DT[idt])
    for ld in (K + 3, K + 8):
        ib, ob = R * ld + 5, R * ld + 16
        gbuf = torch.full((N * ib + 8,), float("nan"), dtype=DT[idt], device="cuda")
        obuf = torch.full((N * ob + 8,), 9.0, dtype=DT[odt], device="cuda")
        gv = gbuf.as_strided((N, R, K), (ib, ld, 1))
        ov = obuf.as_strided((N, R, K), (ob, ld, 1))
        gv.copy_(G)
        o = rn.Orthogonalizer(R, K, batch=N, dtype=idt, out_dtype=odt, in_strides=(ib, ld),
                              out_strides=(ob, ld))
        o.run(gv, out=ov)
        for i in range(N):
            ref = _ref(G[i], 5)
            assert (ov[i].double().cpu() - ref).norm() <= TOL[odt] * ref.norm()
        ov.fill_(9.0)
        assert torch.all(obuf == 9.0)


def test_scale_of_the_gradient_does_not_matter():
    G = _grad(100, 164, 5)
    o = rn.Orthogonalizer(100, 164, out_dtype="f32", eps=0.0)
    a = o.run(G.cuda()).clone()
    for s in (2.0 ** -60, 2.0 ** 60):
        b = o.run((G * s).cuda())
        assert (a - b).norm() <= 1e-5 * a.norm()


def test_zeros_and_wild_values():
    G = torch.stack([torch.zeros(40, 70), _grad(40, 70, 1), _grad(40, 70, 2), _grad(40, 70, 3)])
    ref = _ref(G[3], 5)
    G[1, 3, 4], G[2, 0, 0] = float("nan"), float("inf")
    for odt in ("f32", "bf16"):
        out = rn.Orthogonalizer(40, 70, batch=4, out_dtype=odt).run(G.cuda()).cpu()
        assert torch.all(out[0] == 0)
        assert torch.isnan(out[1].float()).all() and torch.isnan(out[2].float()).all()
        assert (out[3].double() - ref).norm() <= TOL[odt] * ref.norm()


def test_same_bits_another_stream_and_a_graph():
    G = _grad(384, 256, 8).cuda()
    o = rn.Orthogonalizer(384, 256)
    ref = o.run(G).clone()
    assert torch.equal(o.run(G), ref)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    out = o.run(G, stream=s)
    s.synchronize()
    assert torch.equal(out, ref)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        o.run(G, out=out)
    for _ in range(2):
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, ref)


# Thin matrices on one block, on clusters of 2 to 16, and on more blocks than a cluster takes.
@pytest.mark.parametrize("R,K", [(100, 128), (126, 142), (384, 128), (17, 500), (90, 700),
                                 (1100, 128), (33, 1408), (120, 1860), (2048, 128), (2049, 70)])
@pytest.mark.parametrize("N,odt", [(1, "f32"), (3, "bf16")])
def test_thin(R, K, N, odt):
    G = torch.stack([_grad(R, K, 7 * R + K + i, "strong") for i in range(N)])
    o = rn.Orthogonalizer(R, K, batch=N, out_dtype=odt)
    got = o.run(G.cuda()).double().cpu()
    again = o.run(G.cuda()).double().cpu()
    assert o.status() == (0, 0) and torch.equal(got, again)
    for i in range(N):
        ref = _ref(G[i], 5)
        assert (got[i] - ref).norm() <= TOL[odt] * ref.norm()


# Rows that end inside a warp: some of its lanes store nothing, in blocks of more than 64 columns
# between one read of tensor memory and the next.
@pytest.mark.parametrize("R,K", [(1, 128), (31, 96), (33, 65), (97, 127), (128, 40), (127, 100),
                                 (90, 17), (65, 230), (300, 97), (47, 2560)])
@pytest.mark.parametrize("odt", ["f32", "bf16"])
def test_thin_rows_inside_a_warp(R, K, odt):
    G = _grad(R, K, R * K, "noise")
    ld = K + 3
    buf = torch.full((R * ld,), 9.0, dtype=DT[odt], device="cuda")
    o = rn.Orthogonalizer(R, K, out_dtype=odt, out_strides=(R * ld, ld))
    out = buf.as_strided((R, K), (ld, 1))
    o.run(G.cuda(), out=out)
    ref = _ref(G, 5)
    assert (out.double().cpu() - ref).norm() <= TOL[odt] * ref.norm()
    out.fill_(9.0)
    assert torch.all(buf == 9.0) and o.status() == (0, 0)


# Entries over the whole of fp32's range, on every kernel: the squares of all but the middle ones
# leave it, and so does the norm of the largest.
@pytest.mark.parametrize("scale", [1e37, 1e25, 2e18, 1e-12, 1e-18, 3e-30])
@pytest.mark.parametrize("R,K", [(40, 70), (90, 700), (2049, 70), (300, 260)])
def test_entries_of_any_size(R, K, scale):
    G = _grad(R, K, R + K)  # (noise: 5 at most)
    G[3, 5] = 30.0  # the largest scale's largest entry: 3e38
    if scale < 1e-20:
        G[1:] *= 0.01
    G = G * scale
    for odt in ("f32", "bf16"):
        got = rn.Orthogonalizer(R, K, out_dtype=odt, eps=0.0).run(G.cuda()).double().cpu()
        ref = _ref(G, 5, eps=0.0)
        assert (got - ref).norm() <= TOL[odt] * ref.norm()


@pytest.mark.parametrize("R,K", [(40, 70), (300, 260)])
def test_zeros_whatever_eps(R, K):
    for eps in (0.0, 1e-45, 1e-7, 1.0):
        out = rn.Orthogonalizer(R, K, out_dtype="f32", eps=eps).run(torch.zeros(R, K).cuda())
        assert torch.all(out == 0)


def test_eps_counts_beside_the_norm():
    # |G| far below eps: X = G / eps at first, 485 times that in the end
    G = _grad(60, 90, 4) * 1e-9
    for eps in (1e-7, 1e-3):
        got = rn.Orthogonalizer(60, 90, out_dtype="f32", eps=eps).run(G.cuda()).double().cpu()
        ref = _ref(G, 5, eps=eps)
        # (22 bits at a fixed scale: 2^-38 of 1 is the least that X holds)
        assert (got - ref).norm() <= TOL["f32"] * ref.norm() + 485 * 2.0 ** -38 * 73.5
