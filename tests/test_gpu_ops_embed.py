"""Label embedding and its gradient against a plain 64-bit implementation (GPU).

Tolerances: a row is one fp32 product (2^-24 relative), and in bf16 exactly that product rounded
to nearest; a table gradient is a sum of n fp32 terms in some order, whose error
is at most (n + 2) 2^-24 times the sum of the terms' magnitudes.
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


def _inputs(B, U1, V, D, dtype, seed, ids="uniform", full=False):
    g = torch.Generator().manual_seed(seed)
    table = torch.randn(V, D, generator=g).to(DT[dtype])
    u = torch.rand(B, U1, generator=g, dtype=torch.float64)
    if ids == "same":
        i = torch.full((B, U1), V - 1)
    elif ids == "zipf":
        i = (torch.exp(u * np.log(V)) - 1).long().clamp(0, V - 1)
    else:
        i = (u * V).long().clamp(0, V - 1)
    U_len = torch.randint(0, U1, (B,), generator=g)
    U_len[0] = U1 - 1
    if full:
        U_len[:] = U1 - 1
    return table, i.to(torch.int32), U_len.to(torch.int32)


def _rows(i, U_len, V, sos, blank):
    """(label of every row, whether the row exists) on the host."""
    i = i.numpy().astype(np.int64).copy()
    if sos:
        i[:, 0] = blank
    here = np.arange(i.shape[1])[None] <= U_len.numpy()[:, None]
    return i, here


FWD = [(1, 1, 1, 1), (1, 1, 7, 512), (8, 1, 1024, 512), (3, 5, 11, 33), (4, 51, 300, 640),
       (2, 7, 9, 8), (5, 3, 4, 1000), (64, 101, 513, 72)]


@pytest.mark.parametrize("B,U1,V,D", FWD)
@pytest.mark.parametrize("tdt,rdt", [("f32", "f32"), ("f32", "bf16"), ("bf16", "f32"),
                                     ("bf16", "bf16")])
@pytest.mark.parametrize("sos", [True, False])
def test_rows(B, U1, V, D, tdt, rdt, sos):
    table, i, U_len = _inputs(B, U1, V, D, tdt, B + U1 + D)
    blank, scale = V // 2, 1.7
    e = rn.LabelEmbedding(B, U1, V, D, dtype=tdt, out_dtype=rdt, scale=scale, sos=sos, blank=blank)
    dev = i.clone()
    if sos:
        dev[:, 0] = -5  # never read
    dev[torch.arange(U1)[None] > U_len[:, None]] = 1 << 30  # rows that do not exist
    if sos:
        dev[:, 0] = -5
    out = e.fwd(table.cuda(), dev.cuda(), U_len.cuda())
    lab, here = _rows(i, U_len, V, sos, blank)
    ref = table.double().numpy()[lab] * float(np.float32(scale)) * here[..., None]
    got = out.double().cpu().numpy()
    if rdt == "f32":
        assert np.all(np.abs(got - ref) <= U32 * np.abs(ref))
    else:
        one = (table[torch.from_numpy(lab)].float() * scale).to(torch.bfloat16).double().numpy()
        assert np.array_equal(got, one * here[..., None])
    assert e.status() == (0, 0)


@pytest.mark.parametrize("rdt,ld", [("bf16", 40), ("f32", 41), ("bf16", 37)])
def test_strides_leave_the_gaps_alone(rdt, ld):
    B, U1, V, D = 3, 9, 20, 33
    table, i, U_len = _inputs(B, U1, V, D, "bf16", 5)
    buf = torch.full((B * U1 * ld,), 7.0, dtype=DT[rdt], device="cuda")
    out = buf.as_strided((B, U1, D), (U1 * ld, ld, 1))
    wide = torch.full((V, 50), float("nan"), dtype=torch.bfloat16)
    wide[:, :D] = table
    e = rn.LabelEmbedding(B, U1, V, D, out_dtype=rdt, sos=False, ld_table=50, ld_rows=ld)
    e.fwd(wide.cuda()[:, :D], i.cuda(), U_len.cuda(), out=out)
    lab, here = _rows(i, U_len, V, False, 0)
    ref = table.double().numpy()[lab] * here[..., None]
    assert np.array_equal(out.double().cpu().numpy(), ref)
    gaps = buf.view(B * U1, ld)[:, D:]
    assert torch.all(gaps == 7.0)
    # and the gradient, from strided rows into a strided table
    dt = torch.full((V * 50,), 7.0, device="cuda")
    buf.normal_()
    e.bwd(out, i.cuda(), U_len.cuda(), dtable=dt.as_strided((V, D), (50, 1)))
    assert torch.all(dt.view(V, 50)[:, D:] == 7.0)
    _check_grad(dt.view(V, 50)[:, :D], out, lab, here, V, 1.0)


def _check_grad(got, dout, lab, here, V, scale):
    d = dout.double().cpu().numpy() * float(np.float32(scale))
    ref, mag = np.zeros((V, d.shape[-1])), np.zeros((V, d.shape[-1]))
    n = np.bincount(lab[here], minlength=V)
    np.add.at(ref, lab[here], d[here])
    np.add.at(mag, lab[here], np.abs(d[here]))
    err = np.abs(got.double().cpu().numpy() - ref)
    assert np.all(err <= (n[:, None] + 2) * U32 * mag)


BWD = [(1, 1, 1, 1, "uniform"), (1, 1, 300, 512, "uniform"), (3, 5, 11, 33, "uniform"),
       (8, 51, 1024, 512, "uniform"), (16, 81, 5000, 200, "zipf"), (64, 101, 513, 72, "zipf"),
       (300, 101, 40, 64, "same"), (257, 33, 70000, 24, "zipf"), (1, 4097, 3, 40, "uniform"),
       (1024, 101, 2048, 16, "uniform"), (7, 129, 1, 1000, "same"), (200, 65, 65536, 8, "uniform"),
       (2500, 101, 17, 8, "zipf")]


@pytest.mark.parametrize("B,U1,V,D,ids", BWD)
@pytest.mark.parametrize("rdt,sos", [("f32", True), ("bf16", False)])
def test_table_gradient(B, U1, V, D, ids, rdt, sos):
    _, i, U_len = _inputs(B, U1, V, 1, "f32", B + U1 + D, ids)
    blank, scale = V // 3, 0.6
    g = torch.Generator().manual_seed(9)
    dout = torch.randn(B, U1, D, generator=g).to(DT[rdt])
    gone = torch.arange(U1)[None] > U_len[:, None]
    dev, di = dout.clone(), i.clone()
    dev[gone] = float("nan")  # rows that do not exist are never read
    di[gone] = -3
    if sos:
        di[:, 0] = V + 1
    e = rn.LabelEmbedding(B, U1, V, D, out_dtype=rdt, scale=scale, sos=sos, blank=blank)
    args = (dev.cuda(), di.cuda(), U_len.cuda())
    dt = torch.full((V, D), float("nan"), device="cuda")
    e.bwd(*args, dtable=dt)
    lab, here = _rows(i, U_len, V, sos, blank)
    _check_grad(dt, dout, lab, here, V, scale)
    assert e.status() == (0, 0)
    assert torch.equal(e.bwd(*args), dt)  # the same bits again


def test_no_rows_give_a_zero_table():
    e = rn.LabelEmbedding(0, 3, 6, 16)
    dt = e.bwd(torch.empty(0, 3, 16, dtype=torch.bfloat16, device="cuda"),
               torch.empty(0, 3, dtype=torch.int32, device="cuda"))
    assert torch.all(dt == 0)


def test_bad_labels_and_lengths_are_reported_and_left_out():
    B, U1, V, D = 4, 6, 9, 16
    table, i, _ = _inputs(B, U1, V, D, "f32", 3)
    i[1, 2], i[2, 3] = V, -1
    ul = torch.tensor([5, 5, 5, 6], dtype=torch.int32)
    e = rn.LabelEmbedding(B, U1, V, D, dtype="f32", out_dtype="f32", sos=False)
    out = e.fwd(table.cuda(), i.cuda(), ul.cuda()).cpu()
    assert torch.all(out[1, 2] == 0) and torch.all(out[2, 3] == 0) and torch.all(out[3] == 0)
    assert torch.equal(out[0], table[i[0].long()])
    code, word = e.status()
    assert code == 4 and word == (1 << 4) | (1 << 5)  # LENGTH_RANGE first, both bits
    d = torch.randn(B, U1, D)
    lab = i.numpy().astype(np.int64)
    here = np.ones((B, U1), bool)
    here[3], here[1, 2], here[2, 3] = False, False, False
    dt = e.bwd(d.cuda(), i.cuda(), ul.cuda())
    _check_grad(dt, d, np.where(here, lab, 0), here, V, 1.0)


def test_gradient_is_the_derivative():
    # <dE, P> is the difference quotient of sum(hL * R) along P (the map is linear: no step error)
    B, U1, V, D = 3, 7, 12, 24
    table, i, U_len = _inputs(B, U1, V, D, "f32", 21)
    P, R = torch.randn(V, D), torch.randn(B, U1, D)
    e = rn.LabelEmbedding(B, U1, V, D, dtype="f32", out_dtype="f32", scale=2.0)
    dt = e.bwd(R.cuda(), i.cuda(), U_len.cuda()).double().cpu()
    lab, here = _rows(i, U_len, V, True, 0)
    f = lambda E: float((E.double().numpy()[lab] * 2.0 * here[..., None] * R.double().numpy()).sum())
    diff = (f(table + P) - f(table - P)) / 2
    assert abs(float((dt * P).sum()) - diff) <= 1e-5 * float((dt * P).abs().sum())


def test_another_stream_and_a_graph():
    B, U1, V, D = 16, 20, 50, 64
    table, i, U_len = (t.cuda() for t in _inputs(B, U1, V, D, "f32", 2))
    e = rn.LabelEmbedding(B, U1, V, D, dtype="f32", out_dtype="f32")
    d = torch.randn(B, U1, D, device="cuda")
    ref, dref = e.fwd(table, i, U_len).clone(), e.bwd(d, i, U_len).clone()
    out, dt = torch.zeros_like(ref), torch.zeros_like(dref)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        e.fwd(table, i, U_len, out=out)
    e.bwd(d, i, U_len, dtable=dt, stream=s)
    s.synchronize()
    assert torch.equal(out, ref) and torch.equal(dt, dref)
    out.zero_(), dt.zero_()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        e.fwd(table, i, U_len, out=out)
        e.bwd(d, i, U_len, dtable=dt)
    for _ in range(2):
        out.zero_(), dt.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, ref) and torch.equal(dt, dref)


@pytest.mark.parametrize("D", [64, 50, 33])
def test_runs_over_many_chunks_are_this_calls(D):
    # one label in every row: its sum is joined from the partial rows of all chunks, which lie
    # at the same addresses in call after call
    B, U1, V = 64, 101, 5
    _, i, _ = _inputs(B, U1, V, 1, "f32", 1, "same")
    i, e = i.cuda(), rn.LabelEmbedding(B, U1, V, D, out_dtype="f32", sos=False)
    lab, here = _rows(i.cpu(), torch.full((B,), U1 - 1), V, False, 0)
    ds = [torch.randn(B, U1, D, device="cuda") * 4.0 ** k for k in range(6)]
    got = [e.bwd(d, i) for d in ds]  # back to back
    for d, g in zip(ds, got):
        _check_grad(g, d, lab, here, V, 1.0)


# Four rows in flight a lane: from 64 rows per SM on and warp's rows at a time (1, 2 or 4 of them), in
# vectors of 8, 2 and 1 elements; the last warp's rows are fewer than it takes.
@pytest.mark.parametrize("D", [160, 96, 40, 42, 26, 10, 33, 11, 5])
@pytest.mark.parametrize("tdt,rdt", [("f32", "f32"), ("f32", "bf16"), ("bf16", "f32"),
                                     ("bf16", "bf16")])
def test_many_rows(D, tdt, rdt):
    B, U1, V, scale = 397, 101, 700, 1.7
    vec = next(v for v in (8, 2, 1) if D % v == 0)
    per = 1 if D // vec > 16 else 2 if D // vec > 8 else 4
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    assert B * U1 >= 64 * sms * per and B * U1 % (4 * per)
    table, i, U_len = (t.cuda() for t in _inputs(B, U1, V, D, tdt, D))
    e = rn.LabelEmbedding(B, U1, V, D, dtype=tdt, out_dtype=rdt, scale=scale, sos=True, blank=3)
    dev = i.clone()
    dev[:, 0] = -5  # never read
    gone = torch.arange(U1, device="cuda")[None] > U_len[:, None]
    dev[gone] = 1 << 30
    buf = torch.full((B * U1 * D + 64,), 9.0, dtype=DT[rdt], device="cuda")
    out = e.fwd(table, dev, U_len, out=buf[:-64].view(B, U1, D))
    i[:, 0] = 3
    s32 = torch.tensor(scale, dtype=torch.float32, device="cuda")  # exact in 64 bits, one rounding
    ref = (table.double()[i.long()] * s32.double()).float().to(DT[rdt]) * ~gone[..., None]
    assert torch.equal(out, ref) and torch.all(buf[-64:] == 9.0)
    assert e.status() == (0, 0)
