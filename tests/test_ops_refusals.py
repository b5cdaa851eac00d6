"""What the operators of include/rnnt_ops.h refuse on the host, before any launch (CPU).

Addresses are fake and never dereferenced.
"""
import ctypes

import pytest

import asr_tiled_tanh_gb300 as rn
from asr_tiled_tanh_gb300 import build
from asr_tiled_tanh_gb300.ops import RnntEmbedDims, RnntNormDims, RnntOrthDims

INVALID, WS = 1, 3


@pytest.fixture(scope="module")
def lib():
    build.build_library()
    return rn.load()


EMBED = dict(B=2, U1=3, V=7, D=16, blank=0, sos=1, table_dtype=1, row_dtype=1, scale=1.0,
             ld_table=0, ld_rows=0)
NORM = dict(B=2, T=5, C=16, G=4, act=1, dtype=1, eps=1e-5, x_frame=0, x_batch=0, y_frame=0,
            y_batch=0)
ORTH = dict(rows=8, cols=16, batch=1, in_dtype=0, out_dtype=1, steps=5, eps=1e-7, in_ld=0,
            in_batch=0, out_ld=0, out_batch=0)


@pytest.mark.parametrize("bad", [dict(B=-1), dict(U1=0), dict(V=0), dict(D=0), dict(blank=7),
                                 dict(blank=-1), dict(table_dtype=2), dict(row_dtype=3),
                                 dict(ld_table=15), dict(ld_rows=-1), dict(B=1 << 20, U1=1 << 11),
                                 dict(scale=float("inf")), dict(scale=float("nan"))])
def test_embed_dims(lib, bad):
    d = RnntEmbedDims(**{**EMBED, **bad})
    assert lib.rnnt_embed_workspace_bytes(ctypes.byref(d)) == 0
    assert lib.rnnt_embed_fwd(ctypes.byref(d), 256, 256, 256, 256, None, None) == INVALID
    assert lib.rnnt_embed_bwd(ctypes.byref(d), 256, 256, 256, 256, 256, 1 << 40, None,
                              None) == INVALID


@pytest.mark.parametrize("bad", [dict(B=-1), dict(T=0), dict(C=0), dict(G=0), dict(G=3),
                                 dict(act=3), dict(act=-1), dict(dtype=2), dict(eps=-1.0),
                                 dict(eps=float("nan")), dict(x_frame=15), dict(y_frame=8),
                                 dict(x_batch=79), dict(y_batch=16), dict(T=(1 << 20) + 1)])
def test_norm_dims(lib, bad):
    d = RnntNormDims(**{**NORM, **bad})
    assert lib.rnnt_norm_workspace_bytes(ctypes.byref(d)) == 0
    assert lib.rnnt_norm_saved_bytes(ctypes.byref(d)) == 0
    p = [256] * 7
    assert lib.rnnt_norm_fwd(ctypes.byref(d), *p, 1 << 40, None, None) == INVALID
    p = [256] * 10
    assert lib.rnnt_norm_bwd(ctypes.byref(d), *p, 1 << 40, None, None) == INVALID


@pytest.mark.parametrize("bad", [dict(rows=0), dict(cols=-2), dict(batch=-1), dict(in_dtype=2),
                                 dict(out_dtype=5), dict(steps=0), dict(steps=33), dict(eps=-1e-7),
                                 dict(in_ld=15), dict(out_ld=3), dict(batch=2, out_batch=100),
                                 dict(rows=1 << 16, cols=1 << 15), dict(batch=1 << 16)])
def test_orth_dims(lib, bad):
    d = RnntOrthDims(**{**ORTH, **bad})
    assert lib.rnnt_orth_workspace_bytes(ctypes.byref(d)) == 0
    assert lib.rnnt_orth(ctypes.byref(d), 256, 256, 256, 1 << 40, None, None) == INVALID


def _each(lib, fn, dims, names, pos, ws_bytes, required, misaligned):
    """Every required pointer NULL, every pointer off its alignment, a short workspace."""
    base = {n: 0x10000 * (i + 1) for i, n in enumerate(names)}

    def call(a, nws):
        args = [a[n] for n in names]
        args[pos:pos] = []
        out = []
        for n in names:
            out.append(a[n])
            if n == "ws":
                out.append(nws)
        return fn(ctypes.byref(dims), *out, None)

    for n in required:
        assert call({**base, n: None}, ws_bytes) == INVALID, n
    for n, by in misaligned.items():
        assert call({**base, n: base[n] + by}, ws_bytes) == INVALID, n
    if "ws" in names:
        assert call(base, ws_bytes - 1) == WS


def test_embed_pointers(lib):
    d = RnntEmbedDims(**EMBED)
    n = lib.rnnt_embed_workspace_bytes(ctypes.byref(d))
    _each(lib, lib.rnnt_embed_fwd, d, ("ids", "U_len", "table", "rows", "status"), 0, 0,
          ("ids", "table", "rows"), dict(ids=2, U_len=1, table=1, rows=1, status=2))
    _each(lib, lib.rnnt_embed_bwd, d, ("ids", "U_len", "drows", "dtable", "ws", "status"), 0, n,
          ("ids", "drows", "dtable", "ws"),
          dict(ids=2, U_len=1, drows=1, dtable=2, ws=128, status=2))


def test_norm_pointers(lib):
    d = RnntNormDims(**NORM)
    n = lib.rnnt_norm_workspace_bytes(ctypes.byref(d))
    _each(lib, lib.rnnt_norm_fwd, d, ("x", "gamma", "beta", "T_len", "y", "saved", "ws", "status"),
          0, n, ("x", "y", "saved", "ws"),
          dict(x=1, gamma=2, beta=2, T_len=2, y=1, saved=64, ws=16, status=1))
    _each(lib, lib.rnnt_norm_bwd, d,
          ("x", "dy", "gamma", "beta", "T_len", "saved", "dx", "dgamma", "dbeta", "ws", "status"),
          0, n, ("x", "dy", "saved", "dx", "ws"),
          dict(x=1, dy=1, gamma=2, beta=2, T_len=2, saved=64, dx=1, dgamma=2, dbeta=1, ws=16,
               status=1))


def test_orth_pointers(lib):
    d = RnntOrthDims(**ORTH)
    n = lib.rnnt_orth_workspace_bytes(ctypes.byref(d))
    _each(lib, lib.rnnt_orth, d, ("G", "O", "ws", "status"), 0, n, ("G", "O", "ws"),
          dict(G=2, O=1, ws=8, status=2))


def test_null_dims(lib):
    assert lib.rnnt_embed_workspace_bytes(None) == 0
    assert lib.rnnt_norm_saved_bytes(None) == 0
    assert lib.rnnt_orth_workspace_bytes(None) == 0
    assert lib.rnnt_orth(None, 256, 256, 256, 1 << 30, None, None) == INVALID
    assert lib.rnnt_ops_status(None, None, None) == INVALID


def test_names(lib):
    with pytest.raises(ValueError):
        rn.LabelEmbedding(1, 1, 1, 1, dtype="f16", device="cpu")
    with pytest.raises(ValueError):
        rn.FrameNorm(1, 1, 1, 1, act="gelu", device="cpu")
    with pytest.raises(ValueError):
        rn.Orthogonalizer(1, 1, out_dtype="e4m3", device="cpu")
    with pytest.raises(rn.RnntError):
        rn.FrameNorm(1, 1, 10, 3, device="cpu")


def test_tensors_of_another_type_or_layout_are_refused(lib):
    import torch
    o = rn.Orthogonalizer(4, 6, device="cpu")
    with pytest.raises(ValueError):  # not a CUDA tensor
        o.run(torch.zeros(4, 6))
    e = rn.LabelEmbedding(1, 2, 3, 8, device="cpu")
    with pytest.raises(ValueError):
        e.fwd(torch.zeros(3, 8), torch.zeros(1, 2, dtype=torch.int64))
