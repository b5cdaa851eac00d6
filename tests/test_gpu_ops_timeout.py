"""The orthogonalised update's bounded waits, without a fault (GPU).

A test hook leaves out one block's arrival at the grid barrier. Every other wait then runs out
too: the kernel has to record RNNT_ERR_TIMEOUT, wind down and return, and the next call on the
same plan has to give the right result.
"""
import ctypes
import time

import pytest
import torch

import asr_tiled_tanh_gb300 as rn
from asr_tiled_tanh_gb300 import ops

from .test_gpu_ops_orth import DT, TOL, _grad, _ref

TIMEOUT = 6


@pytest.fixture(scope="module", autouse=True)
def _lib():
    rn.load(build_if_missing=True)


def _timeout(dims, G, out, ws, nbytes, status, ns):
    return rn.load().rnnt_testing_orth_timeout(ctypes.byref(dims), G, out, ws, nbytes, status, ns,
                                               None)


def test_the_hook_is_for_blocks_that_meet():
    for R, K in ((64, 64), (100, 2000)):  # one block; a cluster
        d = ops.RnntOrthDims(R, K, 1, 0, 0, 5, 1e-7)
        assert _timeout(d, 4096, 4096, 4096, 1 << 40, None, 1) == 1


@pytest.mark.gpu
@pytest.mark.parametrize("R,K,N,odt", [(300, 300, 1, "bf16"), (640, 640, 2, "bf16"),
                                       (512, 1500, 1, "f32"), (2500, 2500, 1, "bf16"),
                                       (120, 2200, 2, "f32")])
def test_a_lost_arrival_is_reported(R, K, N, odt):
    G = torch.stack([_grad(R, K, i) for i in range(N)]).cuda()
    o = rn.Orthogonalizer(R, K, batch=N, out_dtype=odt)
    out = torch.zeros(N, R, K, dtype=DT[odt], device="cuda")
    torch.cuda.synchronize()
    t0 = time.perf_counter()
    assert _timeout(o.dims, G.data_ptr(), out.data_ptr(), o.ws.data_ptr(), o.ws_bytes,
                    o.status_word.data_ptr(), 50_000_000) == 0
    torch.cuda.synchronize()
    assert time.perf_counter() - t0 < 10.0
    assert o.status() == (TIMEOUT, 1 << TIMEOUT)
    o.status_word.zero_()
    got = o.run(G).double().cpu()
    assert o.status() == (0, 0)
    for i in range(N):
        ref = _ref(G[i], 5)
        assert (got[i] - ref).norm() <= TOL[odt] * ref.norm()
