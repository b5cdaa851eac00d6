"""Tensors that the operators' plans make for the caller belong to the call's stream (GPU).

Memory of the caching allocator is ordered on the stream it was asked for: a result made on
another stream than the one its kernel runs on may lie where that other stream still works.
"""
import pytest
import torch

import asr_tiled_tanh_gb300 as rn

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    rn.load(build_if_missing=True)


def _stream_of(t):
    """Stream of the allocator's segment that holds t."""
    at = t.data_ptr()
    for seg in torch.cuda.memory_snapshot():
        if seg["address"] <= at < seg["address"] + seg["total_size"]:
            return seg["stream"]
    raise AssertionError("not the allocator's memory")


def _calls(stream):
    """(results of every call with `stream`, results on the current stream)"""
    r = lambda *s: torch.randn(*s, device="cuda")
    ids = torch.randint(0, 7, (4, 9), dtype=torch.int32, device="cuda")
    x, G, table, dout = r(4, 9, 64), r(40, 70), r(7, 64), r(4, 9, 64)
    e = rn.LabelEmbedding(4, 9, 7, 64, dtype="f32", out_dtype="f32")
    n = rn.FrameNorm(4, 9, 64, 4, dtype="f32")
    o = rn.Orthogonalizer(40, 70)
    def run(**k):
        return [e.fwd(table, ids, **k), e.bwd(dout, ids, **k), n.fwd(x, **k), *n.bwd(x, dout, **k),
                o.run(G, **k)]
    ref = [t.clone() for t in run()]
    torch.cuda.synchronize()
    return run(stream=stream), ref


@pytest.mark.parametrize("handle", [False, True])
def test_results_belong_to_the_given_stream(handle):
    s = torch.cuda.Stream()
    got, ref = _calls(s.cuda_stream if handle else s)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, ref))
    assert [_stream_of(t) for t in got] == [s.cuda_stream] * len(got)


def test_results_belong_to_the_current_stream():
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got, ref = _calls(None)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, ref))
    assert [_stream_of(t) for t in got] == [s.cuda_stream] * len(got)
