"""A step whose gradients are not finite changes nothing in the training-step example (GPU)."""
import pytest
import torch

from tests.test_gpu_example import _example

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_a_bad_step_is_left_out_everywhere(bad):
    ex = _example()
    model = ex.Transducer(4, 40, 7, 128, 128, 64)
    frames, *rest = ex.batch(4, 40, 7, 128, 64)
    model.step(frames, *rest)
    state = lambda: [t.clone() for d in (model.matrices, model.others, model.velocity,  # noqa: E731
                                         model.low) for t in d.values()]
    before = state()
    worse = frames.clone()
    worse[1, 2, 3] = bad
    model.step(worse, *rest)
    assert all(torch.equal(a, b) for a, b in zip(state(), before))
    assert model.adamw.steps.tolist() == [1, 0]
    loss, _ = model.step(frames, *rest)
    assert bool(torch.isfinite(loss).all()) and model.adamw.steps.tolist() == [2, 0]
    assert all(bool(torch.isfinite(t.float()).all()) for t in state())
    assert not torch.equal(state()[0], before[0])
