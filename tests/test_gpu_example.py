"""The training-step example runs the operators together and its loss falls (GPU)."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _example():
    spec = importlib.util.spec_from_file_location(
        "training_step", os.path.join(ROOT, "examples", "training_step.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def test_loss_falls():
    losses = _example().main(steps=20)
    # the batch is fixed and its frames name the labels: twenty steps learn much of it
    assert losses[-1] < 0.6 * losses[0], losses


def test_frame_gradient_is_the_loss_derivative():
    # along the returned gradient the loss rises by its squared norm (bf16 activations: 10%)
    ex = _example()
    model = ex.Transducer(4, 40, 7, 128, 128, 64, lr=0.0)
    frames, labels, T_len, U_len = ex.batch(4, 40, 7, 128, 64)
    loss, d = model.step(frames, labels, T_len, U_len)
    d = d.float()
    h = 2.0 / d.norm()  # a step of 2 in frames whose rounding is 2^-9 of about 1 each
    up = (frames.float() + h * d).bfloat16()
    down = (frames.float() - h * d).bfloat16()
    diff = (model.step(up, labels, T_len, U_len)[0].double().sum()
            - model.step(down, labels, T_len, U_len)[0].double().sum())
    moved = ((up.float() - down.float()) * d).double().sum()  # after the rounding to bf16
    assert abs(diff - moved) <= 0.1 * moved
