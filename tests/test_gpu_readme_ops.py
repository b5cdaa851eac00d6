"""The README's training-step example runs as written (GPU): both code blocks are executed with
a small synthetic batch bound to the names they use."""
import os
import re

import pytest
import torch

from asr_tiled_tanh_gb300 import synthetic
from tests.helpers import to_device

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_readme_training_step_runs():
    text = open(os.path.join(ROOT, "README.md")).read()
    blocks = re.findall(r"```python\n(.*?)```", text, flags=re.S)
    assert len(blocks) >= 2
    inp = synthetic.custom(B=3, T=40, U=6, HA=64, HL=64, H=64, V=128, dtype="bf16", seed=5)
    ns = dict(B=3, T=40, U=6, HA=64, HL=64, H=64, V=128, groups=8, **to_device(inp))
    ns["frames"] = torch.randn(3, 40, 64, device="cuda").bfloat16()
    ns["gamma"], ns["beta"] = torch.ones(64, device="cuda"), torch.zeros(64, device="cuda")
    ns["table"] = torch.randn(128, 64, device="cuda").bfloat16() / 8
    for block in blocks[:2]:
        exec(compile(block, "README.md", "exec"), ns)
    torch.cuda.synchronize()
    assert ns["dframes"].shape == (3, 40, 64) and ns["dtable"].shape == (128, 64)
    assert bool(torch.isfinite(ns["loss"]).all()) and bool(torch.isfinite(ns["dtable"]).all())
    s = torch.linalg.svdvals(ns["update"].float())
    assert s.max() < 1.25  # a gradient of low rank keeps its zero singular values
    assert all(ns[k].status() == (0, 0) for k in ("r", "norm", "embed", "orth"))
