"""The README's blocks run one after another as written (GPU), on a small synthetic batch bound to
the names that they use; the last one updates the weights."""
import os
import re

import pytest
import torch

from asr_tiled_tanh_gb300 import synthetic
from tests.helpers import to_device

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_every_block_runs():
    text = open(os.path.join(ROOT, "README.md")).read()
    blocks = re.findall(r"```python\n(.*?)```", text, flags=re.S)
    assert len(blocks) == 3
    inp = synthetic.custom(B=3, T=40, U=6, HA=64, HL=64, H=64, V=128, dtype="bf16", seed=5)
    ns = dict(B=3, T=40, U=6, HA=64, HL=64, H=64, V=128, groups=8, **to_device(inp))
    ns["frames"] = torch.randn(3, 40, 64, device="cuda").bfloat16()
    ns["gamma"], ns["beta"] = torch.ones(64, device="cuda"), torch.zeros(64, device="cuda")
    ns["row_scale"], ns["row_shift"] = ns["gamma"].clone(), ns["beta"].clone()
    ns["table"] = torch.randn(128, 64, device="cuda").bfloat16() / 8
    before = ns["table"].clone(), ns["WO"].clone()
    for block in blocks:
        exec(compile(block, "README.md", "exec"), ns)
    torch.cuda.synchronize()
    assert bool(torch.isfinite(ns["loss"]).all())
    assert ns["adamw"].steps.tolist() == [1, 0]
    for master, low, old in zip(ns["weights"], (ns["WO"], ns["table"]), before[::-1]):
        assert torch.equal(low, master.bfloat16()) and not torch.equal(low, old)
    assert all(ns[k].status() == (0, 0) for k in ("r", "norm", "embed", "rows", "orth"))
