"""The example of the decayed layer: prompt, single tokens and training run together."""
import importlib.util
import os

import pytest
import torch

from preconditioned_delta_rule_phase1_gb300 import build as osdn_build

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_example_runs():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    osdn_build.build()
    spec = importlib.util.spec_from_file_location("decayed_layer", os.path.join(ROOT, "examples", "decayed_layer.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    off, loss, status = m.main()
    assert status == 0
    # two ways of rounding the same bf16 activations, a few operations deep
    assert off < 3e-2
    assert loss[-1] < loss[0]
