"""The example serves a model step by step (prompts, fork, CUDA graph replays,
slots cleared and compacted) and gets what whole prompts give."""
from __future__ import annotations

import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_serving_example():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from mamba2_ssm_decode_gb300 import build
    build.build()
    spec = importlib.util.spec_from_file_location("serve_layers",
                                                  os.path.join(ROOT, "examples", "serve_layers.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    # bf16 activations (2^-8 a rounding, a dozen roundings a layer and step) against another
    # order of the same sums
    assert m.main() < 0.03
