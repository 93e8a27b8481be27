"""The example that tunes several tenants' adapters at once: that it runs, what it returns, and that every adapter has learnt something."""

import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_example_runs():
    spec = importlib.util.spec_from_file_location("tune_adapters", os.path.join(ROOT, "examples", "tune_adapters.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    losses, (A, B), words = mod.main(["--tenants", "3", "--tokens", "40", "--prompt", "7", "--hidden", "128", "--words", "640", "--rank",
                                      "8", "--steps", "3"])
    assert len(losses) == 3 and all(l > 0 for l in losses)
    assert A.grad.shape == A.shape and B.grad.shape == B.shape
    assert torch.isfinite(A).all() and torch.isfinite(B).all()
    for a in range(3):     # B starts at 0 and every tenant has tokens with a target
        assert B.grad[a].any() and A.grad[a].any() and B[a].any()
    assert words.shape == (4,) and 0 <= words.min() and words.max() < 640
