"""The example that trains a small output layer with every loss over rows of
logits: each loss falls."""
import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_every_loss_falls():
    spec = importlib.util.spec_from_file_location(
        "train_head", os.path.join(ROOT, "examples", "train_head.py"))
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    history = example.main(steps=8)
    assert list(history) == ["distillation", "policy", "preference", "likelihood"]
    for name, losses in history.items():
        assert all(l == l and abs(l) < 1e6 for l in losses), (name, losses)
        assert losses[-1] < losses[0], (name, losses)
