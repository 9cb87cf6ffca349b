"""The training operators together, as the example runs them: the loss falls and the drafts
that the trained head makes are accepted."""
import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_training_a_head_makes_its_drafts_hold():
    spec = importlib.util.spec_from_file_location(
        "train_head", os.path.join(ROOT, "examples", "train_head.py"))
    ex = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(ex)
    first, last, before, after = ex.train(steps=300, log=None)
    assert first > 5.0 and last < 0.5 * first
    assert before < 1.0 and after > 6.0
