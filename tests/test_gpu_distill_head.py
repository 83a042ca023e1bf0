"""examples/distill_head.py: the norm, the quantizers, the products of a layer and
the distillation loss run together as one training step."""
import importlib.util
import os

import pytest

from gpuhelp import say

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_student_learns():
    spec = importlib.util.spec_from_file_location("distill_head", os.path.join(ROOT, "examples", "distill_head.py"))
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    say("distill_head")
    losses = example.train(steps=12, tokens=512, hidden=512, vocab=2048, say=say)
    assert all(b < a for a, b in zip(losses, losses[1:]))
    again = example.train(steps=3, tokens=512, hidden=512, vocab=2048, say=say)
    assert again == losses[:3]
