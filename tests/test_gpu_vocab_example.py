"""examples/distill_finetune.py: the losses and the optimizer step together make a student
follow its teacher."""

import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.parametrize("loss", ["distill", "ce"])
def test_the_example_learns(loss, capsys):
    spec = importlib.util.spec_from_file_location("distill_finetune", os.path.join(ROOT, "examples", "distill_finetune.py"))
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    history = example.main(["--steps", "40", "--loss", loss, "--vocab", "1501"])
    assert "step" in capsys.readouterr().out
    first, last = history[0], history[-1]
    # the loss falls, and the teacher's tokens become likelier under the student
    assert last[0] < first[0] - 0.1
    assert last[1] > first[1] + 0.1
