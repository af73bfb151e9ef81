"""The vocabulary losses' kernels access rows of logits and gradients through the row's own
functions, which the bounds-checked build tests (a row's ragged ends test each element in
both builds)."""

import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "newton_schulz_orthogonalized_gb300", "csrc")


@pytest.mark.parametrize("name", ["vocab_logprobs.cu", "vocab_distill.cu"])
def test_no_element_is_accessed_past_the_checks(name):
    with open(os.path.join(CSRC, name)) as f:
        lines = f.read().splitlines()
    bare = [f"{name}:{n}: {line.strip()}" for n, line in enumerate(lines, 1) if re.search(r"\b(row|out|later)\.p\b", line)]
    assert not bare, bare
