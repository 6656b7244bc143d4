"""The example that runs the losses and the shard step together: the student
learns what the teacher recorded."""
import os
import sys

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_distill_example_learns():
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    try:
        import distill
    finally:
        sys.path.pop(0)
    lines = []
    first, last, before, after = distill.main(steps=40, log=lines.append)
    assert last < 0.8 * first, lines
    assert after > before + 0.3, lines
